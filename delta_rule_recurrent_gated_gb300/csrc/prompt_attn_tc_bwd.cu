// prompt_attn_tc_bwd.cu -- gradient of causal attention over whole prompts, bf16: the products on the
// fifth-generation tensor cores (dr.h, dr_prompt_attn_bwd).
//
//   p_ij = e^{s_ij - lse_i};  ds_ij = p_ij (dO_i.v_j - D_i);
//   dq_i = scale sum_j ds_ij k_j;   dk_j = scale sum_i ds_ij q_i;   dv_j = sum_i p_ij dO_i
//
// Two kernels, so that every sum has one owner: no atomics, no fp32 image of a gradient in memory, the same
// bits every time.  They form S and dP = dO V^T twice, 7 products where 5 would do.
//   dq:     256 queries of a head, two halves of 128, against 64 keys a stage:
//           S = Q K^T, dP = dO V^T, dQ += dS K.  The halves take turns, as in the forward kernel.
//   dk, dv: 128 keys of a key head, against 64 queries a stage of all query heads that read it, one after another:
//           S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  S^T and dP^T have two buffers, used in turn by
//           the two groups of four warps.
// P and dS go over the columns of their scores as bf16 operands in tensor memory; they never are in shared memory.
#include "f32x2.cuh"
#include "prompt_attn.cuh"
#include "tc_block.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kRows = 128, kStage = 64, kThreads = 384, kInfos = 4;
constexpr int kRegs = 168, kRowRegs = 208, kOtherRegs = 88;  // of a thread: as launched, of the rows' threads, of the others
static_assert(256 * kRowRegs + (kThreads - 256) * kOtherRegs <= kThreads * kRegs, "more than the block has");
constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ uint32_t s_col(int b) { return 64 * b; }        // of half or buffer b
__device__ __forceinline__ uint32_t dp_col(int b) { return 128 + 64 * b; }
__device__ __forceinline__ uint32_t acc_col(int b) { return 256 + 128 * b; }  // dQ of half b; dV, dK

// Rounds run through the blocks forwards and backwards in turn: who gets a round's longer items gets the next one's shorter.
__device__ __forceinline__ long long place(long long k) {
    return k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// 128 rows of a head: four 64-channel column blocks at most.
template <int D> constexpr int kRowTile = kRows * D * 2;
template <int D> constexpr int kStageTile = kStage * D * 2;

// D[128 x 64] = A[128 x d] B[64 x d]^T, both in shared memory.
template <int D> __device__ __forceinline__ void scores(uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
    for (int kk = 0; kk < D; kk += 16)
        mma_bf16(d, a + (kk >> 6) * (kRows * 128 / 16) + (kk & 63) / 8, b + (kk >> 6) * (kStage * 128 / 16) + (kk & 63) / 8,
                 idesc_bf16(kRows, kStage), kk > 0);
}
// D[128 x d] (+)= A[128 x 64] (tensor memory) B[64 x d].
template <int D> __device__ __forceinline__ void gather(uint32_t d, uint32_t a, uint64_t b, bool add) {
#pragma unroll
    for (int kk = 0; kk < kStage; kk += 16) mma_ts(d, a + kk / 2, b + kk * 8, idesc_bf16(kRows, D, false, true), add || kk > 0);
}
// One accumulator row, times f, as bf16.
template <int D> __device__ __forceinline__ void store_row(uint32_t from, __nv_bfloat16* to, float f, bool on) {
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        float y[32];
        tmem_ld32(from + c, y);
        tmem_ld_wait();
        if (on)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                reinterpret_cast<uint4*>(to + c)[q] =
                    make_uint4(pack_bf16(y[8 * q] * f, y[8 * q + 1] * f), pack_bf16(y[8 * q + 2] * f, y[8 * q + 3] * f),
                               pack_bf16(y[8 * q + 4] * f, y[8 * q + 5] * f), pack_bf16(y[8 * q + 6] * f, y[8 * q + 7] * f));
    }
    tc_fence_before();
}
// A tile of 64 rows whose first `rows` belong to the sequence: zeros behind them.
template <int D>
__device__ __forceinline__ bool load_stage(volatile int& dead, uint8_t* tile, const CUtensorMap* map, uint64_t* full,
                                           uint64_t* landed, uint32_t& landings, int head, int row, int rows) {
    const int lane = threadIdx.x & 31;
    uint64_t* bar = rows < kStage ? landed : full;
    if (lane == 0) {
        mbar_arrive_expect_tx(bar, kStageTile<D>);
        load_rows<kStage, D>(tile, map, bar, head, row);
    }
    __syncwarp();
    if (rows < kStage) {
        if (!wait(dead, landed, landings++ & 1)) return false;
        clear_rows<kStage, D>(tile, rows);
        if (lane == 0) mbar_arrive(full);
        __syncwarp();
    }
    return true;
}

// ================================================================== dq
namespace dq {
constexpr int kTile = 2 * kRows, kBuffers = 3;
struct Item {
    int any, row0, len, head, i0;
    int lo[2], hi[2];  // stages of each half (none: lo >= hi)
};
struct Control {
    uint64_t qfull, qempty, kfull[kBuffers], kempty[kBuffers], vfull[kBuffers], vempty[kBuffers], landed;
    uint64_t sfull[2], pfull[2], done[2], drained;
    uint32_t tmem;
    volatile int dead;
    Item item[kInfos];
};
template <int D> struct Smem {
    static constexpr int q = 0, g = 2 * kRowTile<D>, k = 2 * g, v = k + kBuffers * kStageTile<D>,
                         control = v + kBuffers * kStageTile<D>, bytes = control + 1024;
    static_assert(sizeof(Control) <= 1024, "control block");
};
__device__ __forceinline__ Item make_item(const PromptParams& p, long long k) {
    const long long at = place(k);
    Item x = {};
    int seq = 0, tile = 0;
    x.any = find_tile(p.s, kTile, at / p.Hq, seq, tile);
    if (!x.any) return x;
    x.head = (int)(at % p.Hq);
    seq_rows(p.s, seq, x.row0, x.len);
    x.i0 = tile * kTile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int first = x.i0 + h * kRows, end = min(first + kRows, x.len);
        x.lo[h] = p.window ? max(0, first - p.window + 1) / kStage : 0;
        x.hi[h] = first < x.len ? (end + kStage - 1) / kStage : x.lo[h];
    }
    return x;
}
__device__ __forceinline__ int last_stage(const Item& x) { return max(x.hi[0], x.hi[1]); }  // one behind

template <int D>
__device__ __forceinline__ void copy_tiles(const PromptParams& p, const CUtensorMap* mq, const CUtensorMap* mg,
                                           const CUtensorMap* mk, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t n = 0, landings = 0;
    for (long long k = 0;; ++k) {
        const Item x = make_item(p, k);
        if (!wait(ct.dead, &ct.qempty, (k & 1) ^ 1)) return;
        if (lane == 0) {
            ct.item[k % kInfos] = x;
            if (x.any) {
                mbar_arrive_expect_tx(&ct.qfull, 4 * kRowTile<D>);
                for (int h = 0; h < 2; ++h) {
                    const int row = x.row0 + x.i0 + h * kRows;
                    load_rows<kRows, D>(smem + Smem<D>::q + h * kRowTile<D>, mq, &ct.qfull, x.head, row);
                    load_rows<kRows, D>(smem + Smem<D>::g + h * kRowTile<D>, mg, &ct.qfull, x.head, row);
                }
            } else {
                mbar_arrive(&ct.qfull);
            }
        }
        __syncwarp();
        if (!x.any) return;
        const int hk = x.head / p.G;
        for (int t = x.lo[0]; t < last_stage(x); ++t, ++n) {
            const uint32_t buf = n % kBuffers, parity = (n / kBuffers) & 1;
            const int row = x.row0 + t * kStage;
            if (!wait(ct.dead, &ct.kempty[buf], parity ^ 1)) return;
            // keys behind the sequence are summed with a weight of zero: they have to be numbers
            if (!load_stage<D>(ct.dead, smem + Smem<D>::k + buf * kStageTile<D>, mk, &ct.kfull[buf], &ct.landed, landings, hk,
                               row, x.len - t * kStage))
                return;
            if (!wait(ct.dead, &ct.vempty[buf], parity ^ 1)) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(&ct.vfull[buf], kStageTile<D>);
                load_rows<kStage, D>(smem + Smem<D>::v + buf * kStageTile<D>, mv, &ct.vfull[buf], hk, row);
            }
            __syncwarp();
        }
    }
}

template <int D> __device__ __forceinline__ void issue(uint8_t* smem, Control& ct) {
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    const uint64_t q0 = desc_kmajor(Tile{base + Smem<D>::q, kRows}, 0), g0 = desc_kmajor(Tile{base + Smem<D>::g, kRows}, 0);
    const uint64_t k0 = desc_kmajor(Tile{base + Smem<D>::k, kStage}, 0), v0 = desc_kmajor(Tile{base + Smem<D>::v, kStage}, 0);
    const uint64_t kt0 = desc_mnmajor(Tile{base + Smem<D>::k, kStage}, 0);
    uint32_t n = 0, np[2] = {0, 0};  // stages whose dQ was issued
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.qfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        if (!x.any) return;
        const int first = x.lo[0], last = last_stage(x);
        for (int t = first - 1; t < last; ++t) {
            const uint32_t next = t < first ? n : n + 1, nb = next % kBuffers, b = n % kBuffers;
            if (t + 1 < last) {
                if (!wait(ct.dead, &ct.kfull[nb], (next / kBuffers) & 1) || !wait(ct.dead, &ct.vfull[nb], (next / kBuffers) & 1))
                    return;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool sum = t >= x.lo[h] && t < x.hi[h], qk = t + 1 >= x.lo[h] && t + 1 < x.hi[h];
                if (sum) {
                    if (!wait(ct.dead, &ct.pfull[h], np[h]++ & 1)) return;
                    tc_fence_after();
                }
                if (elect_one()) {
                    if (sum) {
                        gather<D>(tm + acc_col(h), tm + s_col(h), kt0 + b * (kStageTile<D> >> 4), t > x.lo[h]);
                        if (t + 1 == x.hi[h]) mma_commit(&ct.done[h]);
                    }
                    if (qk) {
                        scores<D>(tm + s_col(h), q0 + h * (kRowTile<D> >> 4), k0 + nb * (kStageTile<D> >> 4));
                        scores<D>(tm + dp_col(h), g0 + h * (kRowTile<D> >> 4), v0 + nb * (kStageTile<D> >> 4));
                        mma_commit(&ct.sfull[h]);
                    }
                }
                __syncwarp();
            }
            if (elect_one()) {
                if (t >= first) mma_commit(&ct.kempty[b]);
                if (t + 1 < last) mma_commit(&ct.vempty[nb]);
                if (t + 2 == last) mma_commit(&ct.qempty);
            }
            __syncwarp();
            if (t >= first) ++n;
        }
    }
}

template <int D> __device__ __forceinline__ void rows(const PromptParams& p, Control& ct) {
    const int h = threadIdx.x / kRows, r = threadIdx.x % kRows;
    const uint32_t tm = warp_lane_base(ct.tmem), ts = tm + s_col(h), td = tm + dp_col(h);
    const float c2 = p.scale * kLog2e;
    uint32_t n = 0, done = 0;
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.qfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        warp_arrive(&ct.qempty);
        if (!x.any) return;
        const int lo = h ? x.lo[1] : x.lo[0], hi = h ? x.hi[1] : x.hi[0];
        if (lo >= hi) continue;
        const int pos = x.i0 + h * kRows + r, w0 = pos & ~31;
        const bool on = pos < x.len;
        const size_t at = (size_t)(x.row0 + pos) * p.Hq + x.head;
        const float lse = on ? p.lse[at] * -kLog2e : 0.f, delta = on ? -p.delta[at] : 0.f;
        for (int t = lo; t < hi; ++t, ++n) {
            const int j0 = t * kStage;
            if (!wait(ct.dead, &ct.sfull[h], n & 1)) return;
            tc_fence_after();
            float s[kStage], d[kStage];
            tmem_ld32(ts, s);
            tmem_ld32(ts + 32, s + 32);
            tmem_ld32(td, d);
            tmem_ld32(td + 32, d + 32);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kStage; j += 2) {
                float2 z = fma2(make_float2(s[j], s[j + 1]), both(c2), both(lse));
                z = make_float2(ex2(z.x), ex2(z.y));
                z = mul2(z, add2(make_float2(d[j], d[j + 1]), both(delta)));
                s[j] = z.x;
                s[j + 1] = z.y;
            }
            if (j0 + kStage - 1 > w0 || (p.window && j0 <= w0 + 31 - p.window)) {
                const int up = pos - j0, down = p.window ? up - p.window : -1;
#pragma unroll
                for (int j = 0; j < kStage; ++j) s[j] = j <= up && j > down ? s[j] : 0.f;
            }
            uint32_t z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
            tmem_st32(ts, z);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&ct.pfull[h]);
        }
        if (!wait(ct.dead, &ct.done[h], done++ & 1)) return;
        tc_fence_after();
        store_row<D>(tm + acc_col(h), static_cast<__nv_bfloat16*>(p.dq) + (x.row0 + pos) * p.ld_dq + (long long)x.head * D, p.scale, on);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_dq_tc_kernel(const PromptParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                        const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ct = *reinterpret_cast<Control*>(smem + Smem<D>::control);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(&ct.qfull, 1);
        mbar_init(&ct.qempty, 1 + 8);
        mbar_init(&ct.landed, 1);
        mbar_init(&ct.drained, 1);
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&ct.kfull[i], 1);
            mbar_init(&ct.kempty[i], 1);
            mbar_init(&ct.vfull[i], 1);
            mbar_init(&ct.vempty[i], 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&ct.sfull[h], 1);
            mbar_init(&ct.pfull[h], 4);
            mbar_init(&ct.done[h], 1);
        }
        ct.dead = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        rows<D>(p, ct);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) issue<D>(smem, ct), drain(&ct.drained);
        else if (warp == 9) copy_tiles<D>(p, &mq, &mg, &mk, &mv, smem, ct);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ct.dead && threadIdx.x == 0 && p.status) *reinterpret_cast<volatile int32_t*>(p.status) = kErrTimeout;
    if (warp == 0) tmem_dealloc(ct.tmem, 512);
}
}  // namespace dq

// ================================================================== dk, dv
namespace dkv {
constexpr int kBuffers = 4;
struct Item {
    int any, row0, len, head, j0;  // head: of the keys
    int lo, hi;                    // query stages of each query head
};
struct Control {
    uint64_t kvfull, kvempty, full[kBuffers], empty[kBuffers], landed;
    uint64_t sfull[2], pfull[2], done, left, drained;
    uint32_t tmem;
    volatile int dead;
    Item item[kInfos];
    __align__(16) float lse[kBuffers][kStage], delta[kBuffers][kStage];  // negative, lse in base 2
};
template <int D> struct Smem {
    static constexpr int k = 0, v = kRowTile<D>, q = 2 * v, g = q + kBuffers * kStageTile<D>,
                         control = g + kBuffers * kStageTile<D>, bytes = control + 3072;
    static_assert(sizeof(Control) <= 3072, "control block");
};
// Items in the order of the sequences, the first keys first, which have the most queries: the blocks that run at the same
// time then read the same queries.  (All first keys of all sequences first, as in the other kernels, and eight
// sequences of 4096 tokens have 268 MB of them in use, more than L2.)
__device__ __forceinline__ Item make_item(const PromptParams& p, long long k) {
    const long long at = k * gridDim.x + blockIdx.x;
    Item x = {};
    int seq = 0, tile = 0, tiles;
    long long slot;
    x.any = find_tile_in_order(p.s, kRows, 0, at / p.H, seq, tile, tiles, slot);
    if (!x.any) return x;
    x.head = (int)(at % p.H);
    seq_rows(p.s, seq, x.row0, x.len);
    x.j0 = tile * kRows;
    x.lo = x.j0 / kStage;
    const int end = p.window ? (int)min((long long)x.len, (long long)min(x.j0 + kRows, x.len) - 1 + p.window) : x.len;
    x.hi = (end + kStage - 1) / kStage;
    return x;
}

// Warp 9: tiles.  Warp 10: the rows' lse and D, the next stage's already on their way.
template <int D>
__device__ __forceinline__ void copy_tiles(const PromptParams& p, const CUtensorMap* mq, const CUtensorMap* mg,
                                           const CUtensorMap* mk, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t n = 0, landings = 0;
    for (long long k = 0;; ++k) {
        const Item x = make_item(p, k);
        if (!wait(ct.dead, &ct.kvempty, (k & 1) ^ 1)) return;
        if (lane == 0) {
            ct.item[k % kInfos] = x;
            if (x.any) {  // rows of no key get no result, so that they may be anything
                mbar_arrive_expect_tx(&ct.kvfull, 2 * kRowTile<D>);
                load_rows<kRows, D>(smem + Smem<D>::k, mk, &ct.kvfull, x.head, x.row0 + x.j0);
                load_rows<kRows, D>(smem + Smem<D>::v, mv, &ct.kvfull, x.head, x.row0 + x.j0);
            } else {
                mbar_arrive(&ct.kvfull);
            }
        }
        __syncwarp();
        if (!x.any) return;
        for (int h = x.head * p.G; h < (x.head + 1) * p.G; ++h)
            for (int t = x.lo; t < x.hi; ++t, ++n) {
                const uint32_t buf = n % kBuffers;
                if (!wait(ct.dead, &ct.empty[buf], ((n / kBuffers) & 1) ^ 1)) return;
                if (!load_stage<D>(ct.dead, smem + Smem<D>::q + buf * kStageTile<D>, mq, &ct.full[buf], &ct.landed, landings, h,
                                   x.row0 + t * kStage, x.len - t * kStage) ||
                    !load_stage<D>(ct.dead, smem + Smem<D>::g + buf * kStageTile<D>, mg, &ct.full[buf], &ct.landed, landings, h,
                                   x.row0 + t * kStage, x.len - t * kStage))
                    return;
            }
    }
}
__device__ __forceinline__ void copy_stats(const PromptParams& p, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    for (long long k = 0;; ++k) {
        const Item x = make_item(p, k);
        if (!x.any) return;
        const int stages = x.hi - x.lo, total = stages * p.G;
        auto read = [&](int i, float (&l)[2], float (&d)[2]) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int pos = (x.lo + i % stages) * kStage + lane + 32 * j;
                const bool on = i < total && pos < x.len;
                const size_t at = on ? (size_t)(x.row0 + pos) * p.Hq + x.head * p.G + i / stages : 0;
                l[j] = on ? p.lse[at] * -kLog2e : -INFINITY;  // no query: no weight
                d[j] = on ? -p.delta[at] : 0.f;
            }
        };
        float l[2], d[2];
        read(0, l, d);
        for (int i = 0; i < total; ++i, ++n) {
            const uint32_t buf = n % kBuffers;
            float l2[2], d2[2];
            read(i + 1, l2, d2);
            if (!wait(ct.dead, &ct.empty[buf], ((n / kBuffers) & 1) ^ 1)) return;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ct.lse[buf][lane + 32 * j] = l[j];
                ct.delta[buf][lane + 32 * j] = d[j];
                l[j] = l2[j];
                d[j] = d2[j];
            }
            warp_arrive(&ct.full[buf]);
        }
    }
}

template <int D> __device__ __forceinline__ void issue(const PromptParams& p, uint8_t* smem, Control& ct) {
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    const uint64_t k0 = desc_kmajor(Tile{base + Smem<D>::k, kRows}, 0), v0 = desc_kmajor(Tile{base + Smem<D>::v, kRows}, 0);
    const uint64_t q0 = desc_kmajor(Tile{base + Smem<D>::q, kStage}, 0), g0 = desc_kmajor(Tile{base + Smem<D>::g, kStage}, 0);
    const uint64_t qt0 = desc_mnmajor(Tile{base + Smem<D>::q, kStage}, 0), gt0 = desc_mnmajor(Tile{base + Smem<D>::g, kStage}, 0);
    uint32_t n = 0;
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.kvfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        if (!x.any) return;
        const int total = (x.hi - x.lo) * p.G;
        for (int i = -1; i < total; ++i) {
            const uint32_t next = i < 0 ? n : n + 1, nb = next % kBuffers, b = n % kBuffers;
            if (i + 1 < total) {
                if (!wait(ct.dead, &ct.full[nb], (next / kBuffers) & 1)) return;
                tc_fence_after();
                if (elect_one()) {  // over the operands of stage next - 2, whose products were issued before
                    scores<D>(tm + s_col(next & 1), k0, q0 + nb * (kStageTile<D> >> 4));
                    scores<D>(tm + dp_col(next & 1), v0, g0 + nb * (kStageTile<D> >> 4));
                    mma_commit(&ct.sfull[next & 1]);
                    mbar_arrive(&ct.sfull[next & 1]);  // hands on the rows' lse and D, which came with `full`
                    if (i + 2 == total) mma_commit(&ct.kvempty);
                }
                __syncwarp();
            }
            if (i < 0) {
                if (!wait(ct.dead, &ct.left, (k & 1) ^ 1)) return;  // the sums of the item before have been read
                continue;
            }
            if (!wait(ct.dead, &ct.pfull[n & 1], (n >> 1) & 1)) return;
            tc_fence_after();
            if (elect_one()) {
                gather<D>(tm + acc_col(0), tm + s_col(n & 1), gt0 + b * (kStageTile<D> >> 4), i > 0);
                gather<D>(tm + acc_col(1), tm + dp_col(n & 1), qt0 + b * (kStageTile<D> >> 4), i > 0);
                mma_commit(&ct.empty[b]);
                if (i + 1 == total) mma_commit(&ct.done);
            }
            __syncwarp();
            ++n;
        }
    }
}

template <int D> __device__ __forceinline__ void rows(const PromptParams& p, Control& ct) {
    const int grp = threadIdx.x / kRows, r = threadIdx.x % kRows;
    const uint32_t tm = warp_lane_base(ct.tmem), ts = tm + s_col(grp), td = tm + dp_col(grp);
    const float c2 = p.scale * kLog2e;
    uint32_t n = 0;
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.kvfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        warp_arrive(&ct.kvempty);
        if (!x.any) return;
        const int stages = x.hi - x.lo, total = stages * p.G, pos = x.j0 + r, w0 = pos & ~31;
        for (int i = 0; i < total; ++i, ++n) {
            if ((n & 1) != (uint32_t)grp) continue;
            const int i0 = (x.lo + i % stages) * kStage;
            if (!wait(ct.dead, &ct.sfull[grp], (n >> 1) & 1)) return;
            tc_fence_after();
            const float4* lse = reinterpret_cast<const float4*>(ct.lse[n % kBuffers]);
            const float4* delta = reinterpret_cast<const float4*>(ct.delta[n % kBuffers]);
            float s[kStage], d[kStage];
            tmem_ld32(ts, s);
            tmem_ld32(ts + 32, s + 32);
            tmem_ld32(td, d);
            tmem_ld32(td + 32, d + 32);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kStage; j += 4) {
                const float4 l = lse[j / 4];
                float2 z = fma2(make_float2(s[j], s[j + 1]), both(c2), make_float2(l.x, l.y));
                float2 y = fma2(make_float2(s[j + 2], s[j + 3]), both(c2), make_float2(l.z, l.w));
                s[j] = ex2(z.x);
                s[j + 1] = ex2(z.y);
                s[j + 2] = ex2(y.x);
                s[j + 3] = ex2(y.y);
            }
            const bool masked = i0 < w0 + 31 || (p.window && i0 + kStage - 1 >= w0 + p.window);
            const int from = pos - i0, upto = p.window ? from + p.window : kStage;  // queries that see this key
            if (masked)
#pragma unroll
                for (int j = 0; j < kStage; ++j) s[j] = j >= from && j < upto ? s[j] : 0.f;
            uint32_t z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
            tmem_st32(ts, z);
#pragma unroll
            for (int j = 0; j < kStage; j += 4) {
                const float4 e = delta[j / 4];
                const float2 a = mul2(make_float2(s[j], s[j + 1]), add2(make_float2(d[j], d[j + 1]), make_float2(e.x, e.y)));
                const float2 b = mul2(make_float2(s[j + 2], s[j + 3]), add2(make_float2(d[j + 2], d[j + 3]), make_float2(e.z, e.w)));
                d[j] = a.x; d[j + 1] = a.y; d[j + 2] = b.x; d[j + 3] = b.y;
            }
            if (masked)  // a weight of zero times what is not finite is no zero
#pragma unroll
                for (int j = 0; j < kStage; ++j) d[j] = j >= from && j < upto ? d[j] : 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = pack_bf16(d[2 * j], d[2 * j + 1]);
            tmem_st32(td, z);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&ct.pfull[grp]);
        }
        if (!wait(ct.dead, &ct.done, k & 1)) return;
        tc_fence_after();
        const bool on = pos < x.len;
        if (grp == 0)
            store_row<D>(tm + acc_col(0), static_cast<__nv_bfloat16*>(p.dv) + (x.row0 + pos) * p.ld_dv + (long long)x.head * D, 1.f, on);
        else
            store_row<D>(tm + acc_col(1), static_cast<__nv_bfloat16*>(p.dk) + (x.row0 + pos) * p.ld_dk + (long long)x.head * D, p.scale, on);
        warp_arrive(&ct.left);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_dkv_tc_kernel(const PromptParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                         const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ct = *reinterpret_cast<Control*>(smem + Smem<D>::control);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(&ct.kvfull, 1);
        mbar_init(&ct.kvempty, 1 + 8);
        mbar_init(&ct.landed, 1);
        mbar_init(&ct.drained, 1);
        mbar_init(&ct.done, 1);
        mbar_init(&ct.left, 8);
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&ct.full[i], 3);  // queries, gradients, statistics
            mbar_init(&ct.empty[i], 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&ct.sfull[h], 2);
            mbar_init(&ct.pfull[h], 4);
        }
        ct.dead = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        rows<D>(p, ct);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) issue<D>(p, smem, ct), drain(&ct.drained);
        else if (warp == 9) copy_tiles<D>(p, &mq, &mg, &mk, &mv, smem, ct);
        else if (warp == 10) copy_stats(p, ct);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ct.dead && threadIdx.x == 0 && p.status) *reinterpret_cast<volatile int32_t*>(p.status) = kErrTimeout;
    if (warp == 0) tmem_dealloc(ct.tmem, 512);
}
}  // namespace dkv

// The split of the registers must not ask for more than the block is launched with: it would wait for them.
template <typename K> bool fits(K kernel) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) == cudaSuccess && a.numRegs == kRegs;
}

template <int D> cudaError_t launch(const PromptParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready[2] = {};
    static const bool fit = fits(dq::prompt_dq_tc_kernel<D>) && fits(dkv::prompt_dkv_tc_kernel<D>);
    if (!fit) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = set_smem_once(dq::prompt_dq_tc_kernel<D>, dq::Smem<D>::bytes, ready[0]); e != cudaSuccess) return e;
    if (cudaError_t e = set_smem_once(dkv::prompt_dkv_tc_kernel<D>, dkv::Smem<D>::bytes, ready[1]); e != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    auto blocks = [&](long long items) { return (int)(items < sms ? items : sms); };
    const long long ld_g = (long long)p.Hq * D;
    auto maps = [&](CUtensorMap (&m)[4], int own, int other) {  // boxes of `own` query rows and `other` key rows
        return head_rows_map(&m[0], p.q, D, p.Hq, p.rows, p.ld_q, own) && head_rows_map(&m[1], p.dO, D, p.Hq, p.rows, ld_g, own) &&
               head_rows_map(&m[2], p.k, D, p.H, p.rows, p.ld_k, other) && head_rows_map(&m[3], p.v, D, p.H, p.rows, p.ld_v, other);
    };
    CUtensorMap m[4];
    if (!maps(m, kRows, kStage)) return cudaErrorInvalidValue;
    {
        TraceScope ts("prompt_dq_tc", st);
        dq::prompt_dq_tc_kernel<D><<<blocks(most_tiles(p.s, dq::kTile) * p.Hq), kThreads, dq::Smem<D>::bytes, st>>>(p, m[0], m[1], m[2], m[3]);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    if (!maps(m, kStage, kRows)) return cudaErrorInvalidValue;
    // A block for each item, so that one that is through takes the next in order: 1066 us instead of 1425 with a block for
    // each SM and its items dealt out beforehand (b8 t4096, 16 heads of 128, four of keys).
    const long long keys = most_tiles(p.s, kRows) * p.H;
    if (keys >= (1ll << 31)) return cudaErrorInvalidValue;
    TraceScope ts("prompt_dkv_tc", st);
    dkv::prompt_dkv_tc_kernel<D><<<(unsigned)keys, kThreads, dkv::Smem<D>::bytes, st>>>(p, m[0], m[1], m[2], m[3]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_attn_bwd_tc(const PromptParams& p, cudaStream_t st) {
    if (cudaError_t e = prompt_attn_delta(p, DR_BF16, st); e != cudaSuccess) return e;
    return p.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace dr
