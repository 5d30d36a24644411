// prompt_attn_tc_bwd.cu -- gradient of causal attention over whole prompts, bf16: the products on the
// fifth-generation tensor cores (dr.h, dr_prompt_attn_bwd).
//
//   p_ij = e^{s_ij - lse_i};  ds_ij = p_ij (dO_i.v_j - D_i);
//   dq_i = scale sum_j ds_ij k_j;   dk_j = scale sum_i ds_ij q_i;   dv_j = sum_i p_ij dO_i
//
// Two kernels, so that every sum has one owner: no atomics, no fp32 image of a gradient in memory, the same
// bits every time.  They form S and dP = dO V^T twice, 7 products where 5 would do.  8 x 4096 tokens, 16 query heads of
// 128, 4 key heads: dq 563 us (1460 TFLOP/s of its own three products), dk and dv 678 us (1620 TFLOP/s of their four),
// bound by the tensor cores and the operands they read from shared memory; D = dO.o before them 49 us.  That is each alone,
// at 2070 MHz; in a stream of passes the power limit brings the clock to 1957 MHz and them to 601, 717 and 50 us.
//   dq:     128 queries of a head, against 128 keys a stage: S = Q K^T, dP = dO V^T, dQ += dS K, issued as
//           S(n + 1), dP(n + 1), dQ(n).  dP has two buffers in tensor memory, and dS takes the place of its dP.
//   dk, dv: 128 keys of a key head, against 128 queries a stage of all query heads that read it, one after another:
//           S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q, issued as dK(n - 1), dP(n), dV(n), S(n + 1), with P
//           and dS in the places of S and dP.
// While the tensor cores are at one product, the row threads prepare the operand of the next.  (Stages of 64 with two
// buffers for everything were slower: a product of 128 x 64 from shared memory takes 61 cycles where 128 x 128
// takes 66.)  P and dS are bf16 operands in tensor memory; they never are in shared memory.
// Warps 0-3 and 4-7: a row per thread, the first and the second 64 columns of a stage.  Warp 8: products, 9: copies,
// 10: the queries' statistics (dk, dv).
#include "f32x2.cuh"
#include "prompt_attn.cuh"
#include "tc_block.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kRows = 128, kThreads = 384, kInfos = 4, kFirst = 3, kSecond = 2;  // buffers of what a stage needs first and last, and of the rest
constexpr int kRegs = 168, kRowRegs = 208, kOtherRegs = 88;  // of a thread: as launched, of the rows' threads, of the others
static_assert(256 * kRowRegs + (kThreads - 256) * kOtherRegs <= kThreads * kRegs, "more than the block has");
constexpr float kLog2e = 1.44269504088896340736f;

// Rounds run through the blocks forwards and backwards in turn: who gets a round's longer items gets the next one's shorter.
__device__ __forceinline__ long long place(long long k) {
    return k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
template <int D> constexpr int kTileBytes = kRows * D * 2;  // 128 rows of a head

// D[128 x 128] = A[128 x d] B[128 x d]^T, both in shared memory.
template <int D> __device__ __forceinline__ void scores(uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
    for (int kk = 0; kk < D; kk += 16) {  // 16 channels: 32 bytes of a 128-byte row
        const uint32_t off = (kk >> 6) * (kRows * 128 / 16) + (kk & 63) / 8;
        mma_bf16(d, a + off, b + off, idesc_bf16(kRows, kRows), kk > 0);
    }
}
// D[128 x d] (+)= A[128 x 128] B[128 x d], A in tensor memory as the two groups of warps leave it: 64 columns in 32, twice.
template <int D> __device__ __forceinline__ void gather(uint32_t d, uint32_t a, uint64_t b, bool add) {
#pragma unroll
    for (int kk = 0; kk < kRows; kk += 16)
        mma_ts(d, a + (kk >> 6) * 64 + (kk & 63) / 2, b + kk * 8, idesc_bf16(kRows, D, false, true), add || kk > 0);
}
// Columns c0 .. c0 + N - 1 of an accumulator row, times f, as bf16.
template <int N> __device__ __forceinline__ void store_row(uint32_t from, __nv_bfloat16* to, float f, bool on) {
#pragma unroll
    for (int c = 0; c < N; c += 32) {
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
// A tile of which the first `rows` rows belong to the sequence; zeros behind them where `clean`.
template <int D>
__device__ __forceinline__ bool load_tile(volatile int& dead, uint8_t* tile, const CUtensorMap* map, uint64_t* full,
                                          uint64_t* landed, uint32_t& landings, int head, int row, int rows, bool clean) {
    const int lane = threadIdx.x & 31;
    const bool cut = clean && rows < kRows;
    uint64_t* bar = cut ? landed : full;
    if (lane == 0) {
        mbar_arrive_expect_tx(bar, kTileBytes<D>);
        load_rows<kRows, D>(tile, map, bar, head, row);
    }
    __syncwarp();
    if (cut) {
        if (!wait(dead, landed, landings++ & 1)) return false;
        clear_rows<kRows, D>(tile, rows);
        if (lane == 0) mbar_arrive(full);
        __syncwarp();
    }
    return true;
}
// 64 fp32 values as bf16 pairs to 32 columns.
__device__ __forceinline__ void store_operand(uint32_t to, const float (&x)[64]) {
    uint32_t z[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
    tmem_st32(to, z);
    tmem_st_wait();
    tc_fence_before();
}

// ================================================================== dq
namespace dq {
constexpr uint32_t kS = 0, kDP = 128, kDQ = 384;  // columns of tensor memory
struct Item {
    int any, row0, len, head, i0, lo, hi;  // lo, hi: stages of keys
};
struct Control {
    uint64_t qfull, qempty, kfull[kFirst], kempty[kFirst], vfull[kSecond], vempty[kSecond], landed;
    uint64_t sfull, sread, dpfull[2], dsfull[2], done, drained;  // [2]: with the buffers of dP
    uint32_t tmem;
    volatile int dead;
    Item item[kInfos];
};
template <int D> struct Smem {
    static constexpr int q = 0, g = kTileBytes<D>, k = 2 * g, v = k + kFirst * kTileBytes<D>, control = v + kSecond * kTileBytes<D>,
                         bytes = control + 1024;
    static_assert(sizeof(Control) <= 1024, "control block");
};
__device__ __forceinline__ Item make_item(const PromptParams& p, long long k) {
    const long long at = place(k);
    Item x = {};
    int seq = 0, tile = 0;
    x.any = find_tile(p.s, kRows, at / p.Hq, seq, tile);
    if (!x.any) return x;
    x.head = (int)(at % p.Hq);
    seq_rows(p.s, seq, x.row0, x.len);
    x.i0 = tile * kRows;
    x.lo = p.window ? max(0, x.i0 - p.window + 1) / kRows : 0;
    x.hi = tile + 1;
    return x;
}

template <int D>
__device__ __forceinline__ void copy_tiles(const PromptParams& p, const CUtensorMap* mq, const CUtensorMap* mg,
                                           const CUtensorMap* mk, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t landings = 0;
    Ring<kFirst> rk;
    Ring<kSecond> rv;
    long long items = 0;
    [&] {
        for (long long k = 0;; ++k) {
            const Item x = make_item(p, k);
            // queries and the item's data: after the last item's products with its queries, and after the row threads
            // have begun with it (so they are never two items behind)
            if (!wait(ct.dead, &ct.qempty, (k & 1) ^ 1)) return;
            if (lane == 0) {
                ct.item[k % kInfos] = x;
                if (x.any) {
                    mbar_arrive_expect_tx(&ct.qfull, 2 * kTileBytes<D>);
                    load_rows<kRows, D>(smem + Smem<D>::q, mq, &ct.qfull, x.head, x.row0 + x.i0);
                    load_rows<kRows, D>(smem + Smem<D>::g, mg, &ct.qfull, x.head, x.row0 + x.i0);
                } else {
                    mbar_arrive(&ct.qfull);
                }
            }
            __syncwarp();
            ++items;
            if (!x.any) return;
            const int hk = x.head / p.G;
            for (int t = x.lo; t < x.hi; ++t) {
                const int row = x.row0 + t * kRows, rows = x.len - t * kRows;
                // keys behind the sequence are summed with a weight of zero: they have to be numbers
                if (!wait(ct.dead, &ct.kempty[rk.at], rk.phase ^ 1) ||
                    !load_tile<D>(ct.dead, smem + Smem<D>::k + rk.at * kTileBytes<D>, mk, &ct.kfull[rk.at], &ct.landed, landings, hk,
                                  row, rows, true))
                    return;
                rk.step();
                if (!wait(ct.dead, &ct.vempty[rv.at], rv.phase ^ 1) ||
                    !load_tile<D>(ct.dead, smem + Smem<D>::v + rv.at * kTileBytes<D>, mv, &ct.vfull[rv.at], &ct.landed, landings, hk,
                                  row, rows, false))
                    return;
                rv.step();
            }
        }
    }();
    settle(&ct.qfull, items);
    settle(&ct.landed, landings);
    settle(rk, ct.kfull);
    settle(rv, ct.vfull);
}

template <int D> __device__ __forceinline__ void issue(uint8_t* smem, Control& ct) {
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    const uint64_t q0 = desc_kmajor(Tile{base + Smem<D>::q, kRows}, 0), g0 = desc_kmajor(Tile{base + Smem<D>::g, kRows}, 0);
    const uint64_t k0 = desc_kmajor(Tile{base + Smem<D>::k, kRows}, 0), v0 = desc_kmajor(Tile{base + Smem<D>::v, kRows}, 0);
    const uint64_t kt0 = desc_mnmajor(Tile{base + Smem<D>::k, kRows}, 0);
    Ring<kFirst> ahead, behind;  // of K: of S and of dQ
    Ring<kSecond> rv;
    uint32_t ns = 0, nq = 0;  // stages whose S, whose dQ was issued
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.qfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        if (!x.any) return;
        for (int t = x.lo; t <= x.hi; ++t) {
            if (t < x.hi) {
                if (!wait(ct.dead, &ct.kfull[ahead.at], ahead.phase) || !wait(ct.dead, &ct.sread, (ns & 1) ^ 1)) return;
                tc_fence_after();
                if (elect_one()) {
                    scores<D>(tm + kS, q0, k0 + ahead.at * (kTileBytes<D> >> 4));
                    mma_commit(&ct.sfull);
                }
                __syncwarp();
                if (!wait(ct.dead, &ct.vfull[rv.at], rv.phase)) return;
                if (elect_one()) {  // over the dS of two stages before, whose dQ was issued
                    scores<D>(tm + kDP + 128 * (ns & 1), g0, v0 + rv.at * (kTileBytes<D> >> 4));
                    mma_commit(&ct.dpfull[ns & 1]);
                    mma_commit(&ct.vempty[rv.at]);
                    if (t + 1 == x.hi) mma_commit(&ct.qempty);
                }
                __syncwarp();
                ahead.step();
                rv.step();
                ++ns;
            }
            if (t > x.lo) {
                if (!wait(ct.dead, &ct.dsfull[nq & 1], (nq >> 1) & 1)) return;
                tc_fence_after();
                if (elect_one()) {
                    gather<D>(tm + kDQ, tm + kDP + 128 * (nq & 1), kt0 + behind.at * (kTileBytes<D> >> 4), t > x.lo + 1);
                    mma_commit(&ct.kempty[behind.at]);
                    if (t == x.hi) mma_commit(&ct.done);
                }
                __syncwarp();
                behind.step();
                ++nq;
            }
        }
    }
}

template <int D> __device__ __forceinline__ void rows(const PromptParams& p, Control& ct) {
    const int grp = threadIdx.x / kRows, r = threadIdx.x % kRows, c0 = 64 * grp;
    const uint32_t tm = warp_lane_base(ct.tmem);
    const float c2 = p.scale * kLog2e;
    uint32_t n = 0;
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.qfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        warp_arrive(&ct.qempty);
        if (!x.any) return;
        const int pos = x.i0 + r, w0 = pos & ~31;
        const bool on = pos < x.len;
        const size_t at = (size_t)(x.row0 + pos) * p.Hq + x.head;
        const float lse = on ? p.lse[at] * -kLog2e : 0.f, delta = on ? -p.delta[at] : 0.f;
        for (int t = x.lo; t < x.hi; ++t, ++n) {
            const int j0 = t * kRows + c0;
            if (!wait(ct.dead, &ct.sfull, n & 1)) return;
            tc_fence_after();
            float s[64];
            tmem_ld32(tm + kS + c0, s);
            tmem_ld32(tm + kS + c0 + 32, s + 32);
            tmem_ld_wait();
            tc_fence_before();
            warp_arrive(&ct.sread);
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
                const float2 z = fma2(make_float2(s[j], s[j + 1]), both(c2), both(lse));
                s[j] = ex2(z.x);
                s[j + 1] = ex2(z.y);
            }
            if (!wait(ct.dead, &ct.dpfull[n & 1], (n >> 1) & 1)) return;
            tc_fence_after();
            const uint32_t td = tm + kDP + 128 * (n & 1) + c0;
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float d[32];
                tmem_ld32(td + c, d);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 z = mul2(make_float2(s[c + j], s[c + j + 1]), add2(make_float2(d[j], d[j + 1]), both(delta)));
                    s[c + j] = z.x;
                    s[c + j + 1] = z.y;
                }
            }
            if (j0 + 63 > w0 || (p.window && j0 <= w0 + 31 - p.window)) {
                const int up = pos - j0, down = p.window ? up - p.window : -1;
#pragma unroll
                for (int j = 0; j < 64; ++j) s[j] = j <= up && j > down ? s[j] : 0.f;
            }
            store_operand(td, s);
            warp_arrive(&ct.dsfull[n & 1]);
        }
        if (!wait(ct.dead, &ct.done, k & 1)) return;
        tc_fence_after();
        constexpr int N = D / 2;  // the groups' shares of the channels
        store_row<N>(tm + kDQ + N * grp, static_cast<__nv_bfloat16*>(p.dq) + (x.row0 + pos) * p.ld_dq + (long long)x.head * D + N * grp,
                     p.scale, on);
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
        for (uint64_t* one : {&ct.qfull, &ct.landed, &ct.sfull, &ct.dpfull[0], &ct.dpfull[1], &ct.done, &ct.drained}) mbar_init(one, 1);
        for (uint64_t* eight : {&ct.sread, &ct.dsfull[0], &ct.dsfull[1]}) mbar_init(eight, 8);
        mbar_init(&ct.qempty, 1 + 8);
        for (int i = 0; i < kFirst; ++i) mbar_init(&ct.kfull[i], 1), mbar_init(&ct.kempty[i], 1);
        for (int i = 0; i < kSecond; ++i) mbar_init(&ct.vfull[i], 1), mbar_init(&ct.vempty[i], 1);
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
constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 384;  // columns of tensor memory
struct Item {
    int any, row0, len, head, j0;  // head: of the keys
    int lo, hi;                    // query stages of each query head
};
struct Control {
    uint64_t kvfull, kvempty, qfull[kFirst], qempty[kFirst], gfull[kSecond], gempty[kSecond], stfull[2], stempty[2], landed;
    uint64_t sfull, pfull, dpfull, dsfull, done, drained;
    uint32_t tmem;
    volatile int dead;
    Item item[kInfos];
    __align__(16) float lse[2][kRows], delta[2][kRows];  // negative, lse in base 2
};
template <int D> struct Smem {
    static constexpr int k = 0, v = kTileBytes<D>, q = 2 * v, g = q + kFirst * kTileBytes<D>, control = g + kSecond * kTileBytes<D>,
                         bytes = control + 3 * 1024;
    static_assert(sizeof(Control) <= 3 * 1024, "control block");
};
// Dense batches in the order of the sequences, the first keys first, which have the most queries: the blocks that run at
// the same time then read the same queries (all first keys of all sequences first, and eight sequences of 4096 tokens
// have 268 MB of them in use, more than L2).  Packed ones, whose lengths may be far apart, the longest work first: one
// document of 16384 tokens before four short ones 1269 us, 1420 in their order; eight of 4096, 694 and 680.
__device__ __forceinline__ Item make_item(const PromptParams& p, long long k) {
    const long long at = k * gridDim.x + blockIdx.x;
    Item x = {};
    int seq = 0, tile = 0, tiles;
    long long slot;
    if (p.s.cu) {
        x.any = find_tile(p.s, kRows, at / p.H, seq, tile);
        if (!x.any) return x;
        seq_rows(p.s, seq, x.row0, x.len);
        tile = (x.len + kRows - 1) / kRows - 1 - tile;
    } else {
        x.any = find_tile_in_order(p.s, kRows, 0, at / p.H, seq, tile, tiles, slot);
        if (!x.any) return x;
        seq_rows(p.s, seq, x.row0, x.len);
    }
    x.head = (int)(at % p.H);
    x.j0 = tile * kRows;
    x.lo = tile;
    const int end = p.window ? (int)min((long long)x.len, (long long)min(x.j0 + kRows, x.len) - 1 + p.window) : x.len;
    x.hi = (end + kRows - 1) / kRows;
    return x;
}

template <int D>
__device__ __forceinline__ void copy_tiles(const PromptParams& p, const CUtensorMap* mq, const CUtensorMap* mg,
                                           const CUtensorMap* mk, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t landings = 0;
    Ring<kFirst> rq;
    Ring<kSecond> rg;
    long long items = 0;
    [&] {
        for (long long k = 0;; ++k) {
            const Item x = make_item(p, k);
            if (!wait(ct.dead, &ct.kvempty, (k & 1) ^ 1)) return;
            if (lane == 0) {
                ct.item[k % kInfos] = x;
                if (x.any) {  // rows of no key get no result, so that they may be anything
                    mbar_arrive_expect_tx(&ct.kvfull, 2 * kTileBytes<D>);
                    load_rows<kRows, D>(smem + Smem<D>::k, mk, &ct.kvfull, x.head, x.row0 + x.j0);
                    load_rows<kRows, D>(smem + Smem<D>::v, mv, &ct.kvfull, x.head, x.row0 + x.j0);
                } else {
                    mbar_arrive(&ct.kvfull);
                }
            }
            __syncwarp();
            ++items;
            if (!x.any) return;
            for (int h = x.head * p.G; h < (x.head + 1) * p.G; ++h)
                for (int t = x.lo; t < x.hi; ++t) {
                    // queries behind the sequence are summed with weights of zero: they have to be numbers
                    const int row = x.row0 + t * kRows, rows = x.len - t * kRows;
                    if (!wait(ct.dead, &ct.qempty[rq.at], rq.phase ^ 1) ||
                        !load_tile<D>(ct.dead, smem + Smem<D>::q + rq.at * kTileBytes<D>, mq, &ct.qfull[rq.at], &ct.landed, landings, h,
                                      row, rows, true))
                        return;
                    rq.step();
                    if (!wait(ct.dead, &ct.gempty[rg.at], rg.phase ^ 1) ||
                        !load_tile<D>(ct.dead, smem + Smem<D>::g + rg.at * kTileBytes<D>, mg, &ct.gfull[rg.at], &ct.landed, landings, h,
                                      row, rows, true))
                        return;
                    rg.step();
                }
        }
    }();
    settle(&ct.kvfull, items);
    settle(&ct.landed, landings);
    settle(rq, ct.qfull);
    settle(rg, ct.gfull);
}
// The queries' lse and D, the next stage's already on their way.
__device__ __forceinline__ void copy_stats(const PromptParams& p, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    for (long long k = 0;; ++k) {
        const Item x = make_item(p, k);
        if (!x.any) return;
        int t = x.lo, h = x.head * p.G;  // of what is read next
        float l[4], d[4], l2[4], d2[4];
        auto read = [&] {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int pos = t * kRows + lane + 32 * j;
                const bool on = h < (x.head + 1) * p.G && pos < x.len;
                const size_t at = on ? (size_t)(x.row0 + pos) * p.Hq + h : 0;
                l2[j] = on ? p.lse[at] * -kLog2e : -INFINITY;  // no query: no weight
                d2[j] = on ? -p.delta[at] : 0.f;
            }
            if (++t == x.hi) t = x.lo, ++h;
        };
        read();
        for (int i = 0; i < (x.hi - x.lo) * p.G; ++i, ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) l[j] = l2[j], d[j] = d2[j];
            read();
            if (!wait(ct.dead, &ct.stempty[n & 1], ((n >> 1) & 1) ^ 1)) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ct.lse[n & 1][lane + 32 * j] = l[j];
                ct.delta[n & 1][lane + 32 * j] = d[j];
            }
            warp_arrive(&ct.stfull[n & 1]);
        }
    }
}

template <int D> __device__ __forceinline__ void issue(const PromptParams& p, uint8_t* smem, Control& ct) {
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    const uint64_t k0 = desc_kmajor(Tile{base + Smem<D>::k, kRows}, 0), v0 = desc_kmajor(Tile{base + Smem<D>::v, kRows}, 0);
    const uint64_t q0 = desc_kmajor(Tile{base + Smem<D>::q, kRows}, 0), g0 = desc_kmajor(Tile{base + Smem<D>::g, kRows}, 0);
    const uint64_t qt0 = desc_mnmajor(Tile{base + Smem<D>::q, kRows}, 0), gt0 = desc_mnmajor(Tile{base + Smem<D>::g, kRows}, 0);
    Ring<kFirst> ahead, behind;  // of Q: of S and of dK
    Ring<kSecond> rg;
    uint32_t n = 0;  // stages before
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.kvfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        if (!x.any) return;
        const int total = (x.hi - x.lo) * p.G;
        for (int i = -1; i <= total; ++i) {
            if (i > 0) {  // dK of the stage before
                if (!wait(ct.dead, &ct.dsfull, (n - 1) & 1)) return;
                tc_fence_after();
                if (elect_one()) {
                    gather<D>(tm + kDK, tm + kDP, qt0 + behind.at * (kTileBytes<D> >> 4), i > 1);
                    mma_commit(&ct.qempty[behind.at]);
                    if (i == total) mma_commit(&ct.done);
                }
                __syncwarp();
                behind.step();
            }
            if (i >= 0 && i < total) {
                if (!wait(ct.dead, &ct.gfull[rg.at], rg.phase)) return;
                if (elect_one()) {
                    scores<D>(tm + kDP, v0, g0 + rg.at * (kTileBytes<D> >> 4));
                    mma_commit(&ct.dpfull);
                    if (i + 1 == total) mma_commit(&ct.kvempty);
                }
                __syncwarp();
                if (!wait(ct.dead, &ct.pfull, n & 1)) return;
                tc_fence_after();
                if (elect_one()) {
                    gather<D>(tm + kDV, tm + kS, gt0 + rg.at * (kTileBytes<D> >> 4), i > 0);
                    mma_commit(&ct.gempty[rg.at]);
                }
                __syncwarp();
                rg.step();
                ++n;
            }
            if (i + 1 < total) {
                if (!wait(ct.dead, &ct.qfull[ahead.at], ahead.phase)) return;
                if (elect_one()) {  // over P, whose dV was issued
                    scores<D>(tm + kS, k0, q0 + ahead.at * (kTileBytes<D> >> 4));
                    mma_commit(&ct.sfull);
                }
                __syncwarp();
                ahead.step();
            }
        }
    }
}

template <int D> __device__ __forceinline__ void rows(const PromptParams& p, Control& ct) {
    const int grp = threadIdx.x / kRows, r = threadIdx.x % kRows, c0 = 64 * grp;
    const uint32_t tm = warp_lane_base(ct.tmem), ts = tm + kS + c0, td = tm + kDP + c0;
    const float c2 = p.scale * kLog2e;
    uint32_t n = 0;
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.kvfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        warp_arrive(&ct.kvempty);
        if (!x.any) return;
        const int total = (x.hi - x.lo) * p.G, pos = x.j0 + r, w0 = pos & ~31;
        int t = x.lo;
        for (int i = 0; i < total; ++i, ++n) {
            const int i0 = t * kRows + c0;
            if (++t == x.hi) t = x.lo;
            const float4* lse = reinterpret_cast<const float4*>(ct.lse[n & 1] + c0);
            const float4* delta = reinterpret_cast<const float4*>(ct.delta[n & 1] + c0);
            if (!wait(ct.dead, &ct.stfull[n & 1], (n >> 1) & 1) || !wait(ct.dead, &ct.sfull, n & 1)) return;
            tc_fence_after();
            float s[64];
            tmem_ld32(ts, s);
            tmem_ld32(ts + 32, s + 32);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
                const float4 l = lse[j / 4];
                const float2 z = fma2(make_float2(s[j], s[j + 1]), both(c2), make_float2(l.x, l.y));
                const float2 y = fma2(make_float2(s[j + 2], s[j + 3]), both(c2), make_float2(l.z, l.w));
                s[j] = ex2(z.x);
                s[j + 1] = ex2(z.y);
                s[j + 2] = ex2(y.x);
                s[j + 3] = ex2(y.y);
            }
            const bool masked = i0 < w0 + 31 || (p.window && i0 + 63 >= w0 + p.window);
            const int from = pos - i0, upto = p.window ? from + p.window : 64;  // queries that see this key
            if (masked)
#pragma unroll
                for (int j = 0; j < 64; ++j) s[j] = j >= from && j < upto ? s[j] : 0.f;
            store_operand(ts, s);
            warp_arrive(&ct.pfull);
            if (!wait(ct.dead, &ct.dpfull, n & 1)) return;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float d[32];
                tmem_ld32(td + c, d);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 e = delta[(c + j) / 4];
                    const float2 a = mul2(make_float2(s[c + j], s[c + j + 1]), add2(make_float2(d[j], d[j + 1]), make_float2(e.x, e.y)));
                    const float2 b = mul2(make_float2(s[c + j + 2], s[c + j + 3]), add2(make_float2(d[j + 2], d[j + 3]), make_float2(e.z, e.w)));
                    s[c + j] = a.x; s[c + j + 1] = a.y; s[c + j + 2] = b.x; s[c + j + 3] = b.y;
                }
            }
            if (masked)  // a weight of zero times what is not finite is no zero
#pragma unroll
                for (int j = 0; j < 64; ++j) s[j] = j >= from && j < upto ? s[j] : 0.f;
            store_operand(td, s);
            warp_arrive(&ct.stempty[n & 1]);
            warp_arrive(&ct.dsfull);
        }
        if (!wait(ct.dead, &ct.done, k & 1)) return;
        tc_fence_after();
        const bool on = pos < x.len;
        if (grp == 0)
            store_row<D>(tm + kDV, static_cast<__nv_bfloat16*>(p.dv) + (x.row0 + pos) * p.ld_dv + (long long)x.head * D, 1.f, on);
        else
            store_row<D>(tm + kDK, static_cast<__nv_bfloat16*>(p.dk) + (x.row0 + pos) * p.ld_dk + (long long)x.head * D, p.scale, on);
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
        for (uint64_t* one : {&ct.kvfull, &ct.landed, &ct.sfull, &ct.dpfull, &ct.done, &ct.drained}) mbar_init(one, 1);
        for (uint64_t* eight : {&ct.pfull, &ct.dsfull}) mbar_init(eight, 8);
        mbar_init(&ct.kvempty, 1 + 8);
        for (int i = 0; i < kFirst; ++i) mbar_init(&ct.qfull[i], 1), mbar_init(&ct.qempty[i], 1);
        for (int i = 0; i < kSecond; ++i) mbar_init(&ct.gfull[i], 1), mbar_init(&ct.gempty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&ct.stfull[i], 1), mbar_init(&ct.stempty[i], 8);
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
    CUtensorMap m[4];
    if (!head_rows_map(&m[0], p.q, D, p.Hq, p.rows, p.ld_q, kRows) || !head_rows_map(&m[1], p.dO, D, p.Hq, p.rows, ld_g, kRows) ||
        !head_rows_map(&m[2], p.k, D, p.H, p.rows, p.ld_k, kRows) || !head_rows_map(&m[3], p.v, D, p.H, p.rows, p.ld_v, kRows))
        return cudaErrorInvalidValue;
    {
        TraceScope ts("prompt_dq_tc", st);
        dq::prompt_dq_tc_kernel<D><<<blocks(most_tiles(p.s, kRows) * p.Hq), kThreads, dq::Smem<D>::bytes, st>>>(p, m[0], m[1], m[2], m[3]);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    // A block for each item, so that one that is through takes the next in order: with the stages of 64 that this kernel had
    // before, 1066 us instead of 1425 with a block for each SM and its items dealt out beforehand (b8 t4096, 16 heads of
    // 128, four of keys; 678 us with the stages of 128).
    const long long keys = most_tiles(p.s, kRows) * p.H;
    if (keys >= (1ll << 31)) return cudaErrorInvalidValue;
    TraceScope ts("prompt_dkv_tc", st);
    dkv::prompt_dkv_tc_kernel<D><<<(unsigned)keys, kThreads, dkv::Smem<D>::bytes, st>>>(p, m[0], m[1], m[2], m[3]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_attn_bwd_tc(const PromptParams& p, cudaStream_t st) {
    if (cudaError_t e = prompt_attn_delta_bf16(p, st); e != cudaSuccess) return e;
    return p.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace dr
