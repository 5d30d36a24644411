// prompt_attn_tc.cu -- causal attention over whole prompts, bf16, forward: the products on the fifth-generation
// tensor cores (dr.h, dr_prompt_attn_fwd).
//
// A block works on one head and a tile of 256 queries, two halves of 128, over its keys in stages of 128:
//   S = Q K^T   128 x 128 for each half, contraction d;    O += P V   128 x d, contraction 128
// Tensor memory, all 512 columns: S and O of both halves, P (bf16) over the first columns of its S.  The halves
// take turns: while the threads of one form P from its S, the tensor cores work for the other.  Products are
// issued by one warp in the order PV(n), S(n + 1) for each half, so that S(n + 1) being there means that PV(n)
// is done, and the same barrier says both.
// Warps 0-3 and 4-7 hold a row of their half per thread, warp 8 issues products, warps 9 and 10 have tiles copied
// (11: none; registers are handed out by groups of four warps).
//
// 385 us for 8 x 4096 tokens, 16 query heads of 128, 4 key heads: 1430 TFLOP/s.  The two products of a half and stage
// take 1140 cycles of the tensor cores, the chain from one S to the weights being back about 1600 (barriers, tensor
// memory both ways, maxima, powers), of which the other half covers 1140.  Without any powers, maxima and sums it would
// be 365 us.  Slower: all eight warps on one half, 64 columns each, maxima exchanged (428 us); P handed over in one
// piece (388 us); waits that never suspend (396 us); a block for each tile instead of tiles dealt out to 152 (456 us).
//
// Softmax in base 2 against a reference m that follows the row's maximum only when that has passed it by more
// than 8: weights stay below 2^8, which bf16 and the fp32 sums hold as well, and O is rarely rescaled.  P is
// rounded to bf16 as an operand (2^-8 of a weight at most); the sum of the weights takes them unrounded.
#include "f32x2.cuh"
#include "prompt_attn.cuh"
#include "tc_block.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kHalf = 128, kTile = 2 * kHalf, kStage = 128, kThreads = 384, kInfos = 4;
// Keys are needed a stage earlier.  16 documents of 1 to 2500 tokens: 153 us, with two buffers each and one warp for all
// copies 166.
constexpr int kKBuffers = 3, kVBuffers = 2;
// Registers of a thread: as launched, then of the rows' threads and of the others, which give theirs up.
constexpr int kRegs = 168, kRowRegs = 208, kOtherRegs = 88;
static_assert(256 * kRowRegs + (kThreads - 256) * kOtherRegs <= kThreads * kRegs, "more than the block has");
constexpr float kNegInf = -INFINITY, kLn2 = 0.69314718055994530942f, kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.f;
__device__ __forceinline__ uint32_t s_col(int h) { return 128 * h; }
__device__ __forceinline__ uint32_t o_col(int h) { return 256 + 128 * h; }

struct Item {
    int any, row0, len, head, i0;  // any: there is one; rows of its sequence; first query
    int lo[2], hi[2];              // stages of each half (none: lo >= hi)
};
struct Control {
    uint64_t qfull, qempty, kfull[kKBuffers], kempty[kKBuffers], vfull[kVBuffers], vempty[kVBuffers], landed;
    uint64_t sfull[2], pfull[2][2], odone[2], drained;  // pfull: of each half the first and the last 64 columns
    uint32_t tmem;
    volatile int dead;
    Item item[kInfos];
};
template <int D> struct Smem {
    static constexpr int tile = 128 * D * 2, q = 0, k = 2 * tile, v = k + kKBuffers * tile, control = v + kVBuffers * tile,
                         bytes = control + 1024;
    static_assert(sizeof(Control) <= 1024, "control block");
};

// The k-th item of the block: rounds run through the blocks forwards and backwards in turn, so that the blocks that
// get the longer items of one round get the shorter ones of the next.
__device__ __forceinline__ Item make_item(const PromptParams& p, long long k) {
    const long long at = k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    Item x = {};
    int seq = 0, tile = 0;
    x.any = find_tile(p.s, kTile, at / p.Hq, seq, tile);
    if (!x.any) return x;
    x.head = (int)(at % p.Hq);
    seq_rows(p.s, seq, x.row0, x.len);
    x.i0 = tile * kTile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int first = x.i0 + h * kHalf, end = min(first + kHalf, x.len);
        x.lo[h] = p.window ? max(0, first - p.window + 1) / kStage : 0;
        x.hi[h] = first < x.len ? (end + kStage - 1) / kStage : x.lo[h];
    }
    return x;
}
__device__ __forceinline__ int first_stage(const Item& x) { return x.lo[0]; }
__device__ __forceinline__ int last_stage(const Item& x) { return max(x.hi[0], x.hi[1]); }  // one behind

// ------------------------------------------------------------------ warps 9 and 10: copies
// Queries and keys, and the items' data.
template <int D>
__device__ __forceinline__ void copy_keys(const PromptParams& p, const CUtensorMap* mq, const CUtensorMap* mk, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    Ring<kKBuffers> ring;
    long long items = 0;
    [&] {
        for (long long k = 0;; ++k) {
            const Item x = make_item(p, k);
            // after the last item's products with its queries, and after the row threads and the values' copies have begun
            // with it (so they are never two items behind)
            if (!wait(ct.dead, &ct.qempty, (k & 1) ^ 1)) return;
            if (lane == 0) {
                ct.item[k % kInfos] = x;
                if (x.any) {
                    mbar_arrive_expect_tx(&ct.qfull, 2 * Smem<D>::tile);
                    for (int h = 0; h < 2; ++h)
                        load_rows<kHalf, D>(smem + Smem<D>::q + h * Smem<D>::tile, mq, &ct.qfull, x.head, x.row0 + x.i0 + h * kHalf);
                } else {
                    mbar_arrive(&ct.qfull);
                }
            }
            __syncwarp();
            ++items;
            if (!x.any) return;
            for (int t = first_stage(x); t < last_stage(x); ++t) {
                if (!wait(ct.dead, &ct.kempty[ring.at], ring.phase ^ 1)) return;
                if (lane == 0) {  // keys behind the sequence make scores that are hidden
                    mbar_arrive_expect_tx(&ct.kfull[ring.at], Smem<D>::tile);
                    load_rows<kStage, D>(smem + Smem<D>::k + ring.at * Smem<D>::tile, mk, &ct.kfull[ring.at], x.head / p.G,
                                         x.row0 + t * kStage);
                }
                __syncwarp();
                ring.step();
            }
        }
    }();
    settle(&ct.qfull, items);
    settle(ring, ct.kfull);
}
template <int D> __device__ __forceinline__ void copy_values(const PromptParams& p, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t landings = 0;
    Ring<kVBuffers> ring;
    [&] {
        for (long long k = 0;; ++k) {
            if (!wait(ct.dead, &ct.qfull, k & 1)) return;
            const Item x = ct.item[k % kInfos];
            warp_arrive(&ct.qempty);
            if (!x.any) return;
            for (int t = first_stage(x); t < last_stage(x); ++t) {
                if (!wait(ct.dead, &ct.vempty[ring.at], ring.phase ^ 1)) return;
                uint8_t* v = smem + Smem<D>::v + ring.at * Smem<D>::tile;
                const int rows = x.len - t * kStage;
                uint64_t* bar = rows < kStage ? &ct.landed : &ct.vfull[ring.at];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, Smem<D>::tile);
                    load_rows<kStage, D>(v, mv, bar, x.head / p.G, x.row0 + t * kStage);
                }
                __syncwarp();
                if (rows < kStage) {  // values behind the sequence may be anything, and zero times that is not zero
                    if (!wait(ct.dead, &ct.landed, landings++ & 1)) return;
                    clear_rows<kStage, D>(v, rows);
                    if (lane == 0) mbar_arrive(&ct.vfull[ring.at]);
                    __syncwarp();
                }
                ring.step();
            }
        }
    }();
    settle(&ct.landed, landings);
    settle(ring, ct.vfull);
}

// ------------------------------------------------------------------ warp 8: products
template <int D>
__device__ __forceinline__ void issue(const PromptParams& p, uint8_t* smem, Control& ct) {
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    // descriptors of the first buffers; an address step of 16 bytes is 1 in their lowest field
    const uint64_t q0 = desc_kmajor(Tile{base + Smem<D>::q, kHalf}, 0), k0 = desc_kmajor(Tile{base + Smem<D>::k, kStage}, 0);
    const uint64_t v0 = desc_mnmajor(Tile{base + Smem<D>::v, kStage}, 0);
    Ring<kKBuffers> rk;
    Ring<kVBuffers> rv;
    uint32_t np[2] = {0, 0};
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.qfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        if (!x.any) return;
        const int first = first_stage(x), last = last_stage(x);
        for (int t = first - 1; t < last; ++t) {
            if (t >= first && !wait(ct.dead, &ct.vfull[rv.at], rv.phase)) return;
            if (t + 1 < last && !wait(ct.dead, &ct.kfull[rk.at], rk.phase)) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool pv = t >= x.lo[h] && t < x.hi[h], qk = t + 1 >= x.lo[h] && t + 1 < x.hi[h];
                if (pv) {
                    const uint64_t vd = v0 + rv.at * (Smem<D>::tile >> 4);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (!wait(ct.dead, &ct.pfull[h][part], np[h] & 1)) return;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 64 * part; kk < 64 * part + 64; kk += 16)  // 16 positions: 16 rows of 128 bytes
                                mma_ts(tm + o_col(h), tm + s_col(h) + kk / 2, vd + kk * 8, idesc_bf16(kHalf, D, false, true),
                                       t > x.lo[h] || kk > 0);
                            if (part && t + 1 == x.hi[h]) mma_commit(&ct.odone[h]);
                        }
                        __syncwarp();
                    }
                    ++np[h];
                }
                if (elect_one()) {
                    if (qk) {
                        const uint64_t kd = k0 + rk.at * (Smem<D>::tile >> 4), qd = q0 + h * (Smem<D>::tile >> 4);
#pragma unroll
                        for (int kk = 0; kk < D; kk += 16)  // 16 channels: 32 bytes of a 128-byte row
                            mma_bf16(tm + s_col(h), qd + (kk >> 6) * (kHalf * 128 / 16) + (kk & 63) / 8,
                                     kd + (kk >> 6) * (kStage * 128 / 16) + (kk & 63) / 8, idesc_bf16(kHalf, kStage), kk > 0);
                        mma_commit(&ct.sfull[h]);
                    }
                }
                __syncwarp();
            }
            if (elect_one()) {
                if (t >= first) mma_commit(&ct.vempty[rv.at]);
                if (t + 1 < last) mma_commit(&ct.kempty[rk.at]);
                if (t + 2 == last) mma_commit(&ct.qempty);
            }
            __syncwarp();
            if (t >= first) rv.step();
            if (t + 1 < last) rk.step();
        }
    }
}

// ------------------------------------------------------------------ warps 0-7: a row per thread
template <int D> __device__ __forceinline__ void soften(const PromptParams& p, Control& ct) {
    const int h = threadIdx.x / kHalf, r = threadIdx.x % kHalf;
    const uint32_t ts = warp_lane_base(ct.tmem) + s_col(h), to = warp_lane_base(ct.tmem) + o_col(h);
    // Scores in base 2: c2 s, with a negative scale's sign in s.  A scale of zero makes s zero and c2 one, because zero times
    // the -inf of what is hidden is no number.
    const float c2 = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e, sign = p.scale == 0.f ? 0.f : -1.f;
    uint32_t n = 0, done = 0;
    for (long long k = 0;; ++k) {
        if (!wait(ct.dead, &ct.qfull, k & 1)) return;
        const Item x = ct.item[k % kInfos];
        warp_arrive(&ct.qempty);
        if (!x.any) return;
        const int pos = x.i0 + h * kHalf + r, w0 = pos & ~31;  // of the warp's first row
        const int lo = h ? x.lo[1] : x.lo[0], hi = h ? x.hi[1] : x.hi[0];
        if (lo >= hi) continue;
        float m = kNegInf, l = 0.f;  // m: reference, as a product with c2
        for (int t = lo; t < hi; ++t, ++n) {
            const int j0 = t * kStage;
            if (!wait(ct.dead, &ct.sfull[h], n & 1)) return;
            tc_fence_after();
            float s[kStage];
#pragma unroll
            for (int c = 0; c < kStage; c += 32) tmem_ld32(ts + c, s + c);
            tmem_ld_wait();
            if (p.scale <= 0.f)
#pragma unroll
                for (int j = 0; j < kStage; ++j) s[j] *= sign;
            if (j0 + kStage - 1 > w0 || (p.window && j0 <= w0 + 31 - p.window)) {
                const int up = pos - j0, down = p.window ? up - p.window : -1;
#pragma unroll
                for (int j = 0; j < kStage; ++j) s[j] = j <= up && j > down ? s[j] : kNegInf;
            }
            float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int j = 0; j < kStage; j += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], fmaxf(s[j + 2 * q], s[j + 2 * q + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
            const bool grow = top > m + kSlack;
            if (__any_sync(0xffffffffu, grow)) {
                const float m2 = grow ? top : m, f = m == m2 ? 1.f : ex2(m - m2);
                l *= f;
                m = m2;
                if (t > lo) {  // O holds the products of the stages before: S(t) came after them
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float y[32];
                        uint32_t z[32];
                        tmem_ld32(to + c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j] = __float_as_uint(y[j] * f);
                        tmem_st32(to + c, z);
                    }
                }
            }
            const float ref = m == kNegInf ? 0.f : -m;
            float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
            for (int c = 0; c < kStage; c += 64) {
                uint32_t z[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float2 e = fma2(make_float2(s[c + j], s[c + j + 1]), both(c2), both(ref));
                    e = make_float2(ex2(e.x), ex2(e.y));
                    sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], e);
                    z[j / 2] = pack_bf16(e.x, e.y);
                }
                tmem_st32(ts + c / 2, z);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&ct.pfull[h][c / 64]);
            }
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
        }
        if (!wait(ct.dead, &ct.odone[h], done++ & 1)) return;
        tc_fence_after();
        const float inv = 1.f / l;
        const size_t at = (size_t)(x.row0 + pos) * p.Hq + x.head;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
            float y[32];
            tmem_ld32(to + c, y);
            tmem_ld_wait();
            if (pos < x.len) {
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at * D + c);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = make_uint4(pack_bf16(y[8 * q] * inv, y[8 * q + 1] * inv), pack_bf16(y[8 * q + 2] * inv, y[8 * q + 3] * inv),
                                      pack_bf16(y[8 * q + 4] * inv, y[8 * q + 5] * inv), pack_bf16(y[8 * q + 6] * inv, y[8 * q + 7] * inv));
            }
        }
        tc_fence_before();
        if (p.lse && pos < x.len) p.lse[at] = (m + log2f(l)) * kLn2;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_fwd_tc_kernel(const PromptParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ct = *reinterpret_cast<Control*>(smem + Smem<D>::control);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(&ct.qfull, 1);
        mbar_init(&ct.qempty, 1 + 8 + 1);
        mbar_init(&ct.landed, 1);
        mbar_init(&ct.drained, 1);
        for (int i = 0; i < kKBuffers; ++i) mbar_init(&ct.kfull[i], 1), mbar_init(&ct.kempty[i], 1);
        for (int i = 0; i < kVBuffers; ++i) mbar_init(&ct.vfull[i], 1), mbar_init(&ct.vempty[i], 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(&ct.sfull[h], 1);
            mbar_init(&ct.pfull[h][0], 4);
            mbar_init(&ct.pfull[h][1], 4);
            mbar_init(&ct.odone[h], 1);
        }
        ct.dead = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        soften<D>(p, ct);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) issue<D>(p, smem, ct), drain(&ct.drained);
        else if (warp == 9) copy_keys<D>(p, &mq, &mk, smem, ct);
        else if (warp == 10) copy_values<D>(p, &mv, smem, ct);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ct.dead && threadIdx.x == 0 && p.status) *reinterpret_cast<volatile int32_t*>(p.status) = kErrTimeout;
    if (warp == 0) tmem_dealloc(ct.tmem, 512);
}

template <int D> cudaError_t launch(const PromptParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    // the split of the registers must not ask for more than the block is launched with: it would wait for them
    static const bool fits = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, prompt_fwd_tc_kernel<D>) == cudaSuccess && a.numRegs == kRegs;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = set_smem_once(prompt_fwd_tc_kernel<D>, Smem<D>::bytes, ready); e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv;
    if (!head_rows_map(&mq, p.q, D, p.Hq, p.rows, p.ld_q, kHalf) || !head_rows_map(&mk, p.k, D, p.H, p.rows, p.ld_k, kStage) ||
        !head_rows_map(&mv, p.v, D, p.H, p.rows, p.ld_v, kStage))
        return cudaErrorInvalidValue;
    const long long items = most_tiles(p.s, kTile) * p.Hq;
    const int sms = sm_count(), blocks = (int)(items < sms ? items : sms);
    if (blocks < 1) return cudaErrorInvalidDevice;
    TraceScope ts("prompt_fwd_tc", st);
    prompt_fwd_tc_kernel<D><<<blocks, kThreads, Smem<D>::bytes, st>>>(p, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_attn_fwd_tc(const PromptParams& p, cudaStream_t st) {
    return p.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace dr
