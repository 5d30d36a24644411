// linear_attn_tc.cu -- linear attention with a decay for each head, bf16: the chunked scan of linear_attn.cuh on
// the fifth-generation tensor cores.  Chunks of C = 128 tokens, i and j within the chunk, X the state before it,
// a = e^g, n the chunk's tokens:
//   A = Q K^T;  P_ij = beta a^{|i-j|} A_ij (j <= i, reverse j >= i);  out = alpha (P V + diag(a^{out(i)}) Q X)
//   X' = a^n X + K'^T V,  K'_j = beta a^{in(j)} k_j
//   forward: out(i) = i + 1, in(j) = n - 1 - j;  reverse: out(i) = n - 1 - i, in(j) = j + 1
// so no power of a is ever above one, however strong the decay.
//
// A block has a sequence and a head.  The state stays in fp32 registers, a row of it in each thread of four warps;
// what a chunk adds comes from tensor memory, and a bf16 image of the state goes to shared memory for the next
// chunk's queries.  K' is a sum of two bf16 parts (2^-16 of it is lost), so that what the states add up over a
// sequence is not bf16; P, and the state as an operand, are rounded once (2^-8 at most).
// Tensor memory: A with P over it, Q X, P V, K'^T V: 4 x 128 columns.
// Warps 0-3: K' (its high part over K, once A is there), then P.  4-7: output rows.  8-11: state.  12: products,
// 13: copies, through a ring of five tiles in the order K, Q, V.
#include "f32x2.cuh"
#include "linear_attn.cuh"
#include "tc_block.cuh"
#include "trace.cuh"
#include "vec4.cuh"

namespace dr {
namespace {

constexpr int kC = 128, kThreads = 512, kSlots = 5;
// Registers of a thread: as launched, then of the four groups of four warps.
constexpr int kRegs = 128, kWeightRegs = 112, kOutRegs = 112, kStateRegs = 208, kOtherRegs = 80;
static_assert(kWeightRegs + kOutRegs + kStateRegs + kOtherRegs <= 4 * kRegs, "more than the block has");
constexpr uint32_t kA = 0, kQX = 128, kPV = 256, kKV = 384;  // columns of tensor memory

struct Control {
    uint64_t full[kSlots], empty[kSlots], landed, afull, pfull, kfull, dfull, xfull, ofull, oempty, drained;
    uint32_t tmem;
    volatile int dead;
    __align__(16) float power[kC];  // beta a^n
    __align__(16) float column[32];  // a^{31 - j}, reverse a^j
};
template <int DK, int DV> struct Smem {
    static constexpr int slot = kC * (DK > DV ? DK : DV) * 2, low = kSlots * slot, x = low + kC * DK * 2,
                         end = x + DK * DV * 2,
                         // K'^T is read as 128 rows, for 64 channels 64 rows past them that nobody looks at
                         control = end > low + kC * 128 * 2 ? end : low + kC * 128 * 2, bytes = control + 1024;
    static_assert(sizeof(Control) <= 1024, "control block");
};

struct Work {
    int row0, len, chunks;
    __device__ __forceinline__ int at(const ScanParams& p, int n) const { return (p.reverse ? chunks - 1 - n : n) * kC; }
    __device__ __forceinline__ int tokens(int first) const { return min(kC, len - first); }
};

template <int DK, int DV>
__device__ __forceinline__ void copy_tiles(const ScanParams& p, const Work& w, int head, const CUtensorMap* mq,
                                           const CUtensorMap* mk, const CUtensorMap* mv, uint8_t* smem, Control& ct) {
    const int lane = threadIdx.x & 31;
    uint32_t landings = 0, slot = 0, parity = 1;
    for (int n = 0; n < w.chunks; ++n) {
        const int first = w.at(p, n), row = w.row0 + first, rows = w.tokens(first);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (!wait(ct.dead, &ct.empty[slot], parity)) return;
            uint8_t* tile = smem + slot * Smem<DK, DV>::slot;
            // values behind the sequence are summed with weights of zero: they have to be numbers
            const bool cut = i == 2 && rows < kC;
            uint64_t* bar = cut ? &ct.landed : &ct.full[slot];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, kC * (i == 2 ? DV : DK) * 2);
                if (i == 2) load_rows<kC, DV>(tile, mv, bar, head, row);
                else load_rows<kC, DK>(tile, i == 0 ? mk : mq, bar, head, row);
            }
            __syncwarp();
            if (cut) {
                if (!wait(ct.dead, &ct.landed, landings++ & 1)) return;
                clear_rows<kC, DV>(tile, rows);
                if (lane == 0) mbar_arrive(&ct.full[slot]);
                __syncwarp();
            }
            if (++slot == kSlots) { slot = 0; parity ^= 1; }
        }
    }
}

template <int DK, int DV>
__device__ __forceinline__ void issue(const Work& w, uint8_t* smem, Control& ct) {
    using S = Smem<DK, DV>;
    const uint32_t base = smem_u32(smem), tm = ct.tmem;
    const uint64_t row0 = desc_kmajor(Tile{base, kC}, 0), col0 = desc_mnmajor(Tile{base, kC}, 0);  // of slot 0
    const uint64_t low0 = desc_mnmajor(Tile{base + S::low, kC}, 0), x0 = desc_mnmajor(Tile{base + S::x, DK}, 0);
    uint32_t u = 0;
    for (int n = 0; n < w.chunks; ++n) {
        uint32_t slot[3];
#pragma unroll
        for (int i = 0; i < 3; ++i, ++u) {
            slot[i] = u % kSlots;
            if (i < 2 && !wait(ct.dead, &ct.full[slot[i]], (u / kSlots) & 1)) return;
        }
        const uint64_t k = slot[0] * (S::slot >> 4), q = slot[1] * (S::slot >> 4), v = slot[2] * (S::slot >> 4);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DK; kk += 16)  // 16 channels: 32 bytes of a 128-byte row
                mma_bf16(tm + kA, row0 + q + (kk >> 6) * (kC * 128 / 16) + (kk & 63) / 8,
                         row0 + k + (kk >> 6) * (kC * 128 / 16) + (kk & 63) / 8, idesc_bf16(kC, kC), kk > 0);
            mma_commit(&ct.afull);
        }
        __syncwarp();
        if (!wait(ct.dead, &ct.xfull, n & 1) || !wait(ct.dead, &ct.oempty, (n & 1) ^ 1)) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DK; kk += 16)
                mma_bf16(tm + kQX, row0 + q + (kk >> 6) * (kC * 128 / 16) + (kk & 63) / 8, x0 + kk * 8,
                         idesc_bf16(kC, DV, false, true), kk > 0);
        }
        __syncwarp();
        if (!wait(ct.dead, &ct.full[slot[2]], ((u - 1) / kSlots) & 1) || !wait(ct.dead, &ct.kfull, n & 1)) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < kC; kk += 16)  // 16 tokens: 16 rows of 128 bytes
                    mma_bf16(tm + kKV, (part ? low0 : col0 + k) + kk * 8, col0 + v + kk * 8, idesc_bf16(128, DV, true, true),
                             part + kk > 0);
            mma_commit(&ct.dfull);
            mma_commit(&ct.empty[slot[0]]);
        }
        __syncwarp();
        if (!wait(ct.dead, &ct.pfull, n & 1)) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kC; kk += 16)
                mma_ts(tm + kPV, tm + kA + kk / 2, col0 + v + kk * 8, idesc_bf16(kC, DV, false, true), kk > 0);
            mma_commit(&ct.ofull);
            mma_commit(&ct.empty[slot[2]]);
        }
        __syncwarp();
    }
}

// The parts hi + lo of f times two bf16 values: what hi, rounded, leaves of a value is rounded to lo.
__device__ __forceinline__ void split2(uint32_t u, float f, uint32_t& hi, uint32_t& lo) {
    const float2 x = mul2(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), both(f));
    hi = pack_bf16(x.x, x.y);
    lo = pack_bf16(x.x - __uint_as_float(hi << 16), x.y - __uint_as_float(hi & 0xffff0000u));
}
// Warps 0-3, a token per thread: K', which the state waits for, then P.
template <int DK, int DV> __device__ __forceinline__ void weights(const ScanParams& p, const Work& w, int head, uint8_t* smem, Control& ct) {
    const int i = threadIdx.x, warp = i >> 5;
    const uint32_t tm = warp_lane_base(ct.tmem);
    const float g = p.g[head], f_in = p.reverse ? p.scale : 1.f;
    for (int n = 0; n < w.chunks; ++n) {
        const uint32_t u = 3 * n;
        const int tokens = w.tokens(w.at(p, n));
        const float f = i < tokens ? f_in * decay(g, (float)(p.reverse ? i + 1 : tokens - 1 - i)) : 0.f;
        uint8_t* tile = smem + u % kSlots * Smem<DK, DV>::slot;
        if (!wait(ct.dead, &ct.full[u % kSlots], (u / kSlots) & 1) || !wait(ct.dead, &ct.afull, n & 1)) return;
        if (n && !wait(ct.dead, &ct.dfull, (n - 1) & 1)) return;  // the low parts of the chunk before are in use
        tc_fence_after();
#pragma unroll 4
        for (int c = 0; c < DK; c += 8) {
            const uint32_t off = sw128_offset(i, c, kC);
            uint4 u = *reinterpret_cast<const uint4*>(tile + off), hi, lo;
            if (tokens < kC && i >= tokens) u = make_uint4(0, 0, 0, 0);  // behind the sequence: may be no numbers
            split2(u.x, f, hi.x, lo.x);
            split2(u.y, f, hi.y, lo.y);
            split2(u.z, f, hi.z, lo.z);
            split2(u.w, f, hi.w, lo.w);
            *reinterpret_cast<uint4*>(tile + off) = hi;
            *reinterpret_cast<uint4*>(smem + Smem<DK, DV>::low + off) = lo;
        }
        fence_async_smem();
        warp_arrive(&ct.kfull);
        // 32 columns at a time: those that all the warp's rows see take a^{|i-j|} as a row's and a column's factor,
        // both at most one; those on the diagonal one of the powers each; the others are zero
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float s[32];
            uint32_t z[16];
            const int c = 32 * b;
            if (p.reverse ? b < warp : b > warp) {
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = 0;
            } else {
                tmem_ld32(tm + kA + c, s);
                tmem_ld_wait();
                if (b == warp || (p.reverse && tokens < kC)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int back = p.reverse ? c + j - i : i - c - j;
                        s[j] = back >= 0 && c + j < tokens ? s[j] * ct.power[max(back, 0)] : 0.f;
                    }
                } else {
                    const float2 fr = both(p.reverse ? ct.power[c - i] : ct.power[i - c - 31]);
                    const float4* fc = reinterpret_cast<const float4*>(ct.column);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 y = fc[j / 4];
                        const float2 t0 = mul2(make_float2(s[j], s[j + 1]), mul2(fr, make_float2(y.x, y.y)));
                        const float2 t1 = mul2(make_float2(s[j + 2], s[j + 3]), mul2(fr, make_float2(y.z, y.w)));
                        s[j] = t0.x; s[j + 1] = t0.y; s[j + 2] = t1.x; s[j + 3] = t1.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
            }
            tmem_st16(tm + kA + c / 2, z);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&ct.pfull);
    }
}

// Warps 4-7, a token per thread.  A whole chunk's rows leave as tensor stores, from the place of its queries.
template <int DK, int DV>
__device__ __forceinline__ void outputs(const ScanParams& p, const Work& w, int head, const CUtensorMap* mo, uint8_t* smem, Control& ct) {
    const int i = threadIdx.x & (kC - 1);
    const uint32_t tm = warp_lane_base(ct.tmem);
    const float g = p.g[head], f_out = p.reverse ? 1.f : p.scale;
    for (int n = 0; n < w.chunks; ++n) {
        const int first = w.at(p, n), tokens = w.tokens(first);
        const uint32_t slot = (3 * n + 1) % kSlots;
        uint8_t* tile = smem + slot * Smem<DK, DV>::slot;
        const float2 fx = both(f_out * decay(g, (float)(p.reverse ? tokens - 1 - i : i + 1))), fy = both(f_out);
        if (!wait(ct.dead, &ct.ofull, n & 1)) return;
        tc_fence_after();
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + (w.row0 + first + i) * p.ld_o + (long long)head * DV;
#pragma unroll
        for (int c = 0; c < DV; c += 32) {
            float x[32], y[32];
            tmem_ld32(tm + kQX + c, x);
            tmem_ld32(tm + kPV + c, y);
            tmem_ld_wait();
            if (c + 32 == DV) {
                tc_fence_before();
                warp_arrive(&ct.oempty);
            }
            uint32_t z[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 o = fma2(fx, make_float2(x[2 * j], x[2 * j + 1]), mul2(fy, make_float2(y[2 * j], y[2 * j + 1])));
                z[j] = pack_bf16(o.x, o.y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 u = make_uint4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
                if (tokens == kC) *reinterpret_cast<uint4*>(tile + sw128_offset(i, c + 8 * j, kC)) = u;
                else if (i < tokens) reinterpret_cast<uint4*>(to + c)[j] = u;
            }
        }
        if (tokens == kC) fence_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (i == 0) {
            if (tokens == kC) {
#pragma unroll
                for (int c = 0; c < DV; c += 64) tma_store_3d(mo, tile + (c / 64) * kC * 128, c, head, w.row0 + first);
                bulk_commit();
                bulk_wait_read();
            }
            mbar_arrive(&ct.empty[slot]);
        }
        __syncwarp();
    }
    if (i == 0) bulk_wait_all();
}

// Warps 8-11: a row of the state per thread (of the first DK).
template <int DK, int DV>
__device__ __forceinline__ void states(const ScanParams& p, const Work& w, int seq, int head, uint8_t* smem, Control& ct) {
    const int r = threadIdx.x & 127;
    const bool on = r < DK;
    const uint32_t tm = warp_lane_base(ct.tmem);
    const float g = p.g[head];
    const size_t unit = (size_t)seq * p.H + head;
    float x[DV];
#pragma unroll
    for (int c = 0; c < DV; ++c) x[c] = 0.f;
    if (p.x0 && on) {
        if (p.x0_transposed) {
#pragma unroll
            for (int c = 0; c < DV; ++c) x[c] = p.x0[(unit * DV + c) * DK + r];
        } else {
#pragma unroll
            for (int c = 0; c < DV; c += 4) {
                const float4 y = load4(p.x0 + (unit * DK + r) * DV + c);
                x[c] = y.x; x[c + 1] = y.y; x[c + 2] = y.z; x[c + 3] = y.w;
            }
        }
    }
    for (int n = 0; n <= w.chunks; ++n) {
        if (n > 0) {
            if (!wait(ct.dead, &ct.dfull, (n - 1) & 1)) return;  // and the image of the state has been read
            tc_fence_after();
            const float a = decay(g, (float)w.tokens(w.at(p, n - 1)));
#pragma unroll
            for (int c = 0; c < DV; c += 32) {
                float y[32];
                tmem_ld32(tm + kKV + c, y);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) x[c + j] = fmaf(a, x[c + j], y[j]);
            }
            tc_fence_before();
        }
        if (n < w.chunks) {
            if (on)
#pragma unroll
                for (int c = 0; c < DV; c += 16) {
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = x[c + j];
                    tile_store16(smem + Smem<DK, DV>::x, r, c, DK, y);
                }
            fence_async_smem();
            warp_arrive(&ct.xfull);
        }
    }
    if (p.xT && on)
#pragma unroll
        for (int c = 0; c < DV; c += 4) store4(p.xT + (unit * DK + r) * DV + c, make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]));
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_scan_tc_kernel(const ScanParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ct = *reinterpret_cast<Control*>(smem + Smem<DK, DV>::control);
    const int warp = threadIdx.x >> 5, seq = blockIdx.x / p.H, head = blockIdx.x % p.H;
    if (warp == 0) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ct.full[i], 1);
            mbar_init(&ct.empty[i], 1);
        }
        for (uint64_t* one : {&ct.landed, &ct.afull, &ct.dfull, &ct.ofull, &ct.drained}) mbar_init(one, 1);
        for (uint64_t* four : {&ct.pfull, &ct.kfull, &ct.xfull, &ct.oempty}) mbar_init(four, 4);
        ct.dead = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kC) ct.power[threadIdx.x] = (p.reverse ? p.scale : 1.f) * decay(p.g[head], (float)threadIdx.x);
    if (threadIdx.x < 32) ct.column[threadIdx.x] = decay(p.g[head], (float)(p.reverse ? threadIdx.x : 31 - threadIdx.x));
    Work w;
    seq_rows(p.s, seq, w.row0, w.len);
    w.chunks = (w.len + kC - 1) / kC;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWeightRegs));
        weights<DK, DV>(p, w, head, smem, ct);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
        outputs<DK, DV>(p, w, head, &mo, smem, ct);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
        states<DK, DV>(p, w, seq, head, smem, ct);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 12) issue<DK, DV>(w, smem, ct), drain(&ct.drained);
        else if (warp == 13) copy_tiles<DK, DV>(p, w, head, &mq, &mk, &mv, smem, ct);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ct.dead && threadIdx.x == 0 && p.status) *reinterpret_cast<volatile int32_t*>(p.status) = kErrTimeout;
    if (warp == 0) tmem_dealloc(ct.tmem, 512);
}

template <int DK, int DV> cudaError_t launch(const ScanParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    // the split of the registers must not ask for more than the block is launched with: it would wait for them
    static const bool fits = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, linear_scan_tc_kernel<DK, DV>) == cudaSuccess && a.numRegs == kRegs;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = set_smem_once(linear_scan_tc_kernel<DK, DV>, Smem<DK, DV>::bytes, ready); e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mo;
    if (!head_rows_map(&mq, p.q, DK, p.H, p.rows, p.ld_q, kC) || !head_rows_map(&mk, p.k, DK, p.H, p.rows, p.ld_k, kC) ||
        !head_rows_map(&mv, p.v, DV, p.H, p.rows, p.ld_v, kC) || !head_rows_map(&mo, p.out, DV, p.H, p.rows, p.ld_o, kC))
        return cudaErrorInvalidValue;
    TraceScope ts("linear_scan_tc", st);
    linear_scan_tc_kernel<DK, DV><<<p.s.N * p.H, kThreads, Smem<DK, DV>::bytes, st>>>(p, mq, mk, mv, mo);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linear_scan_tc(const ScanParams& p, cudaStream_t st) {
    if (p.dk == 128) return p.dv == 128 ? launch<128, 128>(p, st) : launch<128, 64>(p, st);
    return p.dv == 128 ? launch<64, 128>(p, st) : launch<64, 64>(p, st);
}

}  // namespace dr
