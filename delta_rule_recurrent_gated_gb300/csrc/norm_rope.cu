// norm_rope.cu -- RMS norm of queries and keys for each head with the position rotation in
// the same pass, and its gradient (dr.h, dr_norm_rope_fwd / dr_norm_rope_bwd).
//
// With r = 1 / sqrt(mean x^2 + eps) the row's scale comes out of the rotation: for channel c
// with partner p (the other channel of its pair)
//   y_c = r (x_c A_c + x_p B_c),   A_c = w_c cos,  B_c = -+ w_p sin
// and A, B depend on the token and the channel only, so a thread forms them once for its
// token and uses them for every head it takes.  Backward, with m = R^T dy, g = m w:
//   dx = r (g - x r^2 mean(g x)),   dw_c = sum over tokens and heads of m_c x_c r.
//
// Layout: a group of LANES threads (a power of two, d / 8 of them active) owns a token and a
// run of its heads; a thread owns 8 channels, two pieces of 4 that hold both ends of each of its
// pairs, so nothing but the sums of a row passes between threads.  Products and sums run on
// pairs of fp32 values (fma.rn.f32x2).  Each value is read and written once.
//
// 8 x 4096 tokens, 20 heads of 128, bf16: forward 53.7 us, 6.3 TB/s, bound by HBM; gradient 89.5 us,
// 5.6 TB/s, bound by the loads that 512 threads of 116 registers keep in flight (in blocks of 256 92.2):
// 768 threads with two heads loaded at once take 98 us, a ring of asynchronous copies 113.
#include "chain.cuh"
#include "common.cuh"
#include "f32x2.cuh"
#include "rope.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kRopeThreads = 256, kBwdThreads = 128;
constexpr int kRun = 4;                           // heads that a thread has loaded at once (bf16, backward)
constexpr int kBwdResident = 4;                   // blocks of the backward kernel on an SM
constexpr int kBwdBlocks = 152 * kBwdResident;    // over all runs of heads

// A thread's 8 channels as loaded: two pieces of 4.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int second) {
        a = *reinterpret_cast<const uint2*>(p);
        b = *reinterpret_cast<const uint2*>(p + second);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, int second) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + second);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        x[0] = make_float2(a.x, a.y);
        x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y);
        x[3] = make_float2(b.z, b.w);
    }
};
__device__ __forceinline__ uint32_t pack2(float2 y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int second, const float2 (&y)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(y[0]), pack2(y[1]));
    *reinterpret_cast<uint2*>(p + second) = make_uint2(pack2(y[2]), pack2(y[3]));
}
__device__ __forceinline__ void store8(float* p, int second, const float2 (&y)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
    *reinterpret_cast<float4*>(p + second) = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
}

// What a thread needs of its place: its two pieces of 4 channels begin at ch and ch + second.
struct Lane {
    bool active;     // holds channels at all (d / 8 need not be a power of two)
    bool rotated;    // they are rotated, by angles angle .. angle + 3
    int ch, second, angle;
};
template <int LANES>
__device__ __forceinline__ Lane make_lane(const RopeParams& p) {
    Lane a;
    const int l = threadIdx.x % LANES;
    a.active = 8 * l < p.d;
    a.rotated = 8 * l < p.rot;
    a.angle = 4 * l;
    const bool halves = a.rotated && p.style == DR_ROPE_HALVES;
    a.ch = halves ? 4 * l : 8 * l;
    a.second = halves ? p.rot / 2 : 4;
    return a;
}

// cos and signed sin of the thread's 8 channels at the token's position: the coefficients of
// the rotation y_c = n_c C_c + n_p S_c.  Outside the rotated channels C = 1, S = 0; NaN where
// the position lies outside the table.
__device__ __forceinline__ void coefficients(const RopeParams& p, const Lane& a, long long tok,
                                             float2 (&C)[4], float2 (&S)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { C[i] = both(1.f); S[i] = both(0.f); }
    if (p.rot == 0 || !a.active) return;
    const long long b = tok / p.T;
    long long pos = p.positions ? p.positions[tok] : tok - b * p.T;
    if (p.start) pos += p.start[b];
    if (pos < 0 || pos >= p.table_rows) {
        const float bad = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int i = 0; i < 4; ++i) C[i] = S[i] = both(bad);
        return;
    }
    if (!a.rotated) return;
    const size_t at = (size_t)pos * (p.rot / 2) + a.angle;
    const float4 c = *reinterpret_cast<const float4*>(p.cos_t + at);
    const float4 s = *reinterpret_cast<const float4*>(p.sin_t + at);
    if (p.style == DR_ROPE_PAIRS) {
        C[0] = both(c.x); C[1] = both(c.y); C[2] = both(c.z); C[3] = both(c.w);
        S[0] = make_float2(-s.x, s.x); S[1] = make_float2(-s.y, s.y);
        S[2] = make_float2(-s.z, s.z); S[3] = make_float2(-s.w, s.w);
    } else {
        C[0] = C[2] = make_float2(c.x, c.y);
        C[1] = C[3] = make_float2(c.z, c.w);
        S[0] = make_float2(-s.x, -s.y); S[1] = make_float2(-s.z, -s.w);
        S[2] = make_float2(s.x, s.y); S[3] = make_float2(s.z, s.w);
    }
}

// The partners of a thread's channels: beside them (PAIRS) or in the other piece (halves).  Channels that are not
// rotated (PART: there are such) have none: their factor is 0, and 0 times what is not finite must not reach them.
// With the zeros in every call 8 x 4096 tokens take 54.3 us (without 53.7), the gradient 91.0 (89.5).
template <bool PAIRS, bool PART>
__device__ __forceinline__ void partners(const float2 (&x)[4], const Lane& a, float2 (&q)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i].x = PAIRS ? x[i].y : x[i ^ 2].x;
        q[i].y = PAIRS ? x[i].x : x[i ^ 2].y;
    }
    if (PART && !a.rotated) q[0] = q[1] = q[2] = q[3] = both(0.f);
}

__device__ __forceinline__ void load_weight(const float* w, const Lane& a, float2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = both(1.f);
    if (!w || !a.active) return;
    Vec8<float> v;
    v.load(w + a.ch, a.second);
    v.get(x);
}

template <int LANES> __device__ __forceinline__ float row_sum(float2 a, float2 b) {
    return lane_group_sum<LANES>((a.x + a.y) + (b.x + b.y));
}

// A run of `hp` heads of q (the first nq runs) or of k, the i-th of them.
struct Run {
    bool is_q;
    int h0, h1, H;
};
__device__ __forceinline__ Run make_run(const RopeParams& p, int i) {
    Run r;
    r.is_q = i < p.nq;
    r.H = r.is_q ? p.Hq : p.Hk;
    r.h0 = (r.is_q ? i : i - p.nq) * p.hp;
    r.h1 = min(r.h0 + p.hp, r.H);
    return r;
}

// The thread's channels of heads h .. h + U - 1, zeros from h1 on and where the thread has none.
template <typename T, int U>
__device__ __forceinline__ void load_heads(Vec8<T> (&v)[U], const T* row, const Lane& a, bool on, int h, int h1,
                                           int d) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (on && h + u < h1) v[u].load(row + (h + u) * d, a.second);
        else v[u].zero();
    }
}

template <typename IN, typename OUT, int LANES, bool PAIRS, bool PART>
__global__ void __launch_bounds__(kRopeThreads, sizeof(IN) == 2 ? 4 : 3) norm_rope_fwd_kernel(const RopeParams p) {
    constexpr int kGroups = kRopeThreads / LANES, U = 4;
    chain_wait();
    chain_release();
    const Lane a = make_lane<LANES>(p);
    const Run run = make_run(p, blockIdx.y);
    const long long ld = run.is_q ? p.ld_q : p.ld_k, ldo = run.is_q ? p.ld_oq : p.ld_ok;
    const IN* x0 = static_cast<const IN*>(run.is_q ? p.q : p.k);
    OUT* y0 = static_cast<OUT*>(run.is_q ? p.oq : p.ok);
    const float inv_d = 1.f / p.d;
    // the trip count is the same for a whole block: every lane takes part in the sums
    for (long long base = (long long)blockIdx.x * kGroups; base < p.tokens;
         base += (long long)gridDim.x * kGroups) {
        const long long tok = base + threadIdx.x / LANES;
        const bool on = tok < p.tokens && a.active;
        const IN* xt = x0 + tok * ld + a.ch;
        OUT* yt = y0 + tok * ldo + a.ch;
        Vec8<IN> v[U];
        load_heads<IN, U>(v, xt, a, on, run.h0, run.h1, p.d);
        float2 A[4], B[4];
        {
            float2 w[4], wp[4];
            load_weight(run.is_q ? p.wq : p.wk, a, w);
            partners<PAIRS, PART>(w, a, wp);
            coefficients(p, a, tok < p.tokens ? tok : 0, A, B);
#pragma unroll
            for (int i = 0; i < 4; ++i) { A[i] = mul2(A[i], w[i]); B[i] = mul2(B[i], wp[i]); }
        }
        for (int h = run.h0; h < run.h1; h += U) {
            if (h > run.h0) load_heads<IN, U>(v, xt, a, on, h, run.h1, p.d);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= run.h1) break;  // uniform
                float2 x[4], q[4], y[4], s0 = both(0.f), s1 = both(0.f);
                v[u].get(x);
                s0 = fma2(x[0], x[0], fma2(x[2], x[2], s0));
                s1 = fma2(x[1], x[1], fma2(x[3], x[3], s1));
                const float2 r = both(rsqrtf(fmaf(row_sum<LANES>(s0, s1), inv_d, p.eps)));
                partners<PAIRS, PART>(x, a, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = mul2(r, fma2(x[i], A[i], mul2(q[i], B[i])));
                if (on) store8(yt + (h + u) * p.d, a.second, y);
            }
        }
    }
}

template <typename IN, typename OUT, int LANES, bool PAIRS, bool PART>
__global__ void __launch_bounds__(kBwdThreads, kBwdResident) norm_rope_bwd_kernel(const RopeParams p) {
    constexpr int kGroups = kBwdThreads / LANES, U = sizeof(IN) == 2 ? kRun : kRun / 2;
    __shared__ float sums[kGroups][LANES * 8 + 1];
    chain_wait();
    chain_release();
    const Lane a = make_lane<LANES>(p);
    // the block's run, its place among the run's blocks, and their number
    const bool of_k = (int)blockIdx.x >= p.bq;
    const int runs = of_k ? p.nk : p.nq;
    int place = of_k ? blockIdx.x - p.bq : blockIdx.x;
    const int i = min(place / p.nb, runs - 1);
    place -= i * p.nb;
    const int of = i < runs - 1 ? p.nb : of_k ? p.nbk : p.nbq;
    const Run run = make_run(p, (of_k ? p.nq : 0) + i);
    const long long ld = run.is_q ? p.ld_q : p.ld_k, ldo = run.is_q ? p.ld_oq : p.ld_ok;
    const IN* x0 = static_cast<const IN*>(run.is_q ? p.q : p.k);
    const IN* g0 = static_cast<const IN*>(run.is_q ? p.dyq : p.dyk);
    OUT* y0 = static_cast<OUT*>(run.is_q ? p.oq : p.ok);
    float2 w[4], dw[4];
    load_weight(run.is_q ? p.wq : p.wk, a, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[i] = both(0.f);
    const float inv_d = 1.f / p.d;
    for (long long base = (long long)place * kGroups; base < p.tokens; base += (long long)of * kGroups) {
        const long long tok = base + threadIdx.x / LANES;
        const bool on = tok < p.tokens && a.active;
        const IN* xt = x0 + tok * ld + a.ch;
        const IN* gt = g0 + tok * run.H * p.d + a.ch;
        OUT* yt = y0 + tok * ldo + a.ch;
        Vec8<IN> v[U], dv[U];
        load_heads<IN, U>(v, xt, a, on, run.h0, run.h1, p.d);
        load_heads<IN, U>(dv, gt, a, on, run.h0, run.h1, p.d);
        float2 C[4], S[4];
        coefficients(p, a, tok < p.tokens ? tok : 0, C, S);
#pragma unroll
        for (int i = 0; i < 4; ++i) { S[i].x = -S[i].x; S[i].y = -S[i].y; }  // the transposed rotation
        for (int h = run.h0; h < run.h1; h += U) {
            if (h > run.h0) {
                load_heads<IN, U>(v, xt, a, on, h, run.h1, p.d);
                load_heads<IN, U>(dv, gt, a, on, h, run.h1, p.d);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= run.h1) break;  // uniform
                float2 x[4], m[4], dy[4], q[4], t[4], s0 = both(0.f), s1 = both(0.f), g0s = s0, g1s = s1;
                v[u].get(x);
                dv[u].get(dy);
                partners<PAIRS, PART>(dy, a, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    m[i] = fma2(dy[i], C[i], mul2(q[i], S[i]));
                    t[i] = mul2(m[i], x[i]);
                }
                s0 = fma2(x[0], x[0], fma2(x[2], x[2], s0));
                s1 = fma2(x[1], x[1], fma2(x[3], x[3], s1));
                g0s = fma2(t[0], w[0], fma2(t[2], w[2], g0s));
                g1s = fma2(t[1], w[1], fma2(t[3], w[3], g1s));
                const float ss = row_sum<LANES>(s0, s1), gx = row_sum<LANES>(g0s, g1s);
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                const float2 r2 = both(r), e = both(-r * r * gx * inv_d);
                float2 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = mul2(r2, fma2(x[i], e, mul2(m[i], w[i])));
                    if (on) dw[i] = fma2(t[i], r2, dw[i]);
                }
                if (on) store8(yt + (h + u) * p.d, a.second, y);
            }
        }
    }
    // this block's part of dw, in a fixed order
    const int group = threadIdx.x / LANES;
    if (a.active) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = a.ch + (i >= 2 ? a.second : 0) + 2 * (i & 1);
            sums[group][ch] = dw[i].x;
            sums[group][ch + 1] = dw[i].y;
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kBwdThreads) {
        float s = 0.f;
#pragma unroll 4
        for (int g = 0; g < kGroups; ++g) s += sums[g][c];
        p.part[(size_t)blockIdx.x * p.d + c] = s;
    }
}

// Sums the blocks' parts of dw: block (i, 0) takes 8 channels of dwq, block (i, 1) of dwk.
__global__ void __launch_bounds__(kRopeThreads) norm_rope_dw_kernel(const RopeParams p) {
    __shared__ float sums[32][9];
    const bool is_q = blockIdx.y == 0;
    float* dw = is_q ? p.dwq : p.dwk;
    chain_wait();  // until the parts are there
    chain_release();
    if (!dw) return;
    const int c = threadIdx.x & 7, j = threadIdx.x >> 3, ch = blockIdx.x * 8 + c;
    const int lo = is_q ? 0 : p.bq, hi = is_q ? p.bq : p.bq + p.bk;
    float s = 0.f;
    for (int i = lo + j; i < hi; i += 32) s += p.part[(size_t)i * p.d + ch];
    sums[j][c] = s;
    __syncthreads();
    if (j == 0) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += sums[i][c];
        dw[ch] = s;
    }
}

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// Heads that a group of threads takes: all threads of the GPU get work before a group gets a
// second head; from then on a run of up to 16 heads shares one token's coefficients and reads 4 KB at
// a time.  8 x 4096 tokens, 20 heads of 128, runs of 16 against runs of 4: forward 54 us (62), gradient
// 91 us (93).
// The backward's blocks, all of them resident at once, are shared out by the heads of the runs.
void split(RopeParams& p, int lanes, bool bwd) {
    const long long rows = p.tokens * (p.Hq + p.Hk), groups = 152ll * 2048 / lanes;
    p.hp = rows < 2 * groups ? 1 : rows < 4 * groups ? 2 : rows < 16 * groups ? kRun : 16;
    p.nq = (p.Hq + p.hp - 1) / p.hp;
    p.nk = (p.Hk + p.hp - 1) / p.hp;
    if (!bwd) return;
    const int per = kBwdThreads / lanes;
    const long long tiles = (p.tokens + per - 1) / per;
    auto blocks = [&](int heads) {
        long long n = (long long)kBwdBlocks * heads / (p.Hq + p.Hk);
        n = n < 1 ? 1 : n;
        return (int)(n < tiles ? n : tiles);
    };
    p.nb = blocks(p.hp);
    p.nbq = p.nq ? blocks(p.Hq - (p.nq - 1) * p.hp) : 0;
    p.nbk = p.nk ? blocks(p.Hk - (p.nk - 1) * p.hp) : 0;
    p.bq = p.nq ? (p.nq - 1) * p.nb + p.nbq : 0;
    p.bk = p.nk ? (p.nk - 1) * p.nb + p.nbk : 0;
}

template <typename IN, typename OUT, int LANES, bool PAIRS, bool PART>
cudaError_t launch(const RopeParams& p, bool bwd, cudaStream_t st) {
    constexpr int kGroups = kRopeThreads / LANES;
    if (!bwd) {
        const long long tiles = (p.tokens + kGroups - 1) / kGroups;
        const dim3 grid((unsigned)(tiles < 0x7fffffff ? tiles : 0x7fffffff), p.nq + p.nk);
        TraceScope ts("norm_rope_fwd", st);
        return launch_chained(norm_rope_fwd_kernel<IN, OUT, LANES, PAIRS, PART>, grid, kRopeThreads, 0, st, p);
    }
    {
        TraceScope ts("norm_rope_bwd", st);
        if (cudaError_t e = launch_chained(norm_rope_bwd_kernel<IN, OUT, LANES, PAIRS, PART>, dim3(p.bq + p.bk), kBwdThreads, 0, st, p);
            e != cudaSuccess)
            return e;
    }
    if (!p.dwq && !p.dwk) return cudaSuccess;
    TraceScope ts("norm_rope_dw", st);
    return launch_chained(norm_rope_dw_kernel, dim3(p.d / 8, 2), kRopeThreads, 0, st, p);
}

template <typename IN, typename OUT, int LANES>
cudaError_t by_rotation(const RopeParams& p, bool bwd, cudaStream_t st) {
    if (p.style == DR_ROPE_PAIRS)
        return p.rot < p.d ? launch<IN, OUT, LANES, true, true>(p, bwd, st) : launch<IN, OUT, LANES, true, false>(p, bwd, st);
    return p.rot < p.d ? launch<IN, OUT, LANES, false, true>(p, bwd, st) : launch<IN, OUT, LANES, false, false>(p, bwd, st);
}
template <typename IN, typename OUT>
cudaError_t by_lanes(const RopeParams& p, bool bwd, cudaStream_t st) {
    switch (lanes_of(p.d)) {
        case 4: return by_rotation<IN, OUT, 4>(p, bwd, st);
        case 8: return by_rotation<IN, OUT, 8>(p, bwd, st);
        case 16: return by_rotation<IN, OUT, 16>(p, bwd, st);
        default: return by_rotation<IN, OUT, 32>(p, bwd, st);
    }
}

}  // namespace

size_t norm_rope_part_bytes(RopeParams p) {
    split(p, lanes_of(p.d), true);
    return (size_t)(p.bq + p.bk) * p.d * sizeof(float);
}

cudaError_t norm_rope(RopeParams p, bool bwd, int io, int out, cudaStream_t st) {
    split(p, lanes_of(p.d), bwd);
    if (io == DR_BF16)
        return out == DR_BF16 ? by_lanes<__nv_bfloat16, __nv_bfloat16>(p, bwd, st)
                              : by_lanes<__nv_bfloat16, float>(p, bwd, st);
    return out == DR_BF16 ? by_lanes<float, __nv_bfloat16>(p, bwd, st)
                          : by_lanes<float, float>(p, bwd, st);
}

}  // namespace dr
