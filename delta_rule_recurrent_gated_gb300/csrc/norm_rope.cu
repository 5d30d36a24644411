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
// run of its heads; a thread owns 8 consecutive channels, one 16-byte access of a bf16 row.
// The partner of a "halves" pair sits rot / 16 lanes away (one shuffle), that of a "pairs"
// pair in the same thread.  Both kernels are bound by HBM: each value is read and written once.
#include "common.cuh"
#include "rope.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRun = 4;                           // heads of a run, at most; bf16: all loaded at once
constexpr int kBwdResident = 2;                   // blocks of the backward kernel on an SM
constexpr int kBwdBlocks = 152 * kBwdResident;    // over all runs of heads

template <typename T>
struct Vec8;  // 8 consecutive values as loaded
template <>
struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        u = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    // the values of lane `src` of the warp
    __device__ __forceinline__ Vec8 from_lane(int src) const {
        Vec8 o;
        o.u.x = __shfl_sync(0xffffffffu, u.x, src);
        o.u.y = __shfl_sync(0xffffffffu, u.y, src);
        o.u.z = __shfl_sync(0xffffffffu, u.z, src);
        o.u.w = __shfl_sync(0xffffffffu, u.w, src);
        return o;
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ Vec8 from_lane(int src) const {
        Vec8 o;
        o.a.x = __shfl_sync(0xffffffffu, a.x, src);
        o.a.y = __shfl_sync(0xffffffffu, a.y, src);
        o.a.z = __shfl_sync(0xffffffffu, a.z, src);
        o.a.w = __shfl_sync(0xffffffffu, a.w, src);
        o.b.x = __shfl_sync(0xffffffffu, b.x, src);
        o.b.y = __shfl_sync(0xffffffffu, b.y, src);
        o.b.z = __shfl_sync(0xffffffffu, b.z, src);
        o.b.w = __shfl_sync(0xffffffffu, b.w, src);
        return o;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&y)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&y)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}

// What a thread needs of its place: which channels it holds and where their partners are.
struct Lane {
    int l, ch;      // lane of its group, first channel
    bool active;    // holds channels at all (d / 8 need not be a power of two)
    int partner;    // warp lane that holds the partners (halves)
    float sign;     // halves: -1 in the first half of the rotated channels, +1 in the second, 0 outside
    int angle;      // first angle index of the thread's channels
};
template <int LANES>
__device__ __forceinline__ Lane make_lane(const RopeParams& p) {
    Lane a;
    a.l = threadIdx.x % LANES;
    a.ch = a.l * 8;
    a.active = a.ch < p.d;
    const int half = p.rot / 2, me = threadIdx.x & 31;
    a.partner = me;
    a.sign = 0.f;
    a.angle = 0;
    if (p.style == DR_ROPE_PAIRS) {
        a.angle = a.ch / 2;
    } else if (a.ch < half) {
        a.partner = me + half / 8;
        a.sign = -1.f;
        a.angle = a.ch;
    } else if (a.ch < p.rot) {
        a.partner = me - half / 8;
        a.sign = 1.f;
        a.angle = a.ch - half;
    }
    return a;
}

// cos and signed sin of the thread's 8 channels at the token's position: the coefficients of
// the rotation y_c = n_c C_c + n_p S_c.  Outside the rotated channels C = 1, S = 0; NaN where
// the position lies outside the table.
__device__ __forceinline__ void coefficients(const RopeParams& p, const Lane& a, long long tok,
                                             float (&C)[8], float (&S)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { C[i] = 1.f; S[i] = 0.f; }
    if (p.rot == 0 || !a.active) return;
    const long long b = tok / p.T;
    long long pos = p.positions ? p.positions[tok] : tok - b * p.T;
    if (p.start) pos += p.start[b];
    const bool in = pos >= 0 && pos < p.table_rows;
    const float bad = __uint_as_float(0x7fc00000u);
    if (!in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) C[i] = S[i] = bad;
        return;
    }
    if (a.ch >= p.rot) return;
    const size_t at = (size_t)pos * (p.rot / 2) + a.angle;
    const float4* c4 = reinterpret_cast<const float4*>(p.cos_t + at);
    const float4* s4 = reinterpret_cast<const float4*>(p.sin_t + at);
    if (p.style == DR_ROPE_PAIRS) {
        const float4 c = c4[0], s = s4[0];
        const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            C[2 * j] = C[2 * j + 1] = cv[j];
            S[2 * j] = -sv[j];
            S[2 * j + 1] = sv[j];
        }
    } else {
        const float4 c0 = c4[0], c1 = c4[1], s0 = s4[0], s1 = s4[1];
        const float cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) { C[i] = cv[i]; S[i] = a.sign * sv[i]; }
    }
}

// The partners' values of a thread's 8 channels.
template <typename T>
__device__ __forceinline__ void partners(const Vec8<T>& v, const float (&x)[8], const Lane& a,
                                         bool pairs, float (&xp)[8]) {
    if (pairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) xp[i] = x[i ^ 1];
    } else {
        v.from_lane(a.partner).get(xp);
    }
}

__device__ __forceinline__ void load_weight(const float* w, const Lane& a, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = w && a.active ? w[a.ch + i] : 1.f;
}

// blockIdx.y: a run of `hp` heads of q (the first nq of them) or of k
struct Run {
    bool is_q;
    int h0, h1, H;
};
__device__ __forceinline__ Run make_run(const RopeParams& p) {
    Run r;
    r.is_q = (int)blockIdx.y < p.nq;
    r.H = r.is_q ? p.Hq : p.Hk;
    r.h0 = (r.is_q ? (int)blockIdx.y : (int)blockIdx.y - p.nq) * p.hp;
    r.h1 = min(r.h0 + p.hp, r.H);
    return r;
}

// The thread's channels of heads h .. h + U - 1, zeros from h1 on and where the thread has none.
template <typename T, int U>
__device__ __forceinline__ void load_heads(Vec8<T> (&v)[U], const T* row, bool on, int h, int h1, int d) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (on && h + u < h1) v[u].load(row + (long long)(h + u) * d);
        else v[u].zero();
    }
}

template <typename IN, typename OUT, int LANES>
__global__ void __launch_bounds__(kRopeThreads, 3) norm_rope_fwd_kernel(const RopeParams p) {
    constexpr int kGroups = kRopeThreads / LANES, U = sizeof(IN) == 2 ? kRun : kRun / 2;
    const Lane a = make_lane<LANES>(p);
    const Run run = make_run(p);
    const bool pairs = p.style == DR_ROPE_PAIRS;
    const long long ld = run.is_q ? p.ld_q : p.ld_k, ldo = run.is_q ? p.ld_oq : p.ld_ok;
    const IN* x0 = static_cast<const IN*>(run.is_q ? p.q : p.k);
    OUT* y0 = static_cast<OUT*>(run.is_q ? p.oq : p.ok);
    float w[8];
    load_weight(run.is_q ? p.wq : p.wk, a, w);
    const float inv_d = 1.f / p.d;
    // the trip count is the same for a whole block: every lane takes part in the shuffles
    for (long long base = (long long)blockIdx.x * kGroups; base < p.tokens;
         base += (long long)gridDim.x * kGroups) {
        const long long tok = base + threadIdx.x / LANES;
        const bool on = tok < p.tokens && a.active;
        const IN* xt = x0 + tok * ld + a.ch;
        OUT* yt = y0 + tok * ldo + a.ch;
        Vec8<IN> v[U];
        load_heads<IN, U>(v, xt, on, run.h0, run.h1, p.d);
        float A[8], Bc[8], wp[8];
        coefficients(p, a, tok < p.tokens ? tok : 0, A, Bc);
        if (pairs) {
#pragma unroll
            for (int i = 0; i < 8; ++i) wp[i] = w[i ^ 1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) wp[i] = __shfl_sync(0xffffffffu, w[i], a.partner);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) { A[i] *= w[i]; Bc[i] *= wp[i]; }
        for (int h = run.h0; h < run.h1; h += U) {
            if (h > run.h0) load_heads<IN, U>(v, xt, on, h, run.h1, p.d);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= run.h1) break;  // uniform
                float x[8], xp[8], y[8], ss = 0.f;
                v[u].get(x);
                partners(v[u], x, a, pairs, xp);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                ss = lane_group_sum<LANES>(ss);
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = r * fmaf(x[i], A[i], xp[i] * Bc[i]);
                if (on) store8(yt + (long long)(h + u) * p.d, y);
            }
        }
    }
}

template <typename IN, typename OUT, int LANES>
__global__ void __launch_bounds__(kRopeThreads, kBwdResident) norm_rope_bwd_kernel(const RopeParams p) {
    constexpr int kGroups = kRopeThreads / LANES, U = sizeof(IN) == 2 ? kRun : kRun / 2;
    __shared__ float sums[kGroups][LANES * 8 + 1];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Lane a = make_lane<LANES>(p);
    const Run run = make_run(p);
    const bool pairs = p.style == DR_ROPE_PAIRS;
    const long long ld = run.is_q ? p.ld_q : p.ld_k, ldo = run.is_q ? p.ld_oq : p.ld_ok;
    const IN* x0 = static_cast<const IN*>(run.is_q ? p.q : p.k);
    const IN* g0 = static_cast<const IN*>(run.is_q ? p.dyq : p.dyk);
    OUT* y0 = static_cast<OUT*>(run.is_q ? p.oq : p.ok);
    float w[8], dw[8] = {};
    load_weight(run.is_q ? p.wq : p.wk, a, w);
    const float inv_d = 1.f / p.d;
    for (long long base = (long long)blockIdx.x * kGroups; base < p.tokens;
         base += (long long)gridDim.x * kGroups) {
        const long long tok = base + threadIdx.x / LANES;
        const bool on = tok < p.tokens && a.active;
        const IN* xt = x0 + tok * ld + a.ch;
        const IN* gt = g0 + tok * run.H * p.d + a.ch;
        OUT* yt = y0 + tok * ldo + a.ch;
        Vec8<IN> v[U], dv[U];
        load_heads<IN, U>(v, xt, on, run.h0, run.h1, p.d);
        load_heads<IN, U>(dv, gt, on, run.h0, run.h1, p.d);
        float C[8], S[8];
        coefficients(p, a, tok < p.tokens ? tok : 0, C, S);
        for (int h = run.h0; h < run.h1; h += U) {
            if (h > run.h0) {
                load_heads<IN, U>(v, xt, on, h, run.h1, p.d);
                load_heads<IN, U>(dv, gt, on, h, run.h1, p.d);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= run.h1) break;  // uniform
                float x[8], m[8], dy[8], dyp[8], ss = 0.f, gx = 0.f;
                v[u].get(x);
                dv[u].get(dy);
                partners(dv[u], dy, a, pairs, dyp);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // the transposed rotation: the sine with the other sign
                    m[i] = fmaf(dy[i], C[i], -dyp[i] * S[i]);
                    ss = fmaf(x[i], x[i], ss);
                    gx = fmaf(m[i] * w[i], x[i], gx);
                }
                ss = lane_group_sum<LANES>(ss);
                gx = lane_group_sum<LANES>(gx);
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                const float e = r * r * gx * inv_d;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = r * fmaf(-x[i], e, m[i] * w[i]);
                    if (on) dw[i] = fmaf(m[i], x[i] * r, dw[i]);
                }
                if (on) store8(yt + (long long)(h + u) * p.d, y);
            }
        }
    }
    // this block's part of dw, in a fixed order
    const int group = threadIdx.x / LANES;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[group][a.ch + i] = dw[i];
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kRopeThreads) {
        float s = 0.f;
#pragma unroll 4
        for (int g = 0; g < kGroups; ++g) s += sums[g][c];
        p.part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * p.d + c] = s;
    }
}

// Sums the blocks' parts of dw: block (i, 0) takes 8 channels of dwq, block (i, 1) of dwk.
__global__ void __launch_bounds__(kRopeThreads) norm_rope_dw_kernel(const RopeParams p, int blocks) {
    __shared__ float sums[32][9];
    const bool is_q = blockIdx.y == 0;
    float* dw = is_q ? p.dwq : p.dwk;
    // launched early: until the parts are there (all threads wait, so that the end of this kernel is
    // also the end of the one before)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!dw) return;
    const int c = threadIdx.x & 7, j = threadIdx.x >> 3, ch = blockIdx.x * 8 + c;
    const long long lo = is_q ? 0 : (long long)p.nq * blocks;
    const long long hi = is_q ? (long long)p.nq * blocks : (long long)(p.nq + p.nk) * blocks;
    float s = 0.f;
    for (long long i = lo + j; i < hi; i += 32) s += p.part[i * p.d + ch];
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
// second head; from then on four heads share one token's coefficients (runs of equal length keep
// the backward's blocks, whose number is fixed, equally long).
void split_heads(RopeParams& p, int lanes) {
    const long long rows = p.tokens * (p.Hq + p.Hk), groups = 152ll * 2048 / lanes;
    p.hp = rows < 2 * groups ? 1 : rows < 4 * groups ? 2 : kRun;
    p.nq = (p.Hq + p.hp - 1) / p.hp;
    p.nk = (p.Hk + p.hp - 1) / p.hp;
}

// Blocks of each run in the backward: all of them resident at once.
int bwd_blocks(const RopeParams& p, int lanes) {
    const long long tiles = (p.tokens + kRopeThreads / lanes - 1) / (kRopeThreads / lanes);
    const int runs = p.nq + p.nk, per = runs < kBwdBlocks ? kBwdBlocks / runs : 1;
    return (int)(tiles < per ? tiles : per);
}

template <typename IN, typename OUT, int LANES>
cudaError_t launch(const RopeParams& p, bool bwd, cudaStream_t st) {
    constexpr int kGroups = kRopeThreads / LANES;
    if (!bwd) {
        const long long tiles = (p.tokens + kGroups - 1) / kGroups;
        const dim3 grid((unsigned)(tiles < 0x7fffffff ? tiles : 0x7fffffff), p.nq + p.nk);
        TraceScope ts("norm_rope_fwd", st);
        norm_rope_fwd_kernel<IN, OUT, LANES><<<grid, kRopeThreads, 0, st>>>(p);
        return cudaGetLastError();
    }
    const int blocks = bwd_blocks(p, LANES);
    {
        TraceScope ts("norm_rope_bwd", st);
        norm_rope_bwd_kernel<IN, OUT, LANES><<<dim3(blocks, p.nq + p.nk), kRopeThreads, 0, st>>>(p);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    if (!p.dwq && !p.dwk) return cudaSuccess;
    TraceScope ts("norm_rope_dw", st);
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.d / 8, 2);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, p, blocks);
}

template <typename IN, typename OUT>
cudaError_t by_lanes(const RopeParams& p, bool bwd, cudaStream_t st) {
    switch (lanes_of(p.d)) {
        case 4: return launch<IN, OUT, 4>(p, bwd, st);
        case 8: return launch<IN, OUT, 8>(p, bwd, st);
        case 16: return launch<IN, OUT, 16>(p, bwd, st);
        default: return launch<IN, OUT, 32>(p, bwd, st);
    }
}

}  // namespace

size_t norm_rope_part_bytes(RopeParams p) {
    const int lanes = lanes_of(p.d);
    split_heads(p, lanes);
    return (size_t)(p.nq + p.nk) * bwd_blocks(p, lanes) * p.d * sizeof(float);
}

cudaError_t norm_rope(RopeParams p, bool bwd, int io, int out, cudaStream_t st) {
    split_heads(p, lanes_of(p.d));
    if (io == DR_BF16)
        return out == DR_BF16 ? by_lanes<__nv_bfloat16, __nv_bfloat16>(p, bwd, st)
                              : by_lanes<__nv_bfloat16, float>(p, bwd, st);
    return out == DR_BF16 ? by_lanes<float, __nv_bfloat16>(p, bwd, st)
                          : by_lanes<float, float>(p, bwd, st);
}

}  // namespace dr
