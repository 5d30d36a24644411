// linear_attn.cu -- linear attention with a decay for each head on the CUDA cores, fp32 arithmetic: the
// chunked scan of linear_attn.cuh (dr.h, dr_linear_attn_fwd / dr_linear_attn_bwd) and the recurrent step
// (dr_linear_attn_step).
//
// fp32 prompts only (bf16 ones are scanned on the tensor cores); 2635 packed tokens in 5 sequences, 8 heads of 32 and 64:
// forward 63 us in three kernels, gradient 128 us in five, bound by issue slots and the chain of a chunk (loads, three
// products, 8 us).
//
// The scan in chunks of C = 64 tokens, i and j within the chunk, X the state before it, a = e^g:
//   out_i = sum_{j<=i} a^{i-j} (q_i.k_j) v_j + a^{i+1} X^T q_i;   X' = a^C X + sum_j a^{C-1-j} k_j v_j^T
// (reverse: a^i X^T q_i and X' = a^C X + sum_j a^{C-j} k_j v_j^T).  Columns of v and of the state do not meet,
// so a block has one sequence, one head and up to 32 columns; the products q_i.k_j are formed by each.
#include <algorithm>

#include "common.cuh"
#include "linear_work.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256, kChunk = 64;

template <int DK, int W> struct ScanSmem {  // pitches: 16-byte reads of eight rows meet all banks
    static constexpr int pk = DK + 4, pw = W + 4, pa = kChunk + 4;
    static constexpr int k = kChunk * pk, v = 2 * kChunk * pk, a = v + kChunk * pw, x = a + kChunk * pa,
                         floats = x + DK * pw;
};

// N neighbouring values, N = 1, 2, or a multiple of 4.
template <int N> __device__ __forceinline__ void load_row(float (&x)[N], const float* p) {
    if constexpr (N == 1) {
        x[0] = *p;
    } else if constexpr (N == 2) {
        const float2 y = *reinterpret_cast<const float2*>(p);
        x[0] = y.x; x[1] = y.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 y = *reinterpret_cast<const float4*>(p + i);
            x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
        }
    }
}
// Scans of the same sizes, side by side (blockIdx.z).
struct ScanSet {
    ScanParams p[kMostScans];
};
// ONLY: the segments' own states, from nothing.
template <int DK, int W, bool ONLY>
__global__ void __launch_bounds__(kThreads, 2) linear_scan_kernel(const __grid_constant__ ScanSet set) {
    const ScanParams& p = set.p[blockIdx.z];
    using L = ScanSmem<DK, W>;
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = sm + L::k, *V = sm + L::v, *A = sm + L::a, *X = sm + L::x;
    __shared__ float pw[kChunk + 1];  // a^n
    const int h = blockIdx.x % p.H, w0 = blockIdx.y * W;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    constexpr int WX = W / 16, RX = DK / 16;  // a thread's columns; its rows of the state
    Work w;
    if (!make_work(p, blockIdx.x / p.H, h, w) || (ONLY && (!w.before || w.last))) return;
    const int begin = w.c0 * kScanChunk, end = min(w.len, begin + w.chunks * kScanChunk), len = end - begin;
    const float g = p.g[h];
    if (threadIdx.x <= kChunk) pw[threadIdx.x] = decay(g, (float)threadIdx.x);
    const size_t unit = ((size_t)w.seq * p.H + h) * DK * p.dv;
    const float* from = ONLY ? nullptr : w.before ? w.before : p.x0 ? p.x0 + unit : nullptr;
    const bool turned = p.x0_transposed && !w.before;
    for (int i = threadIdx.x; i < DK * W; i += kThreads) {
        const int r = i / W, c = w0 + i % W;
        X[r * L::pw + i % W] = from ? from[turned ? c * DK + r : r * p.dv + c] : 0.f;
    }
    const float f_in = p.reverse ? p.scale : 1.f, f_out = p.reverse ? 1.f : p.scale;
    const int late = p.reverse ? 1 : 0;
    for (int t0 = 0; t0 < len; t0 += kChunk) {
        const int n = min(kChunk, len - t0);
        __syncthreads();
        auto token = [&](int i) { return (long long)w.row0 + (p.reverse ? end - 1 - t0 - i : begin + t0 + i); };
        {   // everything is on its way before the first of it is stored
            constexpr int NK = kChunk * DK / 4 / kThreads, NV = kChunk * W / 4 / kThreads > 0 ? kChunk * W / 4 / kThreads : 1;
            static_assert(NK * kThreads == kChunk * DK / 4 && NV * kThreads >= kChunk * W / 4, "pieces of the threads");
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 q[NK], k[NK], v[NV];
#pragma unroll
            for (int m = 0; m < NK; ++m) {
                const int i = threadIdx.x + m * kThreads, r = i / (DK / 4), c = (i % (DK / 4)) * 4;
                q[m] = !ONLY && r < n ? load4(static_cast<const float*>(p.q) + token(r) * p.ld_q + (long long)h * DK + c) : zero;
                k[m] = r < n ? load4(static_cast<const float*>(p.k) + token(r) * p.ld_k + (long long)h * DK + c) : zero;
            }
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int i = threadIdx.x + m * kThreads, r = i / (W / 4), c = (i % (W / 4)) * 4;
                v[m] = r < n ? load4(static_cast<const float*>(p.v) + token(r) * p.ld_v + (long long)h * p.dv + w0 + c) : zero;
            }
#pragma unroll
            for (int m = 0; m < NK; ++m) {
                const int i = threadIdx.x + m * kThreads, at = i / (DK / 4) * L::pk + (i % (DK / 4)) * 4;
                if (!ONLY) *reinterpret_cast<float4*>(Q + at) = q[m];
                *reinterpret_cast<float4*>(K + at) = k[m];
            }
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int i = threadIdx.x + m * kThreads;
                if (i < kChunk * W / 4) *reinterpret_cast<float4*>(V + i / (W / 4) * L::pw + (i % (W / 4)) * 4) = v[m];
            }
        }
        __syncthreads();
        if (!ONLY) {  // weights of the pairs: rows 4 ty + i, columns tx + 16 j
            float acc[4][4] = {};
#pragma unroll 4
            for (int c = 0; c < DK; c += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = *reinterpret_cast<const float4*>(Q + (4 * ty + i) * L::pk + c);
                    b[i] = *reinterpret_cast<const float4*>(K + (tx + 16 * i) * L::pk + c);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                        acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                        acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                        acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int back = 4 * ty + i - (tx + 16 * j);
                    A[(4 * ty + i) * L::pa + tx + 16 * j] = back >= 0 ? acc[i][j] * pw[back] * f_in : 0.f;
                }
        }
        __syncthreads();
        if (!ONLY) {  // out: rows 4 ty + i, columns WX tx ..
            float o[4][WX] = {}, r[4][WX] = {};
#pragma unroll 2
            for (int c = 0; c < kChunk; c += 4) {
                float4 a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * L::pa + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float v[WX];
                    load_row(v, V + (c + k) * L::pw + WX * tx);
#pragma unroll
                    for (int w = 0; w < WX; ++w)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i][w] = fmaf(k == 0 ? a[i].x : k == 1 ? a[i].y : k == 2 ? a[i].z : a[i].w, v[w], o[i][w]);
                }
            }
#pragma unroll 2
            for (int c = 0; c < DK; c += 4) {
                float4 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(Q + (4 * ty + i) * L::pk + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[WX];
                    load_row(x, X + (c + k) * L::pw + WX * tx);
#pragma unroll
                    for (int w = 0; w < WX; ++w)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            r[i][w] = fmaf(k == 0 ? q[i].x : k == 1 ? q[i].y : k == 2 ? q[i].z : q[i].w, x[w], r[i][w]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * ty + i < n)
#pragma unroll
                    for (int w = 0; w < WX; ++w) {
                        const float y = f_out * fmaf(pw[4 * ty + i + 1 - late], r[i][w], o[i][w]);
                        static_cast<float*>(p.out)[token(4 * ty + i) * p.ld_o + (long long)h * p.dv + w0 + WX * tx + w] = y;
                    }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n * W; i += kThreads) V[i / W * L::pw + i % W] *= pw[n - 1 - i / W + late] * f_in;
        __syncthreads();
        {   // the state: rows RX ty ..
            float x[RX][WX];
            const float a = pw[n];
#pragma unroll
            for (int i = 0; i < RX; ++i)
#pragma unroll
                for (int w = 0; w < WX; ++w) x[i][w] = a * X[(RX * ty + i) * L::pw + WX * tx + w];
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                float v[WX], k[RX];
                load_row(v, V + j * L::pw + WX * tx);
                load_row(k, K + j * L::pk + RX * ty);
#pragma unroll
                for (int i = 0; i < RX; ++i)
#pragma unroll
                    for (int w = 0; w < WX; ++w) x[i][w] = fmaf(k[i], v[w], x[i][w]);
            }
#pragma unroll
            for (int i = 0; i < RX; ++i)
#pragma unroll
                for (int w = 0; w < WX; ++w) X[(RX * ty + i) * L::pw + WX * tx + w] = x[i][w];
        }
    }
    __syncthreads();
    float* to = ONLY ? const_cast<float*>(w.before) : w.last && p.xT ? p.xT + unit : nullptr;
    if (to)
        for (int i = threadIdx.x; i < DK * W; i += kThreads) to[(i / W) * p.dv + w0 + i % W] = X[(i / W) * L::pw + i % W];
}

template <int DK, int W, bool ONLY> cudaError_t scan(const ScanSet& set, int n, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    constexpr int smem = ScanSmem<DK, W>::floats * 4;
    if (cudaError_t e = set_smem_once(linear_scan_kernel<DK, W, ONLY>, smem, ready); e != cudaSuccess) return e;
    const long long blocks = scan_items(set.p[0]) * set.p[0].H;
    if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
    TraceScope ts(ONLY ? "linear_segments" : "linear_scan", st);
    linear_scan_kernel<DK, W, ONLY><<<dim3((unsigned)blocks, set.p[0].dv / W, n), kThreads, smem, st>>>(set);
    return cudaGetLastError();
}
template <int DK> cudaError_t scan_width(const ScanSet& set, int n, bool only, cudaStream_t st) {
    if (set.p[0].dv == 16) return only ? scan<DK, 16, true>(set, n, st) : scan<DK, 16, false>(set, n, st);
    return only ? scan<DK, 32, true>(set, n, st) : scan<DK, 32, false>(set, n, st);
}
cudaError_t scan_simt(const ScanSet& set, int n, bool only, cudaStream_t st) {
    switch (set.p[0].dk) {
        case 16: return scan_width<16>(set, n, only, st);
        case 32: return scan_width<32>(set, n, only, st);
        case 64: return scan_width<64>(set, n, only, st);
        default: return scan_width<128>(set, n, only, st);
    }
}

// ------------------------------------------------------------------ segments
// The states that the segments begin with, over the segments' own: four values per thread.
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ ScanSet set) {
    const ScanParams& p = set.p[blockIdx.z];
    const int seq = blockIdx.x / p.H, head = blockIdx.x % p.H, R = p.span * kScanChunk, size = p.dk * p.dv;
    int row0, len;
    seq_rows(p.s, seq, row0, len);
    const int tiles = (len + R - 1) / R;
    if (tiles < 2) return;
    const long long slot = slots_before(p.s, R, seq);
    if (slot + tiles > p.slots) return;  // offsets out of order, as in make_work
    const int i = 4 * (blockIdx.y * 256 + threadIdx.x);
    if (i >= size) return;
    const float g = p.g[head];
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.x0) {
        const float* from = p.x0 + ((size_t)seq * p.H + head) * size;
        if (p.x0_transposed) {
            const int r = i / p.dv, c = i % p.dv;
            x = make_float4(from[c * p.dk + r], from[(c + 1) * p.dk + r], from[(c + 2) * p.dk + r], from[(c + 3) * p.dk + r]);
        } else {
            x = load4(from + i);
        }
    }
    const long long step = (p.reverse ? -1ll : 1ll) * p.H * size;
    float* at = p.part + ((slot + (p.reverse ? tiles - 1 : 0)) * p.H + head) * size + i;
    // four segments' own states are read at once (the last segment's was not formed, nothing comes after it)
    for (int n = 0; n < tiles; n += 4) {
        float4 own[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) own[k] = n + k + 1 < tiles ? load4(at + k * step) : x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (n + k >= tiles) break;
            store4(at + k * step, x);
            const int t = p.reverse ? tiles - 1 - n - k : n + k;
            const float a = decay(g, (float)min(R, len - t * R));
            x = make_float4(fmaf(a, x.x, own[k].x), fmaf(a, x.y, own[k].y), fmaf(a, x.z, own[k].z), fmaf(a, x.w, own[k].w));
        }
        at += 4 * step;
    }
}


// ------------------------------------------------------------------ the recurrent step
// A block has one sequence and head, each thread four columns of R rows of the state in registers:
//   X = a X + k_t v_t^T;  o_t = scale X^T q_t
// 64 sequences, 16 heads of 128 x 128: 22 to 24 us for 134 MB of states, 5.7 TB/s, bound by HBM.
// The state is read and written once, a row of it at a time by neighbouring lanes.  The tokens' parts of o
// are summed in shared memory, eight tokens at a time, so that no token waits for another.
constexpr int kTokens = 8;
template <int DK, int DV, typename IO> __global__ void __launch_bounds__(kThreads) linear_step_kernel(const StepParams p) {
    constexpr int L = DV / 4;                                       // lanes of a row
    constexpr int G = kThreads / L < DK ? kThreads / L : DK;        // rows at a time
    constexpr int R = DK / G, GW = 32 / L, PARTS = G / GW > 0 ? G / GW : 1;  // rows of a thread; groups in a warp; warps
    __shared__ __align__(16) float q[kTokens][DK], k[kTokens][DK], v[kTokens][DV], part[kTokens][PARTS][DV];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    const bool on = grp < G;
    float* S = p.state + ((size_t)b * p.H + h) * DK * DV;
    float4 x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = on ? load4(S + (size_t)(grp + i * G) * DV + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float a = expf(p.g[h]);
    for (int t0 = 0; t0 < p.T; t0 += kTokens) {
        const int n = min(kTokens, p.T - t0);
        const long long tok = (long long)b * p.T + t0;
        if (t0) __syncthreads();
        for (int i = threadIdx.x; i < n * (DK / 4); i += kThreads) {
            const int t = i / (DK / 4), c = (i % (DK / 4)) * 4;
            *reinterpret_cast<float4*>(&q[t][c]) = load4(static_cast<const IO*>(p.q) + (tok + t) * p.ld_q + (long long)h * DK + c);
            *reinterpret_cast<float4*>(&k[t][c]) = load4(static_cast<const IO*>(p.k) + (tok + t) * p.ld_k + (long long)h * DK + c);
        }
        for (int i = threadIdx.x; i < n * L; i += kThreads) {
            const int t = i / L, c = (i % L) * 4;
            *reinterpret_cast<float4*>(&v[t][c]) = load4(static_cast<const IO*>(p.v) + (tok + t) * p.ld_v + (long long)h * DV + c);
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on) {
                const float4 w = *reinterpret_cast<const float4*>(&v[t][4 * lane]);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float kk = k[t][grp + i * G], qq = q[t][grp + i * G];
                    x[i].x = fmaf(a, x[i].x, kk * w.x); o.x = fmaf(qq, x[i].x, o.x);
                    x[i].y = fmaf(a, x[i].y, kk * w.y); o.y = fmaf(qq, x[i].y, o.y);
                    x[i].z = fmaf(a, x[i].z, kk * w.z); o.z = fmaf(qq, x[i].z, o.z);
                    x[i].w = fmaf(a, x[i].w, kk * w.w); o.w = fmaf(qq, x[i].w, o.w);
                }
            }
#pragma unroll
            for (int d = L; d < 32; d <<= 1) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
                o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
            }
            if (on && (threadIdx.x & 31) < L) *reinterpret_cast<float4*>(&part[t][threadIdx.x >> 5][4 * lane]) = o;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n * L; i += kThreads) {
            const int t = i / L, c = (i % L) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < PARTS; ++w) {
                const float4 y = *reinterpret_cast<const float4*>(&part[t][w][c]);
                o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
            }
            store4(static_cast<IO*>(p.o) + ((tok + t) * p.H + h) * DV + c,
                   make_float4(p.scale * o.x, p.scale * o.y, p.scale * o.z, p.scale * o.w));
        }
    }
    if (on)
#pragma unroll
        for (int i = 0; i < R; ++i) store4(S + (size_t)(grp + i * G) * DV + 4 * lane, x[i]);
}

template <int DK, int DV, typename IO> cudaError_t step(const StepParams& p, cudaStream_t st) {
    TraceScope ts("linear_step", st);
    linear_step_kernel<DK, DV, IO><<<p.B * p.H, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <int DK, typename IO> cudaError_t step_width(const StepParams& p, cudaStream_t st) {
    switch (p.dv) {
        case 16: return step<DK, 16, IO>(p, st);
        case 32: return step<DK, 32, IO>(p, st);
        case 64: return step<DK, 64, IO>(p, st);
        default: return step<DK, 128, IO>(p, st);
    }
}
template <typename IO> cudaError_t step_of(const StepParams& p, cudaStream_t st) {
    switch (p.dk) {
        case 16: return step_width<16, IO>(p, st);
        case 32: return step_width<32, IO>(p, st);
        case 64: return step_width<64, IO>(p, st);
        default: return step_width<128, IO>(p, st);
    }
}

}  // namespace

// Blocks that run at once; from how many chunks on, and into how few, sequences are split.  On the tensor cores a block
// has an SM to itself and its start costs about two chunks; on the CUDA cores two share one.  The numbers are those of
// 152 SMs; with others sequences would be split in other places, to the same results but for the rounding.
// bf16, forward + gradient in us.  One sequence, 4 heads of 128, whole and split: 8 chunks 33 + 33 and 41 + 42, 12 chunks
// 43 + 43 and 41 + 43, 20 chunks 66 + 66 and 41 + 43: split from 12 on.  Three of 2000 tokens, segments of at least 2, 4
// and 8 chunks: 41 + 53, 48 + 53, 65 + 70; four of 4096, 8 heads of 128: 84 + 175, 84 + 175, 74 + 175.
int scan_span(int io, long long rows, int N, int T, bool packed, int H, int dk, int dv, int scans) {
    if (rows == 0 || N == 0) return 0;
    const bool tc = io == DR_BF16;
    const int room = tc ? 152 : 304, least = tc ? 4 : 1;
    const long long units = (long long)N * H * (tc ? scans : std::max(std::min(dk, dv) / 32, 1));  // on the CUDA cores not all together
    const long long chunks = packed ? rows / kScanChunk + N : (long long)N * ((T + kScanChunk - 1) / kScanChunk);  // of all sequences
    if (chunks < (tc ? 12 : 2)) return 0;
    long long span;
    if (!packed || N == 1) {
        const long long segments = room / units;  // as many as there are blocks for in one go
        if (segments < 2 || chunks / N < (tc ? 12 : 2)) return 0;
        span = (chunks / N + segments - 1) / segments;
    } else {
        // Lengths are known on the device only.  On the tensor cores, where a split costs more, only what is far longer than
        // a block's share of all chunks: never, from 5/2 shares on, from one on (us, forward + gradient):
        //   16 documents of 1 to 2500 tokens, 8 heads of 64 x 128   61 + 146    71 + 163    86 + 164
        //   64 of 1 to 600, the same heads                          59 + 175    77 + 218    80 + 219
        //   8 of 4096, 16 heads of 128                             112 + 296   124 + 314   230 + 315
        //   16384 and four of 50 to 1000, 8 heads of 128           368 + 366   121 + 296    77 + 151
        //   two of 8000 and 30 of 100, 4 heads of 64               165 + 172    65 + 157    44 + 84
        // The 10 to 43 us that a split costs where no sequence is that long are two launches with nothing to do.
        span = ((tc ? 5 : 2) * chunks * (units / N) / 2 + room - 1) / room;
    }
    return (int)std::min<long long>(std::max<long long>(span, least), 1 << 22);
}
long long scan_slots(long long rows, int span) {
    // sequences of several segments: no more than twice as many as whole segments
    return span ? 2 * (rows / ((long long)span * kScanChunk) + 1) : 0;
}

cudaError_t linear_scans(const ScanParams* p, int n, int io, cudaStream_t st) {
    const bool tc = io == DR_BF16 && p->rows > 0;
    auto all = [&](bool only) {
        if (tc) return linear_scans_tc(p, n, only, st);
        for (int i = 0, m; i < n; i += m) {  // scans of the same sizes follow one another
            ScanSet set;
            for (m = 0; i + m < n && p[i + m].dk == p[i].dk && p[i + m].dv == p[i].dv; ++m) set.p[m] = p[i + m];
            if (cudaError_t e = scan_simt(set, m, only, st); e != cudaSuccess) return e;
        }
        return cudaSuccess;
    };
    if (p->rows > 0 && p->span) {
        if (cudaError_t e = all(true); e != cudaSuccess) return e;
        ScanSet set;
        for (int i = 0; i < n; ++i) set.p[i] = p[i];
        TraceScope ts("linear_join", st);
        const dim3 grid((unsigned)(p->s.N * p->H), (p->dk * p->dv + 1023) / 1024, n);
        linear_join_kernel<<<grid, 256, 0, st>>>(set);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    return all(false);
}
cudaError_t linear_step(const StepParams& p, int io, cudaStream_t st) {
    return io == DR_F32 ? step_of<float>(p, st) : step_of<__nv_bfloat16>(p, st);
}

}  // namespace dr
