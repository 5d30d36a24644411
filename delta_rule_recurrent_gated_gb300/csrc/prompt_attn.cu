// prompt_attn.cu -- causal attention over whole prompts in fp32, on the CUDA cores (dr.h, dr_prompt_attn_fwd /
// dr_prompt_attn_bwd), and the first step of the gradient for both types.
//
//   s_ij = scale q_i.k_j for the keys j <= i that the window shows;  p_ij = e^{s_ij - lse_i};
//   o_i = sum_j p_ij v_j;  D_i = dO_i.o_i;  ds_ij = p_ij (dO_i.v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_i ds_ij q_i;  dv_j = sum_i p_ij dO_i
//
// A block holds 64 rows (queries, or keys for dk and dv) and streams the other side in tiles.  Every thread of
// a 16 x 16 arrangement has four rows: its part of the scores, and of the sums a sixteenth of the channels.  dk
// and dv are summed over the query heads of a group in order: no atomics, the same bits every time.
// 2635 packed tokens in 5 sequences, 8 query heads of 64, 2 key heads: forward 148 us, dq 213, dk and dv 244 + 12 (723 with a
// block for each key head, which leaves most SMs idle); bound by the operands from shared memory (about 15 TFLOP/s of the
// products that are formed; 4 x 1024 tokens: shared memory 46 to 57 % busy, issue slots 55 to 58, fp32 pipe 42 to 45, 16
// warps an SM) and by the longest sequence's tiles.
#include "common.cuh"
#include "prompt_attn.cuh"
#include "trace.cuh"
#include "vec4.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256, kRows = 64;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -INFINITY;

// Rows of a tile in shared memory are D + 4 floats apart: 16-byte reads of eight rows meet all banks.
template <int D> constexpr int kPitch = D + 4;

// R rows of a tensor from src on, zeros from row n on.
template <int R, int D>
__device__ __forceinline__ void load_tile(float* dst, const float* src, long long ld, int n) {
    for (int i = threadIdx.x; i < R * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        const float4 x = r < n ? load4(src + r * ld + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + r * kPitch<D> + c) = x;
    }
}
// acc[i][j] = rows (4 ty + i) of A times rows (tx + 16 j) of B.
template <int NJ, int D>
__device__ __forceinline__ void dot_rows(float (&acc)[4][NJ], const float* A, const float* B, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 a[4], b[NJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * kPitch<D> + c);
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kPitch<D> + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}
// acc[i][..] += sum_c W[4 ty + i][c] B[c][..]: channels 4 tx + 64 h .. + 3.
template <int NC, int D>
__device__ __forceinline__ void add_rows(float4 (&acc)[4][D / 64], const float* W, const float* B, int ty, int tx) {
    constexpr int P = NC + 4;
#pragma unroll 2
    for (int c = 0; c < NC; c += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(W + (4 * ty + i) * P + c);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 b = *reinterpret_cast<const float4*>(B + (c + k) * kPitch<D> + 64 * h + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = k == 0 ? w[i].x : k == 1 ? w[i].y : k == 2 ? w[i].z : w[i].w;
                    acc[i][h].x = fmaf(x, b.x, acc[i][h].x);
                    acc[i][h].y = fmaf(x, b.y, acc[i][h].y);
                    acc[i][h].z = fmaf(x, b.z, acc[i][h].z);
                    acc[i][h].w = fmaf(x, b.w, acc[i][h].w);
                }
            }
    }
}
template <int D> __device__ __forceinline__ void clear(float4 (&acc)[4][D / 64]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) acc[i][h] = make_float4(0.f, 0.f, 0.f, 0.f);
}
template <int D>
__device__ __forceinline__ void store_rows(float* dst, long long ld, int n, const float4 (&acc)[4][D / 64], const float (&f)[4],
                                           int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * ty + i < n)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const float4 a = acc[i][h];
                store4(dst + (4 * ty + i) * ld + 64 * h + 4 * tx, make_float4(a.x * f[i], a.y * f[i], a.z * f[i], a.w * f[i]));
            }
}
__device__ __forceinline__ bool sees(const PromptParams& p, int i, int j) { return j <= i && (p.window == 0 || j > i - p.window); }

// The block's tile: warp 0 looks it up for all.
struct Place { int row0, len, tile; bool any; };
__device__ __forceinline__ Place place_of(const PromptParams& p, long long item, bool from_end) {
    __shared__ Place at;
    if (threadIdx.x < 32) {
        Place x;
        int seq = 0;
        x.tile = x.row0 = x.len = 0;
        x.any = find_tile(p.s, kRows, item, seq, x.tile);
        if (x.any) seq_rows(p.s, seq, x.row0, x.len);
        if (from_end) x.tile = (x.len + kRows - 1) / kRows - 1 - x.tile;
        if (threadIdx.x == 0) at = x;
    }
    __syncthreads();
    const Place x = at;
    __syncthreads();
    return x;
}

template <int D> __global__ void __launch_bounds__(kThreads, 2) prompt_fwd_kernel(const PromptParams p) {
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *KV = Q + kRows * kPitch<D>, *P = KV + kRows * kPitch<D>;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, h = blockIdx.y, hk = h / p.G;
    const float c2 = p.scale * kLog2e;
    for (long long item = blockIdx.x;; item += gridDim.x) {
        const Place at = place_of(p, item, false);
        if (!at.any) return;
        const int i0 = at.tile * kRows, ni = min(kRows, at.len - i0);
        load_tile<kRows, D>(Q, static_cast<const float*>(p.q) + (at.row0 + i0) * p.ld_q + (long long)h * D, p.ld_q, ni);
        float4 acc[4][D / 64];
        clear<D>(acc);
        float m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = kNegInf, l[i] = 0.f;
        const int first = p.window ? max(0, i0 - p.window + 1) / kRows : 0;
        for (int t = first; t * kRows < i0 + ni; ++t) {
            const int j0 = t * kRows, nj = min(kRows, at.len - j0);
            __syncthreads();
            load_tile<kRows, D>(KV, static_cast<const float*>(p.k) + (at.row0 + j0) * p.ld_k + (long long)hk * D, p.ld_k, nj);
            __syncthreads();
            float s[4][4];
            dot_rows<4, D>(s, Q, KV, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = kNegInf, sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = sees(p, i0 + 4 * ty + i, j0 + tx + 16 * j) ? s[i][j] * c2 : kNegInf;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m2 = fmaxf(m[i], mx), ref = m2 == kNegInf ? 0.f : m2, f = exp2f(m[i] - ref);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = exp2f(s[i][j] - ref);
                    P[(4 * ty + i) * (kRows + 4) + tx + 16 * j] = e;
                    sum += e;
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                l[i] = l[i] * f + sum;
                m[i] = m2;
#pragma unroll
                for (int h2 = 0; h2 < D / 64; ++h2) {
                    acc[i][h2].x *= f; acc[i][h2].y *= f; acc[i][h2].z *= f; acc[i][h2].w *= f;
                }
            }
            __syncthreads();
            load_tile<kRows, D>(KV, static_cast<const float*>(p.v) + (at.row0 + j0) * p.ld_v + (long long)hk * D, p.ld_v, nj);
            __syncthreads();
            add_rows<kRows, D>(acc, P, KV, ty, tx);
        }
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = 1.f / l[i];
        const long long out = ((long long)(at.row0 + i0) * p.Hq + h);
        store_rows<D>(static_cast<float*>(p.o) + out * D, (long long)p.Hq * D, ni, acc, f, ty, tx);
        if (p.lse && tx == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * ty + i < ni) p.lse[out + (long long)(4 * ty + i) * p.Hq] = (m[i] + log2f(l[i])) * kLn2;
        __syncthreads();
    }
}

// D_i = dO_i.o_i: eight lanes for each row and head.
template <int D, typename IO> __global__ void __launch_bounds__(kThreads) prompt_delta_kernel(const PromptParams p) {
    const long long n = p.rows * p.Hq;
    for (long long i0 = (long long)blockIdx.x * (kThreads / 8); i0 < n; i0 += (long long)gridDim.x * (kThreads / 8)) {
        const long long i = i0 + threadIdx.x / 8;
        float sum = 0.f;
        if (i < n)
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                const long long at = i * D + c + 4 * (threadIdx.x & 7);
                const float4 a = load4(static_cast<const IO*>(p.o) + at), b = load4(static_cast<const IO*>(p.dO) + at);
                sum += (a.x * b.x + a.y * b.y) + (a.z * b.z + a.w * b.w);
            }
        sum = lane_group_sum<8>(sum);
        if (i < n && (threadIdx.x & 7) == 0) p.delta[i] = sum;
    }
}

constexpr int kCols = 32;  // rows of a streamed tile of the backward kernels

template <int D> __global__ void __launch_bounds__(kThreads, 2) prompt_dq_kernel(const PromptParams p) {
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *G = Q + kRows * kPitch<D>, *K = G + kRows * kPitch<D>, *V = K + kCols * kPitch<D>, *W = V + kCols * kPitch<D>;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, h = blockIdx.y, hk = h / p.G;
    const float c2 = p.scale * kLog2e;
    for (long long item = blockIdx.x;; item += gridDim.x) {
        const Place at = place_of(p, item, false);
        if (!at.any) return;
        const int i0 = at.tile * kRows, ni = min(kRows, at.len - i0);
        const long long out = ((long long)(at.row0 + i0) * p.Hq + h);
        load_tile<kRows, D>(Q, static_cast<const float*>(p.q) + (at.row0 + i0) * p.ld_q + (long long)h * D, p.ld_q, ni);
        load_tile<kRows, D>(G, static_cast<const float*>(p.dO) + out * D, (long long)p.Hq * D, ni);
        float lse[4], delta[4], f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool on = 4 * ty + i < ni;
            lse[i] = on ? p.lse[out + (long long)(4 * ty + i) * p.Hq] * kLog2e : 0.f;
            delta[i] = on ? p.delta[out + (long long)(4 * ty + i) * p.Hq] : 0.f;
            f[i] = p.scale;
        }
        float4 acc[4][D / 64];
        clear<D>(acc);
        const int first = p.window ? max(0, i0 - p.window + 1) / kCols : 0;
        for (int t = first; t * kCols < i0 + ni; ++t) {
            const int j0 = t * kCols, nj = min(kCols, at.len - j0);
            __syncthreads();
            load_tile<kCols, D>(K, static_cast<const float*>(p.k) + (at.row0 + j0) * p.ld_k + (long long)hk * D, p.ld_k, nj);
            load_tile<kCols, D>(V, static_cast<const float*>(p.v) + (at.row0 + j0) * p.ld_v + (long long)hk * D, p.ld_v, nj);
            __syncthreads();
            float s[4][2], dp[4][2];
            dot_rows<2, D>(s, Q, K, ty, tx);
            dot_rows<2, D>(dp, G, V, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool on = sees(p, i0 + 4 * ty + i, j0 + tx + 16 * j);
                    W[(4 * ty + i) * (kCols + 4) + tx + 16 * j] = on ? exp2f(fmaf(s[i][j], c2, -lse[i])) * (dp[i][j] - delta[i]) : 0.f;
                }
            __syncthreads();
            add_rows<kCols, D>(acc, W, K, ty, tx);
        }
        store_rows<D>(static_cast<float*>(p.dq) + (at.row0 + i0) * p.ld_dq + (long long)h * D, p.ld_dq, ni, acc, f, ty, tx);
        __syncthreads();
    }
}

template <int D> __global__ void __launch_bounds__(kThreads, 2) prompt_dkv_kernel(const PromptParams p) {
    extern __shared__ __align__(16) float sm[];
    float *K = sm, *V = K + kRows * kPitch<D>, *Q = V + kRows * kPitch<D>, *G = Q + kCols * kPitch<D>, *W = G + kCols * kPitch<D>;
    // a block for each key head, or for each query head where that would be too few: then dk and dv of the query heads
    // go to the workspace, to be summed after
    const bool split = p.heads != nullptr;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, hk = split ? blockIdx.y / p.G : blockIdx.y;
    const int h0 = split ? blockIdx.y : hk * p.G, h1 = split ? h0 + 1 : h0 + p.G;
    const float c2 = p.scale * kLog2e;
    for (long long item = blockIdx.x;; item += gridDim.x) {
        const Place at = place_of(p, item, true);
        if (!at.any) return;
        const int j0 = at.tile * kRows, nj = min(kRows, at.len - j0);
        load_tile<kRows, D>(K, static_cast<const float*>(p.k) + (at.row0 + j0) * p.ld_k + (long long)hk * D, p.ld_k, nj);
        load_tile<kRows, D>(V, static_cast<const float*>(p.v) + (at.row0 + j0) * p.ld_v + (long long)hk * D, p.ld_v, nj);
        float4 dk[4][D / 64], dv[4][D / 64];
        clear<D>(dk);
        clear<D>(dv);
        const int end = p.window ? (int)min((long long)at.len, (long long)j0 + nj - 1 + p.window) : at.len;
        for (int h = h0; h < h1; ++h)
            for (int i0 = j0; i0 < end; i0 += kCols) {
                const int ni = min(kCols, at.len - i0);
                const long long row = ((long long)(at.row0 + i0) * p.Hq + h);
                __syncthreads();
                load_tile<kCols, D>(Q, static_cast<const float*>(p.q) + (at.row0 + i0) * p.ld_q + (long long)h * D, p.ld_q, ni);
                load_tile<kCols, D>(G, static_cast<const float*>(p.dO) + row * D, (long long)p.Hq * D, ni);
                float lse[2], delta[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool on = tx + 16 * j < ni;
                    lse[j] = on ? p.lse[row + (long long)(tx + 16 * j) * p.Hq] * kLog2e : 0.f;
                    delta[j] = on ? p.delta[row + (long long)(tx + 16 * j) * p.Hq] : 0.f;
                }
                __syncthreads();
                float s[4][2], dp[4][2];
                dot_rows<2, D>(s, K, Q, ty, tx);
                dot_rows<2, D>(dp, V, G, ty, tx);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int q = tx + 16 * j;
                        const bool on = q < ni && sees(p, i0 + q, j0 + 4 * ty + i);
                        s[i][j] = on ? exp2f(fmaf(s[i][j], c2, -lse[j])) : 0.f;
                        dp[i][j] = on ? s[i][j] * (dp[i][j] - delta[j]) : 0.f;
                        W[(4 * ty + i) * (kCols + 4) + q] = s[i][j];
                    }
                __syncthreads();
                add_rows<kCols, D>(dv, W, G, ty, tx);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) W[(4 * ty + i) * (kCols + 4) + tx + 16 * j] = dp[i][j];
                __syncthreads();
                add_rows<kCols, D>(dk, W, Q, ty, tx);
            }
        const float one[4] = {1.f, 1.f, 1.f, 1.f}, f[4] = {p.scale, p.scale, p.scale, p.scale};
        if (split) {
            float* to = p.heads + ((at.row0 + j0) * (long long)p.Hq + h0) * D;
            store_rows<D>(to, (long long)p.Hq * D, nj, dk, f, ty, tx);
            store_rows<D>(to + p.rows * p.Hq * D, (long long)p.Hq * D, nj, dv, one, ty, tx);
            __syncthreads();
            continue;
        }
        store_rows<D>(static_cast<float*>(p.dk) + (at.row0 + j0) * p.ld_dk + (long long)hk * D, p.ld_dk, nj, dk, f, ty, tx);
        store_rows<D>(static_cast<float*>(p.dv) + (at.row0 + j0) * p.ld_dv + (long long)hk * D, p.ld_dv, nj, dv, one, ty, tx);
        __syncthreads();
    }
}

// dk and dv of a key head: the sums over its query heads, in order, for the rows of the sequences.
template <int D> __global__ void __launch_bounds__(kThreads) prompt_heads_kernel(const PromptParams p) {
    for (long long item = blockIdx.x;; item += gridDim.x) {
        const Place at = place_of(p, item, false);
        if (!at.any) return;
        const int j0 = at.tile * kRows, nj = min(kRows, at.len - j0), hk = blockIdx.y;
        for (int i = threadIdx.x; i < nj * (D / 4); i += kThreads) {
            const long long row = at.row0 + j0 + i / (D / 4);
            const int c = i % (D / 4) * 4;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const float* from = p.heads + which * p.rows * p.Hq * D + (row * p.Hq + hk * p.G) * D + c;
                float4 sum = load4(from);
                for (int h = 1; h < p.G; ++h) {
                    const float4 x = load4(from + h * D);
                    sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
                }
                store4(which ? static_cast<float*>(p.dv) + row * p.ld_dv + (long long)hk * D + c
                             : static_cast<float*>(p.dk) + row * p.ld_dk + (long long)hk * D + c, sum);
            }
        }
        __syncthreads();
    }
}

template <int D> constexpr int fwd_smem() { return (2 * kRows * kPitch<D> + kRows * (kRows + 4)) * 4; }
template <int D> constexpr int bwd_smem() { return (2 * (kRows + kCols) * kPitch<D> + kRows * (kCols + 4)) * 4; }

template <typename K>
cudaError_t run(const char* name, K kernel, dim3 grid, int smem, std::atomic<unsigned long long>& ready, const PromptParams& p,
                cudaStream_t st) {
    if (cudaError_t e = set_smem_once(kernel, smem, ready); e != cudaSuccess) return e;
    TraceScope ts(name, st);
    kernel<<<grid, kThreads, smem, st>>>(p);
    return cudaGetLastError();
}
unsigned tiles(const PromptParams& p) {
    const long long n = most_tiles(p.s, kRows);
    return (unsigned)(n < (1 << 30) ? n : 1 << 30);
}

template <int D> cudaError_t fwd(const PromptParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready{0};
    return run("prompt_fwd", prompt_fwd_kernel<D>, dim3(tiles(p), p.Hq), fwd_smem<D>(), ready, p, st);
}
template <int D, typename IO> cudaError_t delta(const PromptParams& p, cudaStream_t st) {
    TraceScope ts("prompt_delta", st);
    const long long n = (p.rows * p.Hq + kThreads / 8 - 1) / (kThreads / 8);
    prompt_delta_kernel<D, IO><<<(unsigned)(n < 16384 ? n : 16384), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <int D> cudaError_t bwd(const PromptParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> ready[2] = {};
    if (cudaError_t e = delta<D, float>(p, st); e != cudaSuccess) return e;
    if (cudaError_t e = run("prompt_dq", prompt_dq_kernel<D>, dim3(tiles(p), p.Hq), bwd_smem<D>(), ready[0], p, st); e != cudaSuccess)
        return e;
    if (cudaError_t e = run("prompt_dkv", prompt_dkv_kernel<D>, dim3(tiles(p), p.heads ? p.Hq : p.H), bwd_smem<D>(), ready[1], p, st);
        e != cudaSuccess || !p.heads)
        return e;
    TraceScope ts("prompt_heads", st);
    prompt_heads_kernel<D><<<dim3(tiles(p), p.H), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Two blocks share an SM, 304 run at once: with fewer than twice as many, shared key heads are taken apart.
size_t prompt_attn_heads_bytes(long long rows, int N, int Hq, int H, int d) {
    const long long blocks = (rows / kRows + N) * H;
    return Hq > H && blocks < 608 ? (size_t)(2 * rows) * Hq * d * sizeof(float) : 0;
}
cudaError_t prompt_attn_fwd_simt(const PromptParams& p, cudaStream_t st) { return p.d == 128 ? fwd<128>(p, st) : fwd<64>(p, st); }
cudaError_t prompt_attn_delta_bf16(const PromptParams& p, cudaStream_t st) {
    return p.d == 128 ? delta<128, __nv_bfloat16>(p, st) : delta<64, __nv_bfloat16>(p, st);
}
cudaError_t prompt_attn_bwd_simt(const PromptParams& p, cudaStream_t st) { return p.d == 128 ? bwd<128>(p, st) : bwd<64>(p, st); }

}  // namespace dr
