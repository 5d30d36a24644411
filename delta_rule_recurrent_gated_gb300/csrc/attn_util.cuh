// attn_util.cuh -- what both attention kernels over the 8-bit cache share: the division of their
// work, the 16-bit operands made from codes and queries, and the rows that leave a block.
#pragma once
#include <cuda_fp16.h>

#include "cache_attn.cuh"
#include "chain.cuh"

namespace dr {
namespace {

constexpr float kNegInf = -INFINITY;
constexpr int kBias = 14;  // weights as 16-bit operands reach 2^14
// A weight w = p vs 2^(m - M + bias) is formed as p f with one factor f for a page as long as f is at most 2^100: then
// a p below 2^-126, which ex2 gives as zero, has w below the smallest 16-bit operand.  Where the factor is larger or its
// power of two past fp32 (value scales that are all tiny, or scores far below one whose value scale is small or zero),
// w is taken as one power of two, 2^(s - M + bias + log2 vs).
constexpr float kMaxFactor = 100.f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// ------------------------------------------------------------------ shares of the work
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
// Block i of n <= total takes places share(i) .. share(i + 1) - 1 of the line, at least one;
// holder(at) is the block that has place `at`: total i / n <= at where total i < (at + 1) n.
__device__ __forceinline__ long long share(long long total, int i, int n) { return total * i / n; }
__device__ __forceinline__ int holder(long long total, long long at, int n) {
    return (int)(((at + 1) * n - 1) / total);
}
__device__ __forceinline__ int blocks_used(long long total, int blocks) {
    return total < blocks ? (int)total : blocks;
}

// ------------------------------------------------------------------ operands
// The four codes of `w` as two pairs of 16-bit floats: bytes (0, 2) and (1, 3) of int8 codes,
// bytes (0, 1) and (2, 3) of e4m3 codes.
template <bool E4M3>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& a, uint32_t& b) {
    if (E4M3) {
        asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n"
            " cvt.rn.f16x2.e4m3x2 %0, x;\n cvt.rn.f16x2.e4m3x2 %1, y;\n}\n"
            : "=r"(a), "=r"(b)
            : "r"(w));
    } else {
        // x + 128 in the low bits of 1024 .. 2047, whose spacing is 1; minus 1152 is x exactly
        const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
        uint32_t u = (w & 0x00ff00ffu) ^ 0x64806480u, v = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
        const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&u), off);
        const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&v), off);
        a = *reinterpret_cast<const uint32_t*>(&x);
        b = *reinterpret_cast<const uint32_t*>(&y);
    }
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^x for a whole x, the ends of the range standing for what is beyond them; 0 for -inf and NaN.
__device__ __forceinline__ float pow2i(float x) {
    if (!(x >= -126.f)) return 0.f;
    return __uint_as_float((uint32_t)((int)fminf(x, 127.f) + 127) << 23);
}

// A query row is scaled by up * rest = 2^-e to a largest magnitude of 2^9 .. 2^10, which keeps a bf16
// value exact in 16 bits unless it is below 2^-24 of the row's largest.
__device__ __forceinline__ void query_scale(float top, int& e, float& up, float& rest) {
    e = 0;
    if (top > 0.f && top < INFINITY) frexpf(top, &e), e -= 10;
    const int e1 = max(-100, min(100, e));  // two powers in the range of fp32
    up = pow2i(-(float)e1);
    rest = pow2i((float)(e1 - e));
}
// Whole number with vs < 2^ve.
__device__ __forceinline__ float scale_exponent(float vs) {
    int e;
    frexpf(vs, &e);
    return vs > 0.f ? (float)e : vs == 0.f ? kNegInf : 0.f;
}

// What a warp needs to know of 16 positions.
struct __align__(16) Meta {
    int id;            // page, -1 where the entry is out of range, -2 where no row sees a position
    float ks, vs, ve;  // scales; whole number with vs <= 2^ve
};

// ------------------------------------------------------------------ rows that leave a block
// Part of the workspace of block i: two unfinished tiles, each [rows][d] sums, then [rows] of l, m, M.
__host__ __device__ constexpr size_t tile_floats(int d, int rows) { return (size_t)rows * (d + 3); }

__device__ __forceinline__ void write_row(const AttnParams& p, int b, int h, int row, int ch, int d, float sum,
                                          float l, float m, float M) {
    const int tok = row / p.G, head = h * p.G + row % p.G;
    const size_t at = ((size_t)b * p.c.T + tok) * p.Hq + head;
    // sums are in units of 2^(M - 14), l in units of 2^m
    float f = M - m - kBias;
    float y = sum / l;
    if (f > 100.f || f < -100.f) { y = ldexpf(y, (int)fminf(fmaxf(f, -400.f), 400.f)); }
    else y *= pow2i(f);
    // every value scale is zero; without weights (every score is -inf: a row sees at least its own position) 0 / 0
    if (M == kNegInf && sum == 0.f && l > 0.f) y = 0.f;
    st_any(p.o, at * d + ch, p.out, y);
    if (ch == 0 && p.lse) p.lse[at] = (m + log2f(l)) * kLn2;
}

template <typename K>
int resident_blocks(K kernel, int threads, int smem) {
    int sms = 0, per = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess) return 0;
    return sms * per;
}

}  // namespace
}  // namespace dr
