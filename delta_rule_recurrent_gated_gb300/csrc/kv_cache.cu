// kv_cache.cu -- the paged 8-bit cache of keys and values: append with one scale for each page
// and head, and read back (dr.h, dr_cache_write / dr_cache_read).
//
// A block of the write owns one page of one head, of keys or of values: it takes the largest
// magnitude of the new values, joins it with the scale of what the page already holds, rounds
// the new values to codes and, where the scale grew, the earlier codes again.  No other block
// touches that page and head, so nothing is exchanged between blocks.  The read's blocks are the same.
//
// 8 prompts of 2048 to 4096 tokens, four heads of 128, bf16 to e4m3 and back: append (75 MB) 19 us and read back
// (92 MB) 19 us, 4.5 TB/s for the pair.  A block is a chain of length, values, maximum and codes of about
// 4 us, an SM holds five (append) or eight (read) of them, and a scheduler issues in 55 to 65 % of the cycles.
#include <type_traits>

#include <cuda_fp8.h>

#include "chain.cuh"
#include "f32x2.cuh"
#include "kv_cache.cuh"
#include "trace.cuh"

namespace dr {
namespace {

template <bool E4M3> __device__ __forceinline__ float inv_code_max() {
    return E4M3 ? 1.f / 448.f : 1.f / 127.f;
}
// The nearest codes of four values of magnitude below 128 (448), ties to even, the first in the lowest byte.
template <bool E4M3> __device__ __forceinline__ uint32_t to_codes(float2 a, float2 b) {
    if (E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
    // 1.5 * 2^23 + x has spacing 1: rounded to nearest even, its low byte is the whole number
    const float2 big = make_float2(12582912.f, 12582912.f);
    a = add2(a, big);
    b = add2(b, big);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
template <bool E4M3> __device__ __forceinline__ float from_code(uint32_t byte) {
    if (E4M3) {
        __nv_fp8_e4m3 v;
        v.__x = (__nv_fp8_storage_t)byte;
        return float(v);
    }
    return (float)(int8_t)byte;
}

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

// Codes of x / s for many x and one s.  The quotient is correctly rounded: with y the correctly
// rounded 1 / s and q within a unit of the quotient, q + (x - q s) y is the rounded quotient
// (P. Markstein, IBM J. Res. Dev. 34, 1990); a first such step brings x y to within a unit.  A
// remainder that underflows belongs to a quotient below 2^-20, whose code is zero whatever its last
// bits are; a zero keeps the sign of x.  Scales outside 1e-18 .. 1e18 take the division itself, and
// the bound on the magnitude that a scale among the smallest numbers does not keep.
template <bool E4M3> struct Coder {
    float s, y;
    __device__ __forceinline__ explicit Coder(float d) : s(d), y(1.f / d) {}
    __device__ __forceinline__ bool plain() const { return !(s > 1e-18f && s < 1e18f); }
    __device__ __forceinline__ float2 fast(float2 x) const {
        const float2 y2 = make_float2(y, y), s2 = make_float2(-s, -s);
        float2 q = mul2(x, y2);
        q = fma2(fma2(q, s2, x), y2, q);
        q = fma2(fma2(q, s2, x), y2, q);
        if (E4M3) {
            q.x = __uint_as_float((__float_as_uint(q.x) & 0x7fffffffu) | (__float_as_uint(x.x) & 0x80000000u));
            q.y = __uint_as_float((__float_as_uint(q.y) & 0x7fffffffu) | (__float_as_uint(x.y) & 0x80000000u));
        }
        return q;
    }
    __device__ __forceinline__ float slow(float x) const {
        constexpr float top = E4M3 ? 448.f : 127.f;
        return fminf(fmaxf(x / s, -top), top);
    }
    __device__ __forceinline__ uint2 operator()(const float (&x)[8]) const {
        float2 q[4];
        if (plain()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = make_float2(slow(x[2 * j]), slow(x[2 * j + 1]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = fast(make_float2(x[2 * j], x[2 * j + 1]));
        }
        return make_uint2(to_codes<E4M3>(q[0], q[1]), to_codes<E4M3>(q[2], q[3]));
    }
};

template <typename T> struct Vec8;  // 8 values as loaded
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    // the larger of `top` and the magnitudes, as bits of fp32 (which order as the magnitudes do)
    __device__ __forceinline__ uint32_t magnitude(uint32_t top) const {
        const uint32_t a = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu);
        const uint32_t b = __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu), c = __vmaxu2(a, b);
        return max(top, max(c & 0xffff0000u, c << 16));
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ uint32_t magnitude(uint32_t top) const {
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
        return top;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

// Block x: sequence and its i-th touched page; y: head; z: keys or values.  A page is 128 to 2048
// pieces of 8 values, NV of them a thread.  The new values are read once, into registers: 8 prompts of up to 4096 tokens (4 heads of 128, bf16) take 75 MB of traffic.
// Blocks of a page's threads on an SM: as many as hold the new values and 32 registers more.
constexpr int write_blocks(int threads, int value_regs) {
    const int n = 65536 / (threads * (32 + value_regs));
    return n < 2048 / threads ? n : 2048 / threads;
}
template <typename IN, bool E4M3, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS, write_blocks(THREADS, NV * (int)sizeof(IN) * 2))
    cache_write_kernel(const CacheParams c, const IN* __restrict__ k, long long ld_k,
                       const IN* __restrict__ v, long long ld_v, int pages_per_seq) {
    __shared__ uint32_t red[THREADS / 32];
    chain_wait();
    chain_release();
    const int b = blockIdx.x / pages_per_seq, i = blockIdx.x % pages_per_seq, h = blockIdx.y;
    const bool keys = blockIdx.z == 0;
    int len, n;
    if (!cache_seq(c, b, len, n)) {
        if (threadIdx.x == 0) flag_index_error(c);
        return;
    }
    const int index = len / c.page + i;              // page of the sequence
    const long long first = (long long)index * c.page;  // its first position
    const int lo = i == 0 ? len - (int)first : 0;    // rows lo .. hi - 1 of the page are new
    const int hi = (int)min((long long)c.page, (long long)len + n - first);
    if (lo >= hi) return;
    const int shift = c.d == 128 ? 4 : 3;  // pieces of a row: 16 or 8
    const int from = lo << shift, to = hi << shift;
    const long long ld = keys ? ld_k : ld_v;
    // row r of the page is token first + r - len
    const IN* src = (keys ? k : v) + ((long long)b * c.T + (first - len)) * ld + (long long)h * c.d;
    Vec8<IN> x[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const int j = e * THREADS + threadIdx.x;
        if (j >= from && j < to) x[e].load(src + (j >> shift) * ld + (j & ((1 << shift) - 1)) * 8);
    }
    const int id = cache_page(c, b, index);
    if (id < 0) {
        if (threadIdx.x == 0) flag_index_error(c);
        return;
    }
    const size_t ph = (size_t)id * c.H + h;
    uint8_t* codes = (keys ? c.k : c.v) + ph * c.page * c.d;
    float* scale = (keys ? c.k_scale : c.v_scale) + ph;
    const float s_old = lo > 0 ? *scale : 0.f;

    // largest magnitude, as bits: what is not finite is at least 0x7f800000
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const int j = e * THREADS + threadIdx.x;
        if (j >= from && j < to) top = x[e].magnitude(top);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();  // every thread has read the scale too
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) top = max(top, red[w]);
    const bool finite = top < 0x7f800000u && s_old < __uint_as_float(0x7f800000u);
    const float s = finite ? fmaxf(s_old, __uint_as_float(top) * inv_code_max<E4M3>())
                           : __uint_as_float(0x7fc00000u);
    if (threadIdx.x == 0) *scale = s;

    const Coder<E4M3> code(s);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const int j = e * THREADS + threadIdx.x;
        if (j >= from && j < to) {
            float y[8];
            x[e].get(y);
            *reinterpret_cast<uint2*>(codes + (size_t)j * 8) = s > 0.f ? code(y) : make_uint2(0, 0);
        }
    }
    if (s > s_old && s_old > 0.f) {  // false for NaN
        for (int j = threadIdx.x; j < from; j += THREADS) {
            const uint2 u = *reinterpret_cast<const uint2*>(codes + (size_t)j * 8);
            const uint32_t in[2] = {u.x, u.y};
            float y[8];
#pragma unroll
            for (int m = 0; m < 8; ++m)
                y[m] = __fmul_rn(from_code<E4M3>((in[m >> 2] >> (8 * (m & 3))) & 0xffu), s_old);
            *reinterpret_cast<uint2*>(codes + (size_t)j * 8) = code(y);
        }
    }
}

// Block x: sequence and its i-th page of the call's positions; y: head; z: keys or values.
template <typename OUT, bool E4M3, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS)
    cache_read_kernel(const CacheParams c, OUT* __restrict__ k, OUT* __restrict__ v, int pages_per_seq) {
    chain_wait();
    chain_release();
    const int b = blockIdx.x / pages_per_seq, i = blockIdx.x % pages_per_seq, h = blockIdx.y;
    const bool keys = blockIdx.z == 0;
    OUT* out = keys ? k : v;
    if (!out) return;
    int len, n;
    const bool in = cache_seq(c, b, len, n);
    if (!in) {
        if (threadIdx.x == 0) flag_index_error(c);
        len = n = 0;
    }
    const int index = len / c.page + i;
    const int t0 = i * c.page - len % c.page;  // token of the page's first row
    if (t0 >= c.T) return;
    const int lo = max(0, -t0), hi = min(c.page, c.T - t0), full = min(hi, n - t0);  // rows; with a value
    const int shift = c.d == 128 ? 4 : 3;
    int id = -1;
    if (full > lo) {
        id = cache_page(c, b, index);
        if (id < 0 && threadIdx.x == 0) flag_index_error(c);
    }
    float s = __uint_as_float(0x7fc00000u);
    const uint8_t* codes = c.k;
    if (id >= 0) {
        const size_t ph = (size_t)id * c.H + h;
        s = (keys ? c.k_scale : c.v_scale)[ph];
        codes = (keys ? c.k : c.v) + ph * c.page * c.d;
    }
    uint2 u[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const int j = e * THREADS + threadIdx.x;
        u[e] = make_uint2(0, 0);
        if (id >= 0 && j >= lo << shift && j < full << shift)
            u[e] = *reinterpret_cast<const uint2*>(codes + (size_t)j * 8);
    }
    OUT* dst = out + (((long long)b * c.T + t0) * c.H + h) * c.d;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const int j = e * THREADS + threadIdx.x, row = j >> shift;
        if (row >= lo && row < hi) {
            const bool zero = in && row >= full;
            const uint32_t w[2] = {u[e].x, u[e].y};
            float y[8];
#pragma unroll
            for (int m = 0; m < 8; ++m)
                y[m] = zero ? 0.f : from_code<E4M3>((w[m >> 2] >> (8 * (m & 3))) & 0xffu) * s;
            store8(dst + (long long)row * c.H * c.d + (j & ((1 << shift) - 1)) * 8, y);
        }
    }
}

int pages_of(const CacheParams& c) { return 1 + (c.page - 2 + c.T) / c.page; }  // that T tokens can touch

template <typename IN, bool E4M3, int THREADS, int NV>
cudaError_t write_page(const CacheParams& c, const void* k, long long ld_k, const void* v, long long ld_v,
                       cudaStream_t st) {
    const int pages = pages_of(c);
    TraceScope ts("cache_write", st);
    return launch_chained(cache_write_kernel<IN, E4M3, THREADS, NV>, dim3((unsigned)c.B * pages, c.H, 2), THREADS, 0, st,
                          c, static_cast<const IN*>(k), ld_k, static_cast<const IN*>(v), ld_v, pages);
}
template <typename OUT, bool E4M3, int THREADS, int NV>
cudaError_t read_page(const CacheParams& c, void* k, void* v, cudaStream_t st) {
    const int pages = pages_of(c);
    TraceScope ts("cache_read", st);
    return launch_chained(cache_read_kernel<OUT, E4M3, THREADS, NV>, dim3((unsigned)c.B * pages, c.H, 2), THREADS, 0, st,
                          c, static_cast<OUT*>(k), static_cast<OUT*>(v), pages);
}

// f(threads, pieces of each) for the page's size, as compile-time values
template <typename F> cudaError_t by_page(const CacheParams& c, F f) {
    using std::integral_constant;
    switch (c.page * c.d / 8) {
        case 128: return f(integral_constant<int, 128>(), integral_constant<int, 1>());
        case 256: return f(integral_constant<int, 128>(), integral_constant<int, 2>());
        case 512: return f(integral_constant<int, 128>(), integral_constant<int, 4>());
        case 1024: return f(integral_constant<int, 256>(), integral_constant<int, 4>());
        default: return f(integral_constant<int, 256>(), integral_constant<int, 8>());
    }
}

template <typename IN, bool E4M3>
cudaError_t write_as(const CacheParams& c, const void* k, long long ld_k, const void* v, long long ld_v,
                     cudaStream_t st) {
    return by_page(c, [&](auto threads, auto nv) {
        return write_page<IN, E4M3, decltype(threads)::value, decltype(nv)::value>(c, k, ld_k, v, ld_v, st);
    });
}
template <typename OUT, bool E4M3>
cudaError_t read_as(const CacheParams& c, void* k, void* v, cudaStream_t st) {
    return by_page(c, [&](auto threads, auto nv) {
        return read_page<OUT, E4M3, decltype(threads)::value, decltype(nv)::value>(c, k, v, st);
    });
}

}  // namespace

cudaError_t cache_write(const CacheParams& c, const void* k, long long ld_k, const void* v,
                        long long ld_v, int io, cudaStream_t st) {
    if (c.B == 0 || c.T == 0) return cudaSuccess;
    const bool e4m3 = c.code == DR_CODE_E4M3;
    if (io == DR_BF16)
        return e4m3 ? write_as<__nv_bfloat16, true>(c, k, ld_k, v, ld_v, st)
                    : write_as<__nv_bfloat16, false>(c, k, ld_k, v, ld_v, st);
    return e4m3 ? write_as<float, true>(c, k, ld_k, v, ld_v, st)
                : write_as<float, false>(c, k, ld_k, v, ld_v, st);
}

cudaError_t cache_read(const CacheParams& c, void* k, void* v, int out, cudaStream_t st) {
    if (c.B == 0 || c.T == 0 || (!k && !v)) return cudaSuccess;
    const bool e4m3 = c.code == DR_CODE_E4M3;
    if (out == DR_BF16)
        return e4m3 ? read_as<__nv_bfloat16, true>(c, k, v, st) : read_as<__nv_bfloat16, false>(c, k, v, st);
    return e4m3 ? read_as<float, true>(c, k, v, st) : read_as<float, false>(c, k, v, st);
}

}  // namespace dr
