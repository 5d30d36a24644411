// kv_cache.cu -- the paged 8-bit cache of keys and values: append with one scale for each page
// and head, and read back (dr.h, dr_cache_write / dr_cache_read).
//
// A block of the write owns one page of one head, of keys or of values: it takes the largest
// magnitude of the new values, joins it with the scale of what the page already holds, rounds
// the new values to codes and, where the scale grew, the earlier codes again.  No other block
// touches that page and head, so nothing is exchanged between blocks.
#include <cuda_fp8.h>

#include "kv_cache.cuh"
#include "trace.cuh"

namespace dr {
namespace {

constexpr int kWriteThreads = 128;
constexpr int kReadThreads = 256;

template <bool E4M3> __device__ __forceinline__ float inv_code_max() {
    return E4M3 ? 1.f / 448.f : 1.f / 127.f;
}
// The nearest code of x, ties to even.
template <bool E4M3> __device__ __forceinline__ uint32_t to_code(float x) {
    if (E4M3) return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)(int)fminf(fmaxf(rintf(x), -127.f), 127.f) & 0xffu;
}
template <bool E4M3> __device__ __forceinline__ float from_code(uint32_t byte) {
    if (E4M3) {
        __nv_fp8_e4m3 v;
        v.__x = (__nv_fp8_storage_t)byte;
        return float(v);
    }
    return (float)(int8_t)byte;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
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

// Block x: sequence and its i-th touched page; y: head; z: keys or values.
template <typename IN, bool E4M3>
__global__ void __launch_bounds__(kWriteThreads)
    cache_write_kernel(const CacheParams c, const IN* __restrict__ k, long long ld_k,
                       const IN* __restrict__ v, long long ld_v, int pages_per_seq) {
    __shared__ uint32_t red[kWriteThreads / 32];
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
    const int id = cache_page(c, b, index);
    if (id < 0) {
        if (threadIdx.x == 0) flag_index_error(c);
        return;
    }
    const int vecs = c.d / 8;  // 8-value pieces of a row
    const size_t ph = (size_t)id * c.H + h;
    uint8_t* codes = (keys ? c.k : c.v) + ph * c.page * c.d;
    float* scale = (keys ? c.k_scale : c.v_scale) + ph;
    const long long ld = keys ? ld_k : ld_v;
    // row r of the page is token first + r - len
    const IN* src = (keys ? k : v) + ((long long)b * c.T + (first - len)) * ld + (long long)h * c.d;

    // largest magnitude, as bits: what is not finite is at least 0x7f800000
    uint32_t top = 0;
    for (int j = lo * vecs + threadIdx.x; j < hi * vecs; j += kWriteThreads) {
        float x[8];
        load8(src + (long long)(j / vecs) * ld + (j % vecs) * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    const float s_old = lo > 0 ? *scale : 0.f;
    __syncthreads();  // every thread has read the scale too
#pragma unroll
    for (int w = 0; w < kWriteThreads / 32; ++w) top = max(top, red[w]);
    const bool finite = top < 0x7f800000u && s_old < __uint_as_float(0x7f800000u);
    const float s = finite ? fmaxf(s_old, __uint_as_float(top) * inv_code_max<E4M3>())
                           : __uint_as_float(0x7fc00000u);
    if (threadIdx.x == 0) *scale = s;

    for (int j = lo * vecs + threadIdx.x; j < hi * vecs; j += kWriteThreads) {
        float x[8];
        load8(src + (long long)(j / vecs) * ld + (j % vecs) * 8, x);
        uint32_t w[2] = {0, 0};
        if (s > 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 2] |= to_code<E4M3>(x[e] / s) << (8 * (e & 3));
        }
        *reinterpret_cast<uint2*>(codes + (size_t)j * 8) = make_uint2(w[0], w[1]);
    }
    if (s > s_old && s_old > 0.f) {  // false for NaN
        for (int j = threadIdx.x; j < lo * vecs; j += kWriteThreads) {
            const uint2 u = *reinterpret_cast<const uint2*>(codes + (size_t)j * 8);
            const uint32_t in[2] = {u.x, u.y};
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float was = from_code<E4M3>((in[e >> 2] >> (8 * (e & 3))) & 0xffu);
                w[e >> 2] |= to_code<E4M3>(__fmul_rn(was, s_old) / s) << (8 * (e & 3));
            }
            *reinterpret_cast<uint2*>(codes + (size_t)j * 8) = make_uint2(w[0], w[1]);
        }
    }
}

// A thread reads 8 values of one token and head, of keys (y = 0) or values (y = 1).
template <typename OUT, bool E4M3>
__global__ void __launch_bounds__(kReadThreads)
    cache_read_kernel(const CacheParams c, OUT* __restrict__ k, OUT* __restrict__ v) {
    const bool keys = blockIdx.y == 0;
    OUT* out = keys ? k : v;
    if (!out) return;
    const int vecs = c.d / 8;
    const long long total = (long long)c.B * c.T * c.H * vecs;
    for (long long j = (long long)blockIdx.x * kReadThreads + threadIdx.x; j < total;
         j += (long long)gridDim.x * kReadThreads) {
        const int piece = (int)(j % vecs);
        const long long row = j / vecs;
        const int h = (int)(row % c.H);
        const long long tok = row / c.H;
        const int b = (int)(tok / c.T), t = (int)(tok % c.T);
        int len, n;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.f;
        const bool in = cache_seq(c, b, len, n);
        int id = -1;
        if (in && t < n) id = cache_page(c, b, (len + t) / c.page);
        if (id >= 0) {
            const size_t ph = (size_t)id * c.H + h;
            const float s = (keys ? c.k_scale : c.v_scale)[ph];
            const uint2 u = *reinterpret_cast<const uint2*>(
                (keys ? c.k : c.v) + (ph * c.page + (len + t) % c.page) * c.d + piece * 8);
            const uint32_t w[2] = {u.x, u.y};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = from_code<E4M3>((w[e >> 2] >> (8 * (e & 3))) & 0xffu) * s;
        } else if (!in || t < n) {
            flag_index_error(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(0x7fc00000u);
        }
        store8(out + j * 8, y);
    }
}

template <typename IN>
cudaError_t write_as(const CacheParams& c, const void* k, long long ld_k, const void* v,
                     long long ld_v, cudaStream_t st) {
    const int pages = 1 + (c.page - 2 + c.T) / c.page;  // pages that T tokens can touch
    const dim3 grid((unsigned)c.B * pages, c.H, 2);
    TraceScope ts("cache_write", st);
    if (c.code == DR_CODE_E4M3)
        cache_write_kernel<IN, true><<<grid, kWriteThreads, 0, st>>>(
            c, static_cast<const IN*>(k), ld_k, static_cast<const IN*>(v), ld_v, pages);
    else
        cache_write_kernel<IN, false><<<grid, kWriteThreads, 0, st>>>(
            c, static_cast<const IN*>(k), ld_k, static_cast<const IN*>(v), ld_v, pages);
    return cudaGetLastError();
}

template <typename OUT>
cudaError_t read_as(const CacheParams& c, void* k, void* v, cudaStream_t st) {
    const long long total = (long long)c.B * c.T * c.H * (c.d / 8);
    const long long blocks = (total + kReadThreads - 1) / kReadThreads;
    const dim3 grid((unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 2);
    TraceScope ts("cache_read", st);
    if (c.code == DR_CODE_E4M3)
        cache_read_kernel<OUT, true><<<grid, kReadThreads, 0, st>>>(c, static_cast<OUT*>(k),
                                                                    static_cast<OUT*>(v));
    else
        cache_read_kernel<OUT, false><<<grid, kReadThreads, 0, st>>>(c, static_cast<OUT*>(k),
                                                                     static_cast<OUT*>(v));
    return cudaGetLastError();
}

}  // namespace

cudaError_t cache_write(const CacheParams& c, const void* k, long long ld_k, const void* v,
                        long long ld_v, int io, cudaStream_t st) {
    if (c.B == 0 || c.T == 0) return cudaSuccess;
    return io == DR_BF16 ? write_as<__nv_bfloat16>(c, k, ld_k, v, ld_v, st)
                         : write_as<float>(c, k, ld_k, v, ld_v, st);
}

cudaError_t cache_read(const CacheParams& c, void* k, void* v, int out, cudaStream_t st) {
    if (c.B == 0 || c.T == 0 || (!k && !v)) return cudaSuccess;
    return out == DR_BF16 ? read_as<__nv_bfloat16>(c, k, v, st) : read_as<float>(c, k, v, st);
}

}  // namespace dr
