// kv_cache.cuh -- launch parameters of the paged 8-bit cache (kv_cache.cu, cache_attn.cu) and
// the checks that keep a kernel inside it.
#pragma once
#include "common.cuh"

namespace dr {
constexpr int kMaxPositions = 0x7fff0000;  // positions, rounded up to a page, stay in 32 bits

struct CacheParams {
    int num_pages, H, d, page, code;
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int32_t* status;
    int B, T, table_stride;
    const int32_t *table, *lens, *counts;
};

__device__ __forceinline__ void flag_index_error(const CacheParams& c) {
    if (c.status) *reinterpret_cast<volatile int32_t*>(c.status) = kErrIndex;
}

// The call's tokens of sequence b: `len` positions before them, n of them.  False (nothing of
// the sequence may be touched) where a length or count is outside its range.
__device__ __forceinline__ bool cache_seq(const CacheParams& c, int b, int& len, int& n) {
    len = c.lens[b];
    n = c.counts ? c.counts[b] : c.T;
    return len >= 0 && n >= 0 && n <= c.T && (long long)len + n <= (long long)c.table_stride * c.page &&
           (long long)len + n <= kMaxPositions;
}
// The page that holds position p of sequence b, or -1.
__device__ __forceinline__ int cache_page(const CacheParams& c, int b, int index) {
    const int id = c.table[(size_t)b * c.table_stride + index];
    return id >= 0 && id < c.num_pages ? id : -1;
}

cudaError_t cache_write(const CacheParams& c, const void* k, long long ld_k, const void* v,
                        long long ld_v, int io, cudaStream_t st);
cudaError_t cache_read(const CacheParams& c, void* k, void* v, int out, cudaStream_t st);
}  // namespace dr
