// cache_attn.cuh -- launch parameters of the attention over the paged 8-bit cache.
#pragma once
#include "kv_cache.cuh"

namespace dr {
struct AttnParams {
    CacheParams c;
    int Hq, G;               // query heads; of each cache head
    int window;
    float scale;
    long long ld_q;
    const void* q;
    void* o;
    float* lse;
    int io, out;
    float* part;             // workspace: the blocks' unfinished rows
};

// A few rows of a sequence and cache head at a time, any type (cache_attn.cu).
size_t cache_attn_rows_bytes(int d);
cudaError_t cache_attn_rows(const AttnParams& p, cudaStream_t st);
// 256 rows at a time on the tensor cores, bf16 queries and outputs (cache_attn_tc.cu).
size_t cache_attn_tc_bytes(int d);
cudaError_t cache_attn_tc(const AttnParams& p, cudaStream_t st);
}  // namespace dr
