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

size_t cache_attn_part_bytes(int d);
cudaError_t cache_attn(const AttnParams& p, cudaStream_t st);
}  // namespace dr
