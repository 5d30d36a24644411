// prompt_attn.cuh -- launch parameters of causal attention over whole prompts.
#pragma once
#include <cstddef>

#include "seqs.cuh"

namespace dr {
struct PromptParams {
    Seqs s;
    long long rows;          // of every tensor
    int Hq, H, G, d;         // query heads, key heads, query heads of each key head, channels
    int window;
    float scale;
    long long ld_q, ld_k, ld_v, ld_dq, ld_dk, ld_dv;
    const void *q, *k, *v, *dO;
    void* o;                 // forward: written; backward: read
    float* lse;              // the same (forward: may be null)
    void *dq, *dk, *dv;
    int32_t* status;
    float* delta;            // workspace: sum of dO o for each row and query head
    float* heads;            // workspace: dk, then dv, of each query head [rows, Hq, d]; null: not taken apart
};

// CUDA cores, fp32 (prompt_attn.cu).
cudaError_t prompt_attn_fwd_simt(const PromptParams& p, cudaStream_t st);
cudaError_t prompt_attn_bwd_simt(const PromptParams& p, cudaStream_t st);
size_t prompt_attn_heads_bytes(long long rows, int N, int Hq, int H, int d);  // p.heads (0: null)
// p.delta for bf16, the first step of the gradient.
cudaError_t prompt_attn_delta_bf16(const PromptParams& p, cudaStream_t st);
// Tensor cores, bf16 (prompt_attn_tc.cu, prompt_attn_tc_bwd.cu).
cudaError_t prompt_attn_fwd_tc(const PromptParams& p, cudaStream_t st);
cudaError_t prompt_attn_bwd_tc(const PromptParams& p, cudaStream_t st);
}  // namespace dr
