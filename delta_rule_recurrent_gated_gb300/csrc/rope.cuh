// rope.cuh -- launch parameters of the norm-and-rotation kernels (norm_rope.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace dr {
struct RopeParams {
    long long tokens;           // B * T
    int T, Hq, Hk, d, rot, style, table_rows;
    float eps;
    long long ld_q, ld_k, ld_oq, ld_ok;
    const void *q, *k, *dyq, *dyk;
    const float *wq, *wk, *cos_t, *sin_t;
    const int32_t *positions, *start;
    void *oq, *ok;              // yq, yk (forward) or dq, dk (backward)
    float *dwq, *dwk;
    float* part;                // backward: the blocks' parts of dwq, dwk
    // set by the launcher: heads of a run, runs of q and of k; backward: blocks of a run, of the last run
    // of q and of k, of all runs of q and of k
    int hp, nq, nk, nb, nbq, nbk, bq, bk;
};

size_t norm_rope_part_bytes(RopeParams p);
cudaError_t norm_rope(RopeParams p, bool bwd, int io, int out, cudaStream_t st);
}  // namespace dr
