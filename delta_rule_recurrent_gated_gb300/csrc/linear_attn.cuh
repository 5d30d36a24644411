// linear_attn.cuh -- launch parameters of linear attention with a decay for each head.
//
// One scan serves the forward pass and, with the tensors in other places, all three gradients:
//   out_t = alpha X_t^T q_t,  X_t = e^g X_{t-1} + beta k_t v_t^T   (forward: X_{-1} is the state before)
//   o : (q, k, v) = (q, k, v),   state S    (h0 to hT)         scale on what is read
//   dq: (dO, v, k),              state S^T  (h0)                scale on what is read
//   dk: (v, dO, q), reverse,     state R^T  (dhT)               scale on what is written
//   dv: (k, q, dO), reverse,     state R    (dhT to dh0)        scale on what is written
// Reverse: tokens from the last to the first; the state before the first of them, dhT, reaches that token
// undecayed (hT is the state after it), so every decay of the state has one step less and dh0 one more.
#pragma once
#include <cstddef>

#include "seqs.cuh"

namespace dr {
struct ScanParams {
    Seqs s;
    long long rows;
    int H, dk, dv;               // dk: channels of q and k; dv: of v and out
    long long ld_q, ld_k, ld_v, ld_o;
    const void *q, *k, *v;
    void* out;
    const float* g;              // [H] log-decay of a step
    const float* x0;             // [N, H, dk, dv], transposed: [N, H, dv, dk]; null: zero
    float* xT;                   // [N, H, dk, dv]; null: not wanted
    bool x0_transposed, reverse;
    int32_t* status;
    float scale;                 // of what is read (forward) or written (reverse)
    int span;                    // chunks of a segment; 0: sequences are not split
    long long slots;             // segments that the workspace has room for
    float* part;                 // their states, [slots, H, dk, dv]
};

// Long sequences are split where a block for each sequence and head would leave most of the GPU idle: first every
// segment's own state is formed from nothing, then the states that they begin with are the running sums of
// these, and then all segments are scanned at once.  The first step reads k and v once more.
constexpr int kScanChunk = 128, kMostScans = 3;
// Chunks of a segment (0: not split) for `scans` scans that run together, and how many segments of split sequences
// there can be.
int scan_span(int io, long long rows, int N, int T, bool packed, int H, int dk, int dv, int scans);
long long scan_slots(long long rows, int span);

// n scans (of the same sequences and heads) together.
cudaError_t linear_scans(const ScanParams* p, int n, int io, cudaStream_t st);
// Their kernels on the tensor cores, bf16 with dk and dv 64 or 128, rows > 0 (linear_attn_tc.cu); `only`: the
// segments' own states.
cudaError_t linear_scans_tc(const ScanParams* p, int n, bool only, cudaStream_t st);
// The recurrent step: T tokens of every sequence on the caller's state.
struct StepParams {
    int B, T, H, dk, dv;
    float scale;
    const void *q, *k, *v;
    const float* g;
    float* state;
    void* o;
    long long ld_q, ld_k, ld_v;
};
cudaError_t linear_step(const StepParams& p, int io, cudaStream_t st);
}  // namespace dr
