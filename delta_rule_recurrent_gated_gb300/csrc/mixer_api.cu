// mixer_api.cu -- the C ABI of causal attention over whole prompts and of linear attention with a decay for
// each head (declared in dr.h): argument validation and dispatch to prompt_attn*.cu and linear_attn*.cu.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "common.cuh"
#include "linear_attn.cuh"
#include "prompt_attn.cuh"

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool any_misaligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (misaligned(p)) return true;
    return false;
}
int cuda_status(cudaError_t e) { return e == cudaSuccess ? DR_OK : DR_ERR_CUDA; }
// A distance between rows of `row` values: no overlap, whole 16-byte pieces.
int check_row(long long ld, long long row, int type) {
    if (ld < row || ld >= (1ll << 40)) return DR_ERR_INVALID_ARG;
    return ld * (type == DR_BF16 ? 2 : 4) % 16 ? DR_ERR_ALIGNMENT : DR_OK;
}
// Packed sequences of a call.  To find a tile a warp walks over their offsets, 32 in 0.3 to 1 us, while its block waits: for
// 2^20 of them 33 ms, of the 2 s that a wait may take.  (The walk's 32-bit counters end at 2^31 - 32.)
constexpr int kMostPacked = 1 << 20;
int check_seqs(int B, int T, int num_seqs) {
    if (B < 0 || T < 0 || num_seqs < 0) return DR_ERR_INVALID_ARG;
    if ((long long)B * T >= (1ll << 30)) return DR_ERR_UNSUPPORTED;
    if (num_seqs > kMostPacked && num_seqs != B) return DR_ERR_UNSUPPORTED;
    return DR_OK;
}
// num_seqs has to be that of the layout that the call uses.
int check_layout(int B, int num_seqs, const int32_t* cu) {
    if (cu ? B != 1 : num_seqs != B) return DR_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(cu) & 3 ? DR_ERR_ALIGNMENT : DR_OK;
}
int check_status_word(const int32_t* status) { return reinterpret_cast<uintptr_t>(status) & 3 ? DR_ERR_ALIGNMENT : DR_OK; }

int check_prompt(const dr_prompt_desc* d, bool bwd) {
    if (!d) return DR_ERR_INVALID_ARG;
    if (int rc = check_seqs(d->B, d->T, d->num_seqs); rc != DR_OK) return rc;
    if (d->Hq < 1 || d->H < 1 || d->Hq % d->H || d->d < 1 || d->window < 0 || !std::isfinite(d->scale)) return DR_ERR_INVALID_ARG;
    if (d->io_dtype != DR_BF16 && d->io_dtype != DR_F32) return DR_ERR_INVALID_ARG;
    if (d->d != 64 && d->d != 128) return DR_ERR_UNSUPPORTED;
    if (d->Hq > 65535) return DR_ERR_UNSUPPORTED;  // a grid dimension
    const long long q = (long long)d->Hq * d->d, k = (long long)d->H * d->d;
    const long long lds[][2] = {{d->ld_q, q}, {d->ld_k, k}, {d->ld_v, k}, {d->ld_dq, q}, {d->ld_dk, k}, {d->ld_dv, k}};
    for (int i = 0; i < (bwd ? 6 : 3); ++i)
        if (int rc = check_row(lds[i][0], lds[i][1], d->io_dtype); rc != DR_OK) return rc;
    return check_status_word(d->status);
}
dr::PromptParams prompt_params(const dr_prompt_desc* d, const void* q, const void* k, const void* v, const int32_t* cu) {
    dr::PromptParams p = {};
    p.s = {cu, d->num_seqs, d->T};
    p.rows = (long long)d->B * d->T;
    p.Hq = d->Hq; p.H = d->H; p.G = d->Hq / d->H; p.d = d->d;
    p.window = d->window < d->T ? d->window : 0;  // one that shows everything is none
    p.scale = d->scale;
    p.ld_q = d->ld_q; p.ld_k = d->ld_k; p.ld_v = d->ld_v;
    p.ld_dq = d->ld_dq; p.ld_dk = d->ld_dk; p.ld_dv = d->ld_dv;
    p.q = q; p.k = k; p.v = v;
    p.status = d->status;
    return p;
}

size_t delta_bytes(const dr_prompt_desc* d) { return ((size_t)d->B * d->T * d->Hq * sizeof(float) + 15) / 16 * 16; }
size_t heads_bytes(const dr_prompt_desc* d) {
    return d->io_dtype == DR_F32 ? dr::prompt_attn_heads_bytes((long long)d->B * d->T, d->num_seqs, d->Hq, d->H, d->d) : 0;
}

bool linear_size(int d, int io, bool step) { return d == 64 || d == 128 || ((io == DR_F32 || step) && (d == 16 || d == 32)); }
int check_linear(const dr_linear_desc* d, bool bwd, bool step) {
    if (!d) return DR_ERR_INVALID_ARG;
    if (int rc = check_seqs(d->B, d->T, d->num_seqs); rc != DR_OK) return rc;
    if (d->H < 1 || d->d_k < 1 || d->d_v < 1 || !std::isfinite(d->scale)) return DR_ERR_INVALID_ARG;
    if (d->io_dtype != DR_BF16 && d->io_dtype != DR_F32) return DR_ERR_INVALID_ARG;
    if (!linear_size(d->d_k, d->io_dtype, step) || !linear_size(d->d_v, d->io_dtype, step)) return DR_ERR_UNSUPPORTED;
    if (d->H > 65535 || (long long)d->num_seqs * d->H >= (1ll << 30)) return DR_ERR_UNSUPPORTED;  // grid dimensions
    const long long q = (long long)d->H * d->d_k, v = (long long)d->H * d->d_v;
    const long long lds[][2] = {{d->ld_q, q}, {d->ld_k, q}, {d->ld_v, v}, {d->ld_dq, q}, {d->ld_dk, q}, {d->ld_dv, v}};
    for (int i = 0; i < (bwd ? 6 : 3); ++i)
        if (int rc = check_row(lds[i][0], lds[i][1], d->io_dtype); rc != DR_OK) return rc;
    return check_status_word(d->status);
}
int span_of(const dr_linear_desc* d, bool packed, int scans) {
    return dr::scan_span(d->io_dtype, (long long)d->B * d->T, d->num_seqs, d->T, packed, d->H, d->d_k, d->d_v, scans);
}
dr::ScanParams scan_params(const dr_linear_desc* d, const float* g, const int32_t* cu, void* ws, int scans) {
    dr::ScanParams p = {};
    p.s = {cu, d->num_seqs, d->T};
    p.rows = (long long)d->B * d->T;
    p.H = d->H; p.dk = d->d_k; p.dv = d->d_v;
    p.g = g; p.scale = d->scale; p.status = d->status;
    p.part = static_cast<float*>(ws);
    p.span = span_of(d, cu != nullptr, scans);
    p.slots = dr::scan_slots(p.rows, p.span);
    return p;
}
// Room for the segments' states, whether the sequences come dense or packed, of one scan or of three together.
size_t linear_bytes(const dr_linear_desc* d) {
    const long long rows = (long long)d->B * d->T;
    long long slots = 0;
    for (int scans : {1, 3})
        for (bool packed : {false, true})
            if (packed ? d->B == 1 : d->num_seqs == d->B)
                slots = std::max(slots, scans * dr::scan_slots(rows, span_of(d, packed, scans)));
    return std::max<size_t>(16, (size_t)slots * d->H * d->d_k * d->d_v * sizeof(float));
}

}  // namespace

extern "C" {

int dr_prompt_attn_fwd(const dr_prompt_desc* desc, const void* q, const void* k, const void* v,
                       const int32_t* cu_seqlens, void* o, float* lse, void* stream) {
    int rc = check_prompt(desc, false);
    if (rc != DR_OK) return rc;
    if ((rc = check_layout(desc->B, desc->num_seqs, cu_seqlens)) != DR_OK) return rc;
    dr::PromptParams p = prompt_params(desc, q, k, v, cu_seqlens);
    if (p.rows == 0 || p.s.N == 0) return DR_OK;
    if (!q || !k || !v || !o) return DR_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, o, lse})) return DR_ERR_ALIGNMENT;
    p.o = o; p.lse = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(desc->io_dtype == DR_BF16 ? dr::prompt_attn_fwd_tc(p, st) : dr::prompt_attn_fwd_simt(p, st));
}

size_t dr_prompt_attn_workspace_bytes(const dr_prompt_desc* desc) {
    if (check_prompt(desc, true) != DR_OK) return 0;
    const size_t n = delta_bytes(desc) + heads_bytes(desc);
    return n < 16 ? 16 : n;
}

int dr_prompt_attn_bwd(const dr_prompt_desc* desc, const void* q, const void* k, const void* v,
                       const void* o, const float* lse, const void* dO, const int32_t* cu_seqlens,
                       void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                       void* stream) {
    int rc = check_prompt(desc, true);
    if (rc != DR_OK) return rc;
    if ((rc = check_layout(desc->B, desc->num_seqs, cu_seqlens)) != DR_OK) return rc;
    dr::PromptParams p = prompt_params(desc, q, k, v, cu_seqlens);
    if (p.rows == 0 || p.s.N == 0) return DR_OK;
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return DR_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, o, lse, dO, dq, dk, dv, workspace})) return DR_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < dr_prompt_attn_workspace_bytes(desc)) return DR_ERR_WORKSPACE;
    p.o = const_cast<void*>(o); p.lse = const_cast<float*>(lse); p.dO = dO;
    p.dq = dq; p.dk = dk; p.dv = dv; p.delta = static_cast<float*>(workspace);
    if (heads_bytes(desc)) p.heads = p.delta + delta_bytes(desc) / sizeof(float);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(desc->io_dtype == DR_BF16 ? dr::prompt_attn_bwd_tc(p, st) : dr::prompt_attn_bwd_simt(p, st));
}

size_t dr_linear_attn_workspace_bytes(const dr_linear_desc* desc) {
    return check_linear(desc, false, false) == DR_OK ? linear_bytes(desc) : 0;  // of a forward call alone too
}

int dr_linear_attn_fwd(const dr_linear_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, const float* h0, const int32_t* cu_seqlens, void* o, float* hT,
                       void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_linear(desc, false, false);
    if (rc != DR_OK) return rc;
    if ((rc = check_layout(desc->B, desc->num_seqs, cu_seqlens)) != DR_OK) return rc;
    dr::ScanParams p = scan_params(desc, g, cu_seqlens, workspace, 1);
    if (p.s.N == 0) return DR_OK;
    if (!g || (p.rows > 0 && (!q || !k || !v || !o))) return DR_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, h0, o, hT, workspace})) return DR_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < linear_bytes(desc)) return DR_ERR_WORKSPACE;
    p.q = q; p.k = k; p.v = v; p.out = o;
    p.ld_q = desc->ld_q; p.ld_k = desc->ld_k; p.ld_v = desc->ld_v; p.ld_o = (long long)desc->H * desc->d_v;
    p.x0 = h0; p.xT = hT;
    return cuda_status(dr::linear_scans(&p, 1, desc->io_dtype, static_cast<cudaStream_t>(stream)));
}

int dr_linear_attn_bwd(const dr_linear_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, const float* h0, const void* dO, const float* dhT,
                       const int32_t* cu_seqlens, void* dq, void* dk, void* dv, float* dh0,
                       void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_linear(desc, true, false);
    if (rc != DR_OK) return rc;
    if ((rc = check_layout(desc->B, desc->num_seqs, cu_seqlens)) != DR_OK) return rc;
    const dr::ScanParams base = scan_params(desc, g, cu_seqlens, workspace, 3);
    if (base.s.N == 0) return DR_OK;
    if (!g || (base.rows > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv))) return DR_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, h0, dO, dhT, dq, dk, dv, dh0, workspace})) return DR_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < linear_bytes(desc)) return DR_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long ld_g = (long long)desc->H * desc->d_v, part = base.slots * desc->H * desc->d_k * desc->d_v;
    dr::ScanParams x[3] = {base, base, base};
    x[0].dk = x[1].dk = desc->d_v;  // dq: (dO, v, k), the state transposed
    x[0].dv = x[1].dv = desc->d_k;
    x[0].q = dO; x[0].k = v; x[0].v = k; x[0].out = dq;
    x[0].ld_q = ld_g; x[0].ld_k = desc->ld_v; x[0].ld_v = desc->ld_k; x[0].ld_o = desc->ld_dq;
    x[0].x0 = h0;
    x[1].reverse = x[2].reverse = true;  // dk: (v, dO, q) from the last token to the first, likewise
    x[1].q = v; x[1].k = dO; x[1].v = q; x[1].out = dk;
    x[1].ld_q = desc->ld_v; x[1].ld_k = ld_g; x[1].ld_v = desc->ld_q; x[1].ld_o = desc->ld_dk;
    x[1].x0 = x[2].x0 = dhT;
    x[0].x0_transposed = x[1].x0_transposed = true;
    x[2].q = k; x[2].k = q; x[2].v = dO; x[2].out = dv;  // dv: (k, q, dO)
    x[2].ld_q = desc->ld_k; x[2].ld_k = desc->ld_q; x[2].ld_v = ld_g; x[2].ld_o = desc->ld_dv;
    x[2].xT = dh0;
    x[1].part += part;
    x[2].part += 2 * part;
    if (base.rows == 0) return cuda_status(dr::linear_scans(x + 2, 1, desc->io_dtype, st));
    return cuda_status(dr::linear_scans(x, 3, desc->io_dtype, st));
}

int dr_linear_attn_step(const dr_linear_desc* desc, const void* q, const void* k, const void* v,
                        const float* g, float* state, void* o, void* stream) {
    int rc = check_linear(desc, false, true);
    if (rc != DR_OK) return rc;
    if (desc->num_seqs != desc->B) return DR_ERR_INVALID_ARG;
    if (desc->B == 0 || desc->T == 0) return DR_OK;
    if (!q || !k || !v || !g || !state || !o) return DR_ERR_INVALID_ARG;
    if (any_misaligned({q, k, v, g, state, o})) return DR_ERR_ALIGNMENT;
    dr::StepParams p = {};
    p.B = desc->B; p.T = desc->T; p.H = desc->H; p.dk = desc->d_k; p.dv = desc->d_v;
    p.scale = desc->scale;
    p.q = q; p.k = k; p.v = v; p.g = g; p.state = state; p.o = o;
    p.ld_q = desc->ld_q; p.ld_k = desc->ld_k; p.ld_v = desc->ld_v;
    return cuda_status(dr::linear_step(p, desc->io_dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
