// attn_api.cu -- the C ABI of the softmax-attention layer (declared in dr.h): argument
// validation and dispatch to norm_rope.cu, kv_cache.cu and cache_attn.cu.
#include <cmath>
#include <cstdint>

#include "cache_attn.cuh"
#include "rope.cuh"

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? DR_OK : DR_ERR_CUDA; }
bool known_type(int t) { return t == DR_BF16 || t == DR_F32; }
long long value_bytes(int t) { return t == DR_BF16 ? 2 : 4; }
// A distance between rows of `row` values: no overlap, whole 16-byte pieces.
int check_row(long long ld, long long row, int type) {
    if (ld < row || ld >= (1ll << 40)) return DR_ERR_INVALID_ARG;
    return ld * value_bytes(type) % 16 ? DR_ERR_ALIGNMENT : DR_OK;
}

int check_rope(const dr_rope_desc* d, bool bwd) {
    if (!d) return DR_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->Hq < 0 || d->Hk < 0 || d->Hq + (long long)d->Hk < 1 || d->d < 1)
        return DR_ERR_INVALID_ARG;
    if (d->rot < 0 || d->rot > d->d || d->table_rows < 0) return DR_ERR_INVALID_ARG;
    if (d->style != DR_ROPE_HALVES && d->style != DR_ROPE_PAIRS) return DR_ERR_INVALID_ARG;
    if (!known_type(d->io_dtype) || !known_type(d->out_dtype) || !known_type(d->grad_dtype))
        return DR_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return DR_ERR_INVALID_ARG;
    if (d->d % 8 || d->d > 256 || d->rot % 16) return DR_ERR_UNSUPPORTED;
    if (d->Hq > 8192 || d->Hk > 8192) return DR_ERR_UNSUPPORTED;  // runs of heads are a grid dimension
    const int out = bwd ? d->grad_dtype : d->out_dtype;
    int rc = DR_OK;
    if (d->Hq > 0) {
        rc = check_row(d->ld_q, (long long)d->Hq * d->d, d->io_dtype);
        if (rc == DR_OK) rc = check_row(d->ld_oq, (long long)d->Hq * d->d, out);
    }
    if (rc == DR_OK && d->Hk > 0) {
        rc = check_row(d->ld_k, (long long)d->Hk * d->d, d->io_dtype);
        if (rc == DR_OK) rc = check_row(d->ld_ok, (long long)d->Hk * d->d, out);
    }
    return rc;
}

dr::RopeParams rope_params(const dr_rope_desc* d) {
    dr::RopeParams p = {};
    p.tokens = (long long)d->B * d->T;
    p.T = d->T; p.Hq = d->Hq; p.Hk = d->Hk; p.d = d->d; p.rot = d->rot; p.style = d->style;
    p.table_rows = d->table_rows; p.eps = d->eps;
    p.ld_q = d->ld_q; p.ld_k = d->ld_k; p.ld_oq = d->ld_oq; p.ld_ok = d->ld_ok;
    return p;
}

int check_cache(const dr_cache* c) {
    if (!c || c->num_pages < 0 || c->H < 1 || c->d < 1 || c->page < 1) return DR_ERR_INVALID_ARG;
    if (c->code != DR_CODE_I8 && c->code != DR_CODE_E4M3) return DR_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return DR_ERR_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return DR_ERR_UNSUPPORTED;
    if (c->H > 65535) return DR_ERR_UNSUPPORTED;  // a grid dimension
    return DR_OK;
}
int check_call(const dr_cache* c, const dr_cache_seqs* s) {
    int rc = check_cache(c);
    if (rc != DR_OK) return rc;
    if (!s || s->B < 0 || s->T < 0 || s->table_stride < 0) return DR_ERR_INVALID_ARG;
    if (s->B == 0 || s->T == 0) return DR_OK;
    if (!s->lens || (s->table_stride > 0 && !s->page_table)) return DR_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return DR_ERR_INVALID_ARG;
    const void* ptrs[] = {c->k, c->v, c->k_scale, c->v_scale, s->page_table, s->lens, s->counts};
    for (const void* p : ptrs)
        if (misaligned(p)) return DR_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(c->status) & 3) return DR_ERR_ALIGNMENT;
    if ((long long)s->B * s->T >= (1ll << 30)) return DR_ERR_UNSUPPORTED;
    return DR_OK;
}
dr::CacheParams cache_params(const dr_cache* c, const dr_cache_seqs* s) {
    dr::CacheParams p = {};
    p.num_pages = c->num_pages; p.H = c->H; p.d = c->d; p.page = c->page; p.code = c->code;
    p.k = static_cast<uint8_t*>(c->k); p.v = static_cast<uint8_t*>(c->v);
    p.k_scale = c->k_scale; p.v_scale = c->v_scale; p.status = c->status;
    p.B = s->B; p.T = s->T; p.table_stride = s->table_stride;
    p.table = s->page_table; p.lens = s->lens; p.counts = s->counts;
    return p;
}

int check_attn(const dr_cache* c, const dr_attn_desc* d, int B, int T) {
    int rc = check_cache(c);
    if (rc != DR_OK) return rc;
    if (!d || B < 0 || T < 0 || d->Hq < 1 || d->Hq % c->H || d->window < 0 || !std::isfinite(d->scale))
        return DR_ERR_INVALID_ARG;
    if (!known_type(d->io_dtype) || !known_type(d->out_dtype)) return DR_ERR_INVALID_ARG;
    if ((long long)B * T * d->Hq >= (1ll << 30)) return DR_ERR_UNSUPPORTED;
    return check_row(d->ld_q, (long long)d->Hq * c->d, d->io_dtype);
}

// Which kernel, by the rows of a sequence and cache head (query tokens times the query heads that share
// it): the kernel for few rows reads the cache once for each 16 of them (8 where a type is fp32), and from 33
// on a tile of 256 on the tensor cores is the faster even partly filled.  us, and in brackets on the tensor
// cores, four cache heads; four sequences of 8000 positions, heads of 128: 16 rows 24.1 (34.8), 32 rows 34.8
// (34.8), 36 rows 42.8 (35.0), 256 rows 129 (39.6); heads of 64: 32 rows 23.1 (29.6), 36 rows 29.4 (29.9), 64
// rows 35.3 (30.0), 256 rows 89.2 (32.8).  64 sequences of 4000, heads of 128: 16 rows 82.6 (131), 32 rows 150
// (132), 36 rows 205 (133); heads of 64: 16 rows 57.2 (129), 32 rows 102 (129), 36 rows 139 (129).  fp32 types
// need the split operands of the other kernel.
constexpr int kTcRows = 33;
bool on_tensor_cores(const dr_cache* c, const dr_attn_desc* d, int T) {
    return d->io_dtype == DR_BF16 && d->out_dtype == DR_BF16 && (long long)T * (d->Hq / c->H) >= kTcRows;
}
size_t attn_bytes(const dr_cache* c, const dr_attn_desc* d, int T) {
    return on_tensor_cores(c, d, T) ? dr::cache_attn_tc_bytes(c->d) : dr::cache_attn_rows_bytes(c->d);
}

}  // namespace

extern "C" {

int dr_norm_rope_fwd(const dr_rope_desc* desc, const void* q, const void* k, const float* wq,
                     const float* wk, const float* cos_table, const float* sin_table,
                     const int32_t* positions, const int32_t* start, void* yq, void* yk,
                     void* stream) {
    int rc = check_rope(desc, false);
    if (rc != DR_OK) return rc;
    dr::RopeParams p = rope_params(desc);
    if (p.tokens == 0) return DR_OK;
    if (desc->Hq > 0 && (!q || !yq)) return DR_ERR_INVALID_ARG;
    if (desc->Hk > 0 && (!k || !yk)) return DR_ERR_INVALID_ARG;
    if (desc->rot > 0 && desc->table_rows > 0 && (!cos_table || !sin_table)) return DR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, wq, wk, cos_table, sin_table, positions, start, yq, yk};
    for (const void* ptr : ptrs)
        if (misaligned(ptr)) return DR_ERR_ALIGNMENT;
    p.q = q; p.k = k; p.wq = wq; p.wk = wk; p.cos_t = cos_table; p.sin_t = sin_table;
    p.positions = positions; p.start = start; p.oq = yq; p.ok = yk;
    return cuda_status(dr::norm_rope(p, false, desc->io_dtype, desc->out_dtype,
                                     static_cast<cudaStream_t>(stream)));
}

size_t dr_norm_rope_workspace_bytes(const dr_rope_desc* desc) {
    if (check_rope(desc, true) != DR_OK) return 0;
    const size_t n = dr::norm_rope_part_bytes(rope_params(desc));
    return n ? n : 16;
}

int dr_norm_rope_bwd(const dr_rope_desc* desc, const void* q, const void* k, const float* wq,
                     const float* wk, const float* cos_table, const float* sin_table,
                     const int32_t* positions, const int32_t* start, const void* dyq,
                     const void* dyk, void* dq, void* dk, float* dwq, float* dwk,
                     void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_rope(desc, true);
    if (rc != DR_OK) return rc;
    dr::RopeParams p = rope_params(desc);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((dwq && !wq) || (dwk && !wk)) return DR_ERR_INVALID_ARG;
    if (p.tokens > 0) {
        if (desc->Hq > 0 && (!q || !dyq || !dq)) return DR_ERR_INVALID_ARG;
        if (desc->Hk > 0 && (!k || !dyk || !dk)) return DR_ERR_INVALID_ARG;
        if (desc->rot > 0 && desc->table_rows > 0 && (!cos_table || !sin_table)) return DR_ERR_INVALID_ARG;
    }
    const void* ptrs[] = {q, k, wq, wk, cos_table, sin_table, positions, start, dyq, dyk, dq, dk,
                          dwq, dwk, workspace};
    for (const void* ptr : ptrs)
        if (misaligned(ptr)) return DR_ERR_ALIGNMENT;
    if (p.tokens == 0) {  // an empty sum
        const size_t bytes = (size_t)desc->d * sizeof(float);
        if (dwq && cudaMemsetAsync(dwq, 0, bytes, st) != cudaSuccess) return DR_ERR_CUDA;
        if (dwk && cudaMemsetAsync(dwk, 0, bytes, st) != cudaSuccess) return DR_ERR_CUDA;
        return DR_OK;
    }
    if (!workspace || workspace_bytes < dr_norm_rope_workspace_bytes(desc)) return DR_ERR_WORKSPACE;
    p.q = q; p.k = k; p.wq = wq; p.wk = wk; p.cos_t = cos_table; p.sin_t = sin_table;
    p.positions = positions; p.start = start; p.dyq = dyq; p.dyk = dyk; p.oq = dq; p.ok = dk;
    p.dwq = dwq; p.dwk = dwk; p.part = static_cast<float*>(workspace);
    return cuda_status(dr::norm_rope(p, true, desc->io_dtype, desc->grad_dtype, st));
}

int dr_cache_write(const dr_cache* cache, const dr_cache_seqs* seqs, const void* k, long long ld_k,
                   const void* v, long long ld_v, int io_dtype, void* stream) {
    int rc = check_call(cache, seqs);
    if (rc != DR_OK) return rc;
    if (!known_type(io_dtype)) return DR_ERR_INVALID_ARG;
    for (long long ld : {ld_k, ld_v})
        if ((rc = check_row(ld, (long long)cache->H * cache->d, io_dtype)) != DR_OK) return rc;
    if (seqs->B == 0 || seqs->T == 0) return DR_OK;
    if (!k || !v) return DR_ERR_INVALID_ARG;
    if (misaligned(k) || misaligned(v)) return DR_ERR_ALIGNMENT;
    return cuda_status(dr::cache_write(cache_params(cache, seqs), k, ld_k, v, ld_v, io_dtype,
                                       static_cast<cudaStream_t>(stream)));
}

int dr_cache_read(const dr_cache* cache, const dr_cache_seqs* seqs, void* k, void* v, int out_dtype,
                  void* stream) {
    int rc = check_call(cache, seqs);
    if (rc != DR_OK) return rc;
    if (!known_type(out_dtype)) return DR_ERR_INVALID_ARG;
    if (misaligned(k) || misaligned(v)) return DR_ERR_ALIGNMENT;
    return cuda_status(dr::cache_read(cache_params(cache, seqs), k, v, out_dtype,
                                      static_cast<cudaStream_t>(stream)));
}

size_t dr_cache_attn_workspace_bytes(const dr_cache* cache, const dr_attn_desc* desc, int B, int T) {
    if (check_attn(cache, desc, B, T) != DR_OK) return 0;
    return attn_bytes(cache, desc, T);
}

int dr_cache_attn(const dr_cache* cache, const dr_cache_seqs* seqs, const dr_attn_desc* desc,
                  const void* q, void* o, float* lse, void* workspace, size_t workspace_bytes,
                  void* stream) {
    int rc = check_call(cache, seqs);
    if (rc != DR_OK) return rc;
    if ((rc = check_attn(cache, desc, seqs->B, seqs->T)) != DR_OK) return rc;
    if (seqs->B == 0 || seqs->T == 0) return DR_OK;
    if (!q || !o) return DR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, o, lse, workspace};
    for (const void* ptr : ptrs)
        if (misaligned(ptr)) return DR_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < attn_bytes(cache, desc, seqs->T)) return DR_ERR_WORKSPACE;
    dr::AttnParams p = {};
    p.c = cache_params(cache, seqs);
    p.Hq = desc->Hq;
    p.G = desc->Hq / cache->H;
    p.window = desc->window;
    p.scale = desc->scale;
    p.ld_q = desc->ld_q;
    p.q = q; p.o = o; p.lse = lse;
    p.io = desc->io_dtype; p.out = desc->out_dtype;
    p.part = static_cast<float*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(on_tensor_cores(cache, desc, seqs->T) ? dr::cache_attn_tc(p, st)
                                                             : dr::cache_attn_rows(p, st));
}

}  // extern "C"
