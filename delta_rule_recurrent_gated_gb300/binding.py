"""ctypes binding of libdr.so (include/dr.h).  Argument marshalling only: every
step of the forward and backward runs in the library's CUDA kernels; PyTorch
only allocates device memory and supplies the stream.

There is no fallback: if libdr.so is missing or a call fails, this module
raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdr.so")

DR_OK, DR_ERR_INVALID_ARG, DR_ERR_UNSUPPORTED, DR_ERR_WORKSPACE, DR_ERR_ALIGNMENT, \
    DR_ERR_CUDA, DR_ERR_TIMEOUT, DR_ERR_SCRATCH_LIMIT, DR_ERR_INDEX = range(9)
DR_DELTANET, DR_GDN, DR_KDA, DR_GDN2 = 0, 1, 2, 3
DR_BF16, DR_F32 = 0, 1
DR_FLAG_REUSE_FWD = 1
DR_FLAG_PREPARE_INPUTS = 2
VARIANTS = {"deltanet": DR_DELTANET, "gdn": DR_GDN, "kda": DR_KDA, "gdn2": DR_GDN2}


class DrDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("d_k", ctypes.c_int), ("d_v", ctypes.c_int), ("chunk", ctypes.c_int),
        ("variant", ctypes.c_int), ("io_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int), ("scale", ctypes.c_float), ("flags", ctypes.c_int),
        ("num_seqs", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
        ("chunk_table", ctypes.c_void_p), ("chunk_offsets", ctypes.c_void_p),
        ("num_chunks", ctypes.c_int),
    ]


ROPE_STYLES = {"halves": 0, "pairs": 1}
CACHE_CODES = {"i8": 0, "e4m3": 1}


class DrRopeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "Hq", "Hk", "d", "rot", "style", "io_dtype",
                                            "out_dtype", "grad_dtype", "table_rows")]
    _fields_ += [("eps", ctypes.c_float)]
    _fields_ += [(n, ctypes.c_longlong) for n in ("ld_q", "ld_k", "ld_oq", "ld_ok")]


class DrCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("num_pages", "H", "d", "page", "code")]
    _fields_ += [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "status")]


class DrCacheSeqs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int), ("lens", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


class DrAttnDesc(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int), ("io_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("window", ctypes.c_int), ("scale", ctypes.c_float), ("ld_q", ctypes.c_longlong)]


class DrPromptDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "Hq", "H", "d", "num_seqs", "io_dtype", "window")]
    _fields_ += [("scale", ctypes.c_float)]
    _fields_ += [(n, ctypes.c_longlong) for n in ("ld_q", "ld_k", "ld_v", "ld_dq", "ld_dk", "ld_dv")]
    _fields_ += [("status", ctypes.c_void_p)]


class DrLinearDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "H", "d_k", "d_v", "num_seqs", "io_dtype")]
    _fields_ += [("scale", ctypes.c_float)]
    _fields_ += [(n, ctypes.c_longlong) for n in ("ld_q", "ld_k", "ld_v", "ld_dq", "ld_dk", "ld_dv")]
    _fields_ += [("status", ctypes.c_void_p)]


class DrError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)}")


_lib = None


def load(path: str = LIB_PATH):
    """Open libdr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libdr.so not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    D = ctypes.POINTER(DrDesc)
    lib.dr_workspace_bytes.argtypes = [D]
    lib.dr_workspace_bytes.restype = S
    lib.dr_plan_varlen.argtypes = [P, I, I, P, P, I, P]
    lib.dr_plan_varlen.restype = I
    lib.dr_fwd.argtypes = [D] + [P] * 8 + [P, S, P]
    lib.dr_fwd.restype = I
    lib.dr_bwd.argtypes = [D] + [P] * 14 + [P, S, P]
    lib.dr_bwd.restype = I
    lib.dr_fwd_u.argtypes = [D] + [P] * 9 + [P, S, P]
    lib.dr_fwd_u.restype = I
    lib.dr_bwd_u.argtypes = [D] + [P] * 15 + [P, S, P]
    lib.dr_bwd_u.restype = I
    lib.dr_check_status.argtypes = [P, P]
    lib.dr_check_status.restype = I
    lib.dr_error_string.argtypes = [I]
    lib.dr_error_string.restype = ctypes.c_char_p
    lib.dr_fwd_noalloc.argtypes = [D] + [P] * 8 + [P]
    lib.dr_fwd_noalloc.restype = I
    lib.dr_decode.argtypes = [D] + [P] * 7 + [P]
    lib.dr_decode.restype = I
    lib.dr_gdn2_decode.argtypes = [D] + [P] * 8 + [P]
    lib.dr_gdn2_decode.restype = I
    lib.dr_selftest_wait.argtypes = [P, I, ctypes.c_longlong, P]
    lib.dr_selftest_wait.restype = I
    lib.dr_gdn2_fwd.argtypes = [D] + [P] * 9 + [P, S, P]
    lib.dr_gdn2_fwd.restype = I
    lib.dr_gdn2_bwd.argtypes = [D] + [P] * 16 + [P, S, P]
    lib.dr_gdn2_bwd.restype = I
    R, C, Q, A = (ctypes.POINTER(x) for x in (DrRopeDesc, DrCache, DrCacheSeqs, DrAttnDesc))
    L = ctypes.c_longlong
    lib.dr_norm_rope_fwd.argtypes = [R] + [P] * 11
    lib.dr_norm_rope_fwd.restype = I
    lib.dr_norm_rope_workspace_bytes.argtypes = [R]
    lib.dr_norm_rope_workspace_bytes.restype = S
    lib.dr_norm_rope_bwd.argtypes = [R] + [P] * 15 + [S, P]
    lib.dr_norm_rope_bwd.restype = I
    lib.dr_cache_write.argtypes = [C, Q, P, L, P, L, I, P]
    lib.dr_cache_write.restype = I
    lib.dr_cache_read.argtypes = [C, Q, P, P, I, P]
    lib.dr_cache_read.restype = I
    lib.dr_cache_attn_workspace_bytes.argtypes = [C, A, I, I]
    lib.dr_cache_attn_workspace_bytes.restype = S
    lib.dr_cache_attn.argtypes = [C, Q, A] + [P] * 4 + [S, P]
    lib.dr_cache_attn.restype = I
    M, N = ctypes.POINTER(DrPromptDesc), ctypes.POINTER(DrLinearDesc)
    lib.dr_prompt_attn_fwd.argtypes = [M] + [P] * 7
    lib.dr_prompt_attn_fwd.restype = I
    lib.dr_prompt_attn_workspace_bytes.argtypes = [M]
    lib.dr_prompt_attn_workspace_bytes.restype = S
    lib.dr_prompt_attn_bwd.argtypes = [M] + [P] * 11 + [S, P]
    lib.dr_prompt_attn_bwd.restype = I
    lib.dr_linear_attn_workspace_bytes.argtypes = [N]
    lib.dr_linear_attn_workspace_bytes.restype = S
    lib.dr_linear_attn_fwd.argtypes = [N] + [P] * 9 + [S, P]
    lib.dr_linear_attn_fwd.restype = I
    lib.dr_linear_attn_bwd.argtypes = [N] + [P] * 13 + [S, P]
    lib.dr_linear_attn_bwd.restype = I
    lib.dr_linear_attn_step.argtypes = [N] + [P] * 7
    lib.dr_linear_attn_step.restype = I
    lib.dr_trace_enable.argtypes = [I]
    lib.dr_trace_enable.restype = I
    lib.dr_trace_count.argtypes = []
    lib.dr_trace_count.restype = I
    lib.dr_trace_reset.argtypes = []
    lib.dr_trace_reset.restype = None
    lib.dr_trace_get.argtypes = [I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float)]
    lib.dr_trace_get.restype = I
    _lib = lib
    return lib


def error_string(code: int) -> str:
    return load().dr_error_string(int(code)).decode()


def _check(code: int, where: str):
    if code != DR_OK:
        raise DrError(code, where)


# ------------------------------------------------------------------ raw C-ABI calls
def workspace_bytes(desc: DrDesc) -> int:
    return int(load().dr_workspace_bytes(ctypes.byref(desc)))


def plan_varlen(cu_seqlens_host, chunk: int):
    """(chunk_table [n,2] int32, chunk_offsets [N+1] int32, n) for host offsets."""
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    N = len(cu) - 1
    n = ctypes.c_int(0)
    lib = load()
    _check(lib.dr_plan_varlen(cu.ctypes.data, N, chunk, None, None, 0, ctypes.byref(n)),
           "dr_plan_varlen")
    table = np.zeros((max(n.value, 1), 2), dtype=np.int32)
    offs = np.zeros(N + 1, dtype=np.int32)
    _check(lib.dr_plan_varlen(cu.ctypes.data, N, chunk, table.ctypes.data, offs.ctypes.data,
                              n.value, ctypes.byref(n)), "dr_plan_varlen")
    return table[:n.value], offs, n.value


def dr_fwd(desc, q, k, v, beta, g, h0, o, hT, ws, ws_bytes, stream) -> int:
    return load().dr_fwd(ctypes.byref(desc), q, k, v, beta, g, h0, o, hT, ws, ws_bytes, stream)


def dr_fwd_u(desc, q, k, v, beta, g, h0, o, hT, u, ws, ws_bytes, stream) -> int:
    return load().dr_fwd_u(ctypes.byref(desc), q, k, v, beta, g, h0, o, hT, u, ws, ws_bytes,
                           stream)


def dr_bwd_u(desc, q, k, v, beta, g, h0, dO, dhT, dU, dq, dk, dv, dbeta, dg, dh0, ws, ws_bytes,
             stream) -> int:
    return load().dr_bwd_u(ctypes.byref(desc), q, k, v, beta, g, h0, dO, dhT, dU, dq, dk, dv,
                           dbeta, dg, dh0, ws, ws_bytes, stream)


def dr_bwd(desc, q, k, v, beta, g, h0, dO, dhT, dq, dk, dv, dbeta, dg, dh0, ws, ws_bytes,
           stream) -> int:
    return load().dr_bwd(ctypes.byref(desc), q, k, v, beta, g, h0, dO, dhT, dq, dk, dv, dbeta,
                         dg, dh0, ws, ws_bytes, stream)


def dr_decode(desc, q, k, v, beta, g, state, o, stream) -> int:
    return load().dr_decode(ctypes.byref(desc), q, k, v, beta, g, state, o, stream)


def dr_gdn2_fwd(desc, q, k, v, erase, write, g, h0, o, hT, ws, ws_bytes, stream) -> int:
    return load().dr_gdn2_fwd(ctypes.byref(desc), q, k, v, erase, write, g, h0, o, hT, ws,
                              ws_bytes, stream)


def dr_gdn2_bwd(desc, q, k, v, erase, write, g, h0, dO, dhT, dq, dk, dv, derase, dwrite, dg, dh0,
                ws, ws_bytes, stream) -> int:
    return load().dr_gdn2_bwd(ctypes.byref(desc), q, k, v, erase, write, g, h0, dO, dhT, dq, dk,
                              dv, derase, dwrite, dg, dh0, ws, ws_bytes, stream)


def selftest_wait(ws, arrive: bool, limit_ns: int, stream) -> int:
    return load().dr_selftest_wait(ws, 1 if arrive else 0, int(limit_ns), stream)


def check_status(ws, stream) -> int:
    return load().dr_check_status(ws, stream)


def trace_enable(max_launches: int) -> None:
    _check(load().dr_trace_enable(int(max_launches)), "dr_trace_enable")


def trace_read():
    """[(kernel name, milliseconds)] of the traced launches, in launch order."""
    lib = load()
    out = []
    for i in range(lib.dr_trace_count()):
        name = ctypes.c_char_p()
        ms = ctypes.c_float()
        _check(lib.dr_trace_get(i, ctypes.byref(name), ctypes.byref(ms)), "dr_trace_get")
        out.append((name.value.decode(), float(ms.value)))
    return out


# ------------------------------------------------------------------ torch-level helpers
def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dt(t) -> int:
    import torch
    return DR_BF16 if t.dtype == torch.bfloat16 else DR_F32


class Problem:
    """Descriptor + device-side chunk plan + workspace for one problem shape.

    Build once per shape; `forward` / `backward` then enqueue the library calls
    on the current torch stream.  With ``prepare`` the calls take raw q, k, beta
    logits and gate arguments (DR_FLAG_PREPARE_INPUTS) and the gradients are with
    respect to those.
    """

    def __init__(self, variant, B, T, H, dk, dv, chunk=64, io="bf16", out="f32",
                 grad="f32", scale=1.0, cu_seqlens=None, device="cuda", prepare=False):
        import torch
        self.device = torch.device(device)
        d = DrDesc()
        d.B, d.T, d.H, d.d_k, d.d_v, d.chunk = B, T, H, dk, dv, chunk
        d.variant = VARIANTS[variant] if isinstance(variant, str) else int(variant)
        code = {"bf16": DR_BF16, "f32": DR_F32}
        d.io_dtype, d.out_dtype, d.grad_dtype = code[io], code[out], code[grad]
        d.scale = float(scale)
        self.base_flags = DR_FLAG_PREPARE_INPUTS if prepare else 0
        d.flags = self.base_flags
        self._keep = []
        if cu_seqlens is not None:
            cu_host = [int(x) for x in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist")
                                        else cu_seqlens)]
            table, offs, n = plan_varlen(cu_host, chunk)
            cu_d = torch.tensor(cu_host, dtype=torch.int32, device=self.device)
            tab_d = torch.tensor(table.reshape(-1) if n else [0, 0], dtype=torch.int32,
                                 device=self.device)
            off_d = torch.tensor(offs, dtype=torch.int32, device=self.device)
            self._keep += [cu_d, tab_d, off_d]
            d.num_seqs = len(cu_host) - 1
            d.cu_seqlens, d.chunk_table, d.chunk_offsets = cu_d.data_ptr(), tab_d.data_ptr(), off_d.data_ptr()
            d.num_chunks = n
        else:
            d.num_seqs = B
            d.cu_seqlens = d.chunk_table = d.chunk_offsets = None
            d.num_chunks = 0
        self.desc = d
        self.N = d.num_seqs
        nbytes = workspace_bytes(d)
        if nbytes == 0:
            raise DrError(DR_ERR_UNSUPPORTED, "dr_workspace_bytes")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.io_dtype = torch.bfloat16 if io == "bf16" else torch.float32
        self.out_dtype = torch.bfloat16 if out == "bf16" else torch.float32
        self.grad_dtype = torch.bfloat16 if grad == "bf16" else torch.float32

    def _stream(self):
        import torch
        return torch.cuda.current_stream(self.device).cuda_stream

    def forward(self, q, k, v, beta, g=None, h0=None, o=None, hT=None, want_hT=True, u=None):
        """o, hT; with `u` (a [B,T,H,dv] tensor of the output dtype) also the write
        beta r of every token (dr_fwd_u)."""
        import torch
        d = self.desc
        if o is None:
            o = torch.empty(d.B, d.T, d.H, d.d_v, dtype=self.out_dtype, device=self.device)
        if hT is None and want_hT:
            hT = torch.empty(self.N, d.H, d.d_k, d.d_v, dtype=torch.float32, device=self.device)
        if u is None:
            _check(dr_fwd(d, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0), _ptr(o),
                          _ptr(hT), self.ws.data_ptr(), self.ws.numel(), self._stream()), "dr_fwd")
        else:
            _check(dr_fwd_u(d, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0), _ptr(o),
                            _ptr(hT), _ptr(u), self.ws.data_ptr(), self.ws.numel(),
                            self._stream()), "dr_fwd_u")
        return o, hT

    def backward(self, q, k, v, beta, g, h0, dO, dhT=None, reuse_fwd=False, out=None, dU=None):
        import torch
        d = self.desc
        if out is None:
            out = {
                "dq": torch.empty(d.B, d.T, d.H, d.d_k, dtype=self.grad_dtype, device=self.device),
                "dk": torch.empty(d.B, d.T, d.H, d.d_k, dtype=self.grad_dtype, device=self.device),
                "dv": torch.empty(d.B, d.T, d.H, d.d_v, dtype=self.grad_dtype, device=self.device),
                "dbeta": torch.empty(d.B, d.T, d.H, dtype=torch.float32, device=self.device),
                "dg": None if g is None else torch.empty_like(g, dtype=torch.float32),
                "dh0": torch.empty(self.N, d.H, d.d_k, d.d_v, dtype=torch.float32,
                                   device=self.device),
            }
        d.flags = self.base_flags | (DR_FLAG_REUSE_FWD if reuse_fwd else 0)
        try:
            if dU is None:
                _check(dr_bwd(d, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
                              _ptr(dO), _ptr(dhT), _ptr(out["dq"]), _ptr(out["dk"]),
                              _ptr(out["dv"]), _ptr(out["dbeta"]), _ptr(out["dg"]),
                              _ptr(out["dh0"]), self.ws.data_ptr(), self.ws.numel(),
                              self._stream()), "dr_bwd")
            else:
                _check(dr_bwd_u(d, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
                                _ptr(dO), _ptr(dhT), _ptr(dU), _ptr(out["dq"]), _ptr(out["dk"]),
                                _ptr(out["dv"]), _ptr(out["dbeta"]), _ptr(out["dg"]),
                                _ptr(out["dh0"]), self.ws.data_ptr(), self.ws.numel(),
                                self._stream()), "dr_bwd_u")
        finally:
            d.flags = self.base_flags
        return out

    def status(self) -> int:
        return check_status(self.ws.data_ptr(), self._stream())


class Decoder:
    """Descriptor for the recurrent (token-by-token) step: `step` enqueues dr_decode
    on the current torch stream and updates `state` ([B, H, dk, dv] fp32) in place."""

    def __init__(self, variant, B, T, H, dk, dv, io="bf16", out="f32", scale=1.0,
                 device="cuda", prepare=False):
        import torch
        self.device = torch.device(device)
        d = DrDesc()
        d.B, d.T, d.H, d.d_k, d.d_v, d.chunk = B, T, H, dk, dv, 1
        d.variant = VARIANTS[variant] if isinstance(variant, str) else int(variant)
        code = {"bf16": DR_BF16, "f32": DR_F32}
        d.io_dtype, d.out_dtype, d.grad_dtype = code[io], code[out], code[out]
        d.scale = float(scale)
        d.flags = DR_FLAG_PREPARE_INPUTS if prepare else 0
        d.num_seqs = B
        d.cu_seqlens = d.chunk_table = d.chunk_offsets = None
        d.num_chunks = 0
        self.desc = d
        self.out_dtype = torch.bfloat16 if out == "bf16" else torch.float32

    def step(self, q, k, v, beta, g, state, o=None):
        import torch
        d = self.desc
        if o is None:
            o = torch.empty(d.B, d.T, d.H, d.d_v, dtype=self.out_dtype, device=self.device)
        _check(dr_decode(d, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(state), _ptr(o),
                         torch.cuda.current_stream(self.device).cuda_stream), "dr_decode")
        return o

    def step_gdn2(self, q, k, v, erase, write, g, state, o=None):
        """Gated DeltaNet-2 (a Decoder built with variant "gdn2"): dr_gdn2_decode."""
        import torch
        d = self.desc
        if o is None:
            o = torch.empty(d.B, d.T, d.H, d.d_v, dtype=self.out_dtype, device=self.device)
        _check(load().dr_gdn2_decode(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(erase),
                                     _ptr(write), _ptr(g), _ptr(state), _ptr(o),
                                     torch.cuda.current_stream(self.device).cuda_stream),
               "dr_gdn2_decode")
        return o


class Gdn2Problem(Problem):
    """Gated DeltaNet-2 (dr_gdn2_fwd / dr_gdn2_bwd): the erase gate [B,T,H,dk] and the
    write gate [B,T,H,dv] take the place of beta."""

    def __init__(self, B, T, H, dk, dv, chunk=64, io="bf16", out="f32", grad="f32",
                 scale=1.0, cu_seqlens=None, device="cuda"):
        super().__init__("gdn2", B, T, H, dk, dv, chunk=chunk, io=io, out=out, grad=grad,
                         scale=scale, cu_seqlens=cu_seqlens, device=device)

    def forward(self, q, k, v, erase, write, g, h0=None, o=None, hT=None, want_hT=True):
        import torch
        d = self.desc
        if o is None:
            o = torch.empty(d.B, d.T, d.H, d.d_v, dtype=self.out_dtype, device=self.device)
        if hT is None and want_hT:
            hT = torch.empty(self.N, d.H, d.d_k, d.d_v, dtype=torch.float32, device=self.device)
        _check(dr_gdn2_fwd(d, _ptr(q), _ptr(k), _ptr(v), _ptr(erase), _ptr(write), _ptr(g),
                           _ptr(h0), _ptr(o), _ptr(hT), self.ws.data_ptr(), self.ws.numel(),
                           self._stream()), "dr_gdn2_fwd")
        return o, hT

    def backward(self, q, k, v, erase, write, g, h0, dO, dhT=None, out=None, reuse_fwd=False):
        import torch
        d = self.desc
        if out is None:
            f32 = dict(dtype=torch.float32, device=self.device)
            out = {
                "dq": torch.empty(d.B, d.T, d.H, d.d_k, dtype=self.grad_dtype, device=self.device),
                "dk": torch.empty(d.B, d.T, d.H, d.d_k, dtype=self.grad_dtype, device=self.device),
                "dv": torch.empty(d.B, d.T, d.H, d.d_v, dtype=self.grad_dtype, device=self.device),
                "derase": torch.empty(d.B, d.T, d.H, d.d_k, **f32),
                "dwrite": torch.empty(d.B, d.T, d.H, d.d_v, **f32),
                "dg": torch.empty(d.B, d.T, d.H, **f32),
                "dh0": torch.empty(self.N, d.H, d.d_k, d.d_v, **f32),
            }
        d.flags = DR_FLAG_REUSE_FWD if reuse_fwd else 0
        try:
            _check(dr_gdn2_bwd(d, _ptr(q), _ptr(k), _ptr(v), _ptr(erase), _ptr(write), _ptr(g),
                               _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(out["dq"]), _ptr(out["dk"]),
                               _ptr(out["dv"]), _ptr(out["derase"]), _ptr(out["dwrite"]),
                               _ptr(out["dg"]), _ptr(out["dh0"]), self.ws.data_ptr(),
                               self.ws.numel(), self._stream()), "dr_gdn2_bwd")
        finally:
            d.flags = 0
        return out


# ------------------------------------------------------------------ softmax-attention layer
# A step of a serving loop makes these calls for a few microseconds of work on the device, so the
# argument checks compare whole shapes and ask for strides only where a tensor is not contiguous.
def _rows(t, shape, what, index):
    """Elements between the token rows of t, a tensor of the given shape [B, T, heads, d] on device `index`:
    contiguous, or a range of heads of a wider contiguous tensor."""
    if t.shape == shape and t.get_device() == index:
        B, T, H, D = shape
        if t.is_contiguous():
            return H * D
        s = t.stride()
        ld = s[1] if T > 1 else s[0]
        if (D == 1 or s[3] == 1) and (H == 1 or s[2] == D) and (T == 1 or B == 1 or s[0] == T * ld):
            return ld if B * T > 1 else H * D
    raise ValueError(f"{what}: shape {tuple(t.shape)} strides {t.stride()} on {t.device} is no {tuple(shape)} "
                     f"in the memory of device {index} with whole token rows at one distance")


def _address(t, dtype, shape, what, index):
    """Address of a contiguous tensor of the given type and shape on device `index`, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)} in the memory of "
                         f"device {index}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


_TORCH_TYPES = {"bf16": "bfloat16", "f32": "float32"}
_TYPE_CODES = {"bf16": DR_BF16, "f32": DR_F32}


def _torch_type(name):
    import torch
    return getattr(torch, _TORCH_TYPES[name])


class _Calls:
    """The device of a plan, its current stream, its allocations and workspaces."""

    def _at(self, device):
        import torch
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None and torch.cuda.is_available():
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._torch, self._f32, self._i32 = torch, torch.float32, torch.int32
        self._lib = load()
        self._index = self.device.index
        # the handle alone where torch offers it: building a Stream object costs more than a launch
        self._raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if self._raw is None or self._index is None:
            self._raw = lambda _: torch.cuda.current_stream(self.device).cuda_stream
        self._current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

    def _stream(self):
        """The current stream of the plan's device, which has to be the current one: a launch goes to the current
        device, and the default stream has the same handle on each."""
        if self._current() != self._index:
            raise ValueError(f"a plan of device {self._index} was called while device {self._current()} is the current one")
        return self._raw(self._index)

    def _empty(self, shape, dtype):
        return self._torch.empty(shape, dtype=dtype, device=self.device)

    def _workspace(self, stream):
        """A workspace for the calls of this thread on a stream: calls on another stream may run at the same
        time, and another thread's may put its kernels between the two of a call."""
        key = (self._ws_bytes, stream, threading.get_ident())
        ws = self._spaces.get(key)
        if ws is None:
            ws = self._spaces[key] = self._empty(self._ws_bytes, self._torch.uint8)
        return ws


class HeadNormRope(_Calls):
    """RMS norm of queries and keys for each head with the position rotation in the same pass
    (dr_norm_rope_fwd / dr_norm_rope_bwd) for one problem shape.

    q [B, T, Hq, d] and k [B, T, Hk, d] may be head ranges of one packed projection.  The position
    of token (b, t) is ``positions[b, t]`` (default t) plus ``start[b]`` (default 0), a row of the
    tables cos, sin [rows, rot / 2].

    A plan may be used on any stream of its device and by several threads: the gradient's
    workspace is one for each of both, kept with the plan."""

    def __init__(self, B, T, Hq, Hk, d, rot=None, style="halves", io="bf16", out="bf16", grad="bf16",
                 eps=1e-6, device="cuda"):
        self._at(device)
        e = DrRopeDesc()
        e.B, e.T, e.Hq, e.Hk, e.d = B, T, Hq, Hk, d
        e.rot = d if rot is None else rot
        e.style = ROPE_STYLES[style]
        e.io_dtype, e.out_dtype, e.grad_dtype = _TYPE_CODES[io], _TYPE_CODES[out], _TYPE_CODES[grad]
        e.eps = float(eps)
        e.ld_q = e.ld_oq = Hq * d
        e.ld_k = e.ld_ok = Hk * d
        e.table_rows = 0
        self.desc, self._ref = e, ctypes.byref(e)
        self._layouts = {}
        self.io_dtype, self.out_dtype, self.grad_dtype = map(_torch_type, (io, out, grad))
        self._q, self._k, self._w, self._rot = (B, T, Hq, d), (B, T, Hk, d), (d,), e.rot
        self._fwd, self._bwd = self._lib.dr_norm_rope_fwd, self._lib.dr_norm_rope_bwd
        self._spaces, self._ws_bytes = {}, int(self._lib.dr_norm_rope_workspace_bytes(self._ref))
        if self._ws_bytes == 0:
            raise DrError(DR_ERR_UNSUPPORTED, "dr_norm_rope_workspace_bytes")

    def _layout(self, ld_q, ld_k, ld_oq, ld_ok, table_rows):
        """The descriptor of calls with these row distances and rows of the tables.  It is not changed
        afterwards: the library reads it while other threads call."""
        key = (ld_q, ld_k, ld_oq, ld_ok, table_rows)
        ref = self._layouts.get(key)
        if ref is None:
            e = DrRopeDesc.from_buffer_copy(self.desc)
            e.ld_q, e.ld_k, e.ld_oq, e.ld_ok, e.table_rows = key
            ref = self._layouts[key] = ctypes.byref(e)
        return ref

    def _inputs(self, q, k, wq, wk, cos, sin, positions, start, ld_oq, ld_ok):
        """Checks the inputs of a call, and returns its descriptor and their addresses."""
        e, f32, i32, w, index = self.desc, self._f32, self._i32, self._w, self._index
        qp = kp = None
        ld_q, ld_k, rows = e.ld_q, e.ld_k, 0
        if self._q[2]:
            if q.dtype is not self.io_dtype:
                raise ValueError(f"q: expected {self.io_dtype}, got {q.dtype}")
            ld_q, qp = _rows(q, self._q, "q", index), q.data_ptr()
        if self._k[2]:
            if k.dtype is not self.io_dtype:
                raise ValueError(f"k: expected {self.io_dtype}, got {k.dtype}")
            ld_k, kp = _rows(k, self._k, "k", index), k.data_ptr()
        wqp, wkp = _address(wq, f32, w, "wq", index), _address(wk, f32, w, "wk", index)
        cp = sp = None
        if self._rot:
            rows = cos.shape[0]
            table = (rows, self._rot // 2)
            cp, sp = _address(cos, f32, table, "cos", index), _address(sin, f32, table, "sin", index)
        return (self._layout(ld_q, ld_k, ld_oq, ld_ok, rows), qp, kp, wqp, wkp, cp, sp,
                _address(positions, i32, self._q[:2], "positions", index),
                _address(start, i32, self._q[:1], "start", index))

    def _output(self, t, shape, dtype, what):
        """A given output, or a new one, and its row distance."""
        if t is None:
            return self._torch.empty(shape, dtype=dtype, device=self.device), shape[2] * shape[3]
        if t.dtype is not dtype:
            raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
        return t, _rows(t, shape, what, self._index)

    def forward(self, q, k, wq, wk, cos, sin, positions=None, start=None, yq=None, yk=None):
        """yq, yk in the output type (given: written there, in place where it is q or k itself)."""
        yq, ld_oq = self._output(yq, self._q, self.out_dtype, "yq")
        yk, ld_ok = self._output(yk, self._k, self.out_dtype, "yk")
        rc = self._fwd(*self._inputs(q, k, wq, wk, cos, sin, positions, start, ld_oq, ld_ok), yq.data_ptr(),
                       yk.data_ptr(), self._stream())
        if rc:
            raise DrError(rc, "dr_norm_rope_fwd")
        return yq, yk

    def backward(self, q, k, wq, wk, cos, sin, dyq, dyk, positions=None, start=None, out=None):
        """{dq, dk, dwq, dwk} for the incoming gradients dyq, dyk (contiguous, of the input type)."""
        w, f32, index = self._w, self._f32, self._index
        given = out or {}
        dq, ld_oq = self._output(given.get("dq"), self._q, self.grad_dtype, "dq")
        dk, ld_ok = self._output(given.get("dk"), self._k, self.grad_dtype, "dk")
        dwq, dwk = given.get("dwq"), given.get("dwk")
        if out is None:
            empty, device = self._torch.empty, self.device
            dwq = None if wq is None else empty(w, dtype=f32, device=device)
            dwk = None if wk is None else empty(w, dtype=f32, device=device)
        stream = self._stream()
        rc = self._bwd(*self._inputs(q, k, wq, wk, cos, sin, positions, start, ld_oq, ld_ok),
                       _address(dyq, self.io_dtype, self._q, "dyq", index),
                       _address(dyk, self.io_dtype, self._k, "dyk", index), dq.data_ptr(), dk.data_ptr(),
                       _address(dwq, f32, w, "dwq", index), _address(dwk, f32, w, "dwk", index),
                       self._workspace(stream).data_ptr(), self._ws_bytes, stream)
        if rc:
            raise DrError(rc, "dr_norm_rope_bwd")
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


class KvCache(_Calls):
    """A paged cache of keys and values in 8 bits ("i8" or "e4m3") with one scale for each page and
    head (dr_cache_write / dr_cache_read).  ``buffers`` = (k codes, v codes, k scales, v scales)
    takes existing device memory: codes [num_pages, H, page, d] of one byte each, scales
    [num_pages, H] fp32."""

    def __init__(self, num_pages, H, d, page=64, code="i8", buffers=None, device="cuda"):
        import torch
        self._at(device)
        kind = torch.int8 if code == "i8" else torch.float8_e4m3fn
        if buffers is None:
            buffers = [torch.zeros(num_pages, H, page, d, dtype=torch.int8, device=self.device).view(kind)
                       for _ in range(2)]
            buffers += [torch.zeros(num_pages, H, dtype=torch.float32, device=self.device) for _ in range(2)]
        self.k, self.v, self.k_scale, self.v_scale = buffers
        for t, what in ((self.k, "k codes"), (self.v, "v codes")):
            _address(t, kind, (num_pages, H, page, d), what, self._index)
        for t, what in ((self.k_scale, "k scales"), (self.v_scale, "v scales")):
            _address(t, torch.float32, (num_pages, H), what, self._index)
        self.word = torch.zeros(4, dtype=torch.int32, device=self.device)
        self._spaces = {}  # workspaces of the attention plans
        c = DrCache()
        c.num_pages, c.H, c.d, c.page, c.code = num_pages, H, d, page, CACHE_CODES[code]
        c.k, c.v = self.k.data_ptr(), self.v.data_ptr()
        c.k_scale, c.v_scale = self.k_scale.data_ptr(), self.v_scale.data_ptr()
        c.status = self.word.data_ptr()
        self.desc, self._ref = c, ctypes.byref(c)
        self._heads = (H, d)
        self._io = {torch.bfloat16: DR_BF16, torch.float32: DR_F32}
        self._out = {"bf16": (torch.bfloat16, DR_BF16), "f32": (torch.float32, DR_F32)}
        self._write, self._read = self._lib.dr_cache_write, self._lib.dr_cache_read

    def seqs(self, B, table, lens, counts, T):
        """The call's positions: T tokens (or counts[b] <= T) after lens[b], in the pages of table
        [B, pages]."""
        i32, pages, index = self._i32, table.shape[-1], self._index
        return DrCacheSeqs(B, T, _address(table, i32, (B, pages), "table", index), pages,
                           _address(lens, i32, (B,), "lens", index), _address(counts, i32, (B,), "counts", index))

    def write(self, k, v, table, lens, counts=None):
        """Append k, v [B, T, H, d] (bf16 or fp32, or head ranges of a packed projection) after the
        first lens[b] positions of every sequence."""
        code = self._io.get(k.dtype)
        if code is None or v.dtype is not k.dtype:
            raise ValueError("k, v: expected two bf16 or two fp32 tensors")
        B, T = k.shape[:2]
        shape, index = (B, T, *self._heads), self._index
        s = self.seqs(B, table, lens, counts, T)
        rc = self._write(self._ref, ctypes.byref(s), k.data_ptr(), _rows(k, shape, "k", index), v.data_ptr(),
                         _rows(v, shape, "v", index), code, self._stream())
        if rc:
            raise DrError(rc, "dr_cache_write")

    def read(self, table, lens, counts, T, out="bf16", k=None, v=None):
        """k, v [B, T, H, d]: the values at positions lens[b] .. lens[b] + counts[b] - 1, zeros after."""
        dtype, code = self._out[out]
        B = lens.shape[0]
        s = self.seqs(B, table, lens, counts, T)
        shape, index = (B, T, *self._heads), self._index
        empty, device = self._torch.empty, self.device
        k = empty(shape, dtype=dtype, device=device) if k is None else k
        v = empty(shape, dtype=dtype, device=device) if v is None else v
        rc = self._read(self._ref, ctypes.byref(s), _address(k, dtype, shape, "k", index),
                        _address(v, dtype, shape, "v", index), code, self._stream())
        if rc:
            raise DrError(rc, "dr_cache_read")
        return k, v

    def status(self) -> int:
        """DR_OK, or DR_ERR_INDEX after a call met a page number, length or count out of range."""
        return check_status(self.word.data_ptr(), self._stream())

    def clear_status(self) -> None:
        self.word.zero_()


class CacheAttention(_Calls):
    """Attention of up to T query tokens of each of B sequences over a KvCache (dr_cache_attn).

    A plan may be used on any stream of its device and by several threads: there is a workspace for each of
    both.  The workspaces are the cache's, for all plans over it, so that a plan itself is only a
    descriptor.  Graphs that were captured on one stream share its workspace, so they are replayed one
    after another."""

    def __init__(self, cache, B, T, Hq, io="bf16", out="bf16", scale=None, window=0):
        self._at(cache.device)
        self.cache, self.B, self.T = cache, B, T
        d = cache.desc.d
        a = DrAttnDesc(Hq, _TYPE_CODES[io], _TYPE_CODES[out], window,
                       d ** -0.5 if scale is None else float(scale), Hq * d)
        self.desc, self._ref = a, ctypes.byref(a)
        self._layouts = {a.ld_q: self._ref}  # descriptors by row distance, not changed afterwards
        self.io_dtype, self.out_dtype = _torch_type(io), _torch_type(out)
        self._shape = (B, T, Hq, d)
        n = int(self._lib.dr_cache_attn_workspace_bytes(cache._ref, self._ref, B, T))
        if n == 0:
            raise DrError(DR_ERR_UNSUPPORTED, "dr_cache_attn_workspace_bytes")
        self._spaces, self._ws_bytes, self._attn = cache._spaces, n, self._lib.dr_cache_attn

    @property
    def ws(self):
        """The workspace of this thread's calls on the current stream."""
        return self._workspace(self._stream())

    def forward(self, q, table, lens, counts=None, o=None, lse=None, want_lse=False):
        """o [B, T, Hq, d] and lse [B, T, Hq] (or None): query t of sequence b is the position
        lens[b] + t, which the cache already holds."""
        shape, cache, index = self._shape, self.cache, self._index
        if q.dtype is not self.io_dtype:
            raise ValueError(f"q: expected {self.io_dtype}, got {q.dtype}")
        ld_q = _rows(q, shape, "q", index)
        ref = self._layouts.get(ld_q)
        if ref is None:
            a = DrAttnDesc.from_buffer_copy(self.desc)
            a.ld_q = ld_q
            ref = self._layouts[ld_q] = ctypes.byref(a)
        s = cache.seqs(self.B, table, lens, counts, self.T)
        empty, device = self._torch.empty, self.device
        o = empty(shape, dtype=self.out_dtype, device=device) if o is None else o
        lse = empty(shape[:3], dtype=self._f32, device=device) if lse is None and want_lse else lse
        stream = self._stream()
        rc = self._attn(cache._ref, ctypes.byref(s), ref, q.data_ptr(),
                        _address(o, self.out_dtype, shape, "o", index),
                        _address(lse, self._f32, shape[:3], "lse", index),
                        self._workspace(stream).data_ptr(), self._ws_bytes, stream)
        if rc:
            raise DrError(rc, "dr_cache_attn")
        return o, lse


# ------------------------------------------------------------------ token mixers over whole prompts
class _Mixer(_Calls):
    """What the plans of PromptAttention and LinearAttention share: tensors as rows of heads, sequences
    dense [B, T] or packed into the rows of one (B = 1, ``seqs`` of them, offsets ``cu`` at each call)."""

    def _plan(self, desc, seqs, io, word):
        d = self.desc = desc
        if seqs is not None and d.B != 1:
            raise ValueError("packed sequences are the rows of one batch: B has to be 1")
        d.num_seqs = d.B if seqs is None else seqs
        d.io_dtype = _TYPE_CODES[io]
        self.io_dtype, self._cu = _torch_type(io), None if seqs is None else (seqs + 1,)
        self._refs, self._spaces = {}, {}
        self._zeroed = None
        if word is None:
            cuda = self._torch.cuda
            word = self._torch.zeros(4, dtype=self._i32, device=self.device)
            if self.device.type == "cuda" and not cuda.is_current_stream_capturing():
                self._zeroed = cuda.current_stream(self.device).record_event()
        else:
            _address(word, self._i32, (4,), "word", self._index if self.device.type == "cuda" else -1)
        self.word = word
        d.status = word.data_ptr()

    def status(self) -> int:
        """DR_OK, or DR_ERR_TIMEOUT after a kernel's bounded wait ran out (of any plan with the same word)."""
        stream, zeroed = self._stream(), self._zeroed
        if zeroed is not None:
            # the zeros may still wait on the stream the plan was made on (a kernel's report comes two seconds after it at
            # the earliest)
            self._torch.cuda.current_stream(self.device).wait_event(zeroed)
        code = check_status(self.word.data_ptr(), stream)
        self._zeroed = None
        return code

    def _ref(self, lds):
        """The descriptor of calls with these six row distances.  It is not changed afterwards: the library
        reads it while other threads call."""
        ref = self._refs.get(lds)
        if ref is None:
            d = type(self.desc).from_buffer_copy(self.desc)
            d.ld_q, d.ld_k, d.ld_v, d.ld_dq, d.ld_dk, d.ld_dv = lds
            ref = self._refs[lds] = ctypes.byref(d)
        return ref

    def _offsets(self, cu):
        if (cu is None) != (self._cu is None):
            raise ValueError("cu: the offsets of packed sequences go with a plan that was made with seqs")
        return None if cu is None else _address(cu, self._i32, self._cu, "cu", self._index)

    def _in(self, t, shape, what):
        """Row distance and address of an input."""
        if t.dtype is not self.io_dtype:
            raise ValueError(f"{what}: expected {self.io_dtype}, got {t.dtype}")
        return _rows(t, shape, what, self._index), t.data_ptr()

    def _out(self, t, shape, what):
        """A given gradient or a new one, its row distance and address."""
        if t is None:
            t = self._empty(shape, self.io_dtype)
        return (t, *self._in(t, shape, what))


class PromptAttention(_Mixer):
    """Causal softmax attention over whole prompts and its gradient (dr_prompt_attn_fwd / dr_prompt_attn_bwd):
    q [B, T, Hq, d], k and v [B, T, H, d], which may be head ranges of one packed projection; query head h
    reads key head h // (Hq // H).

    ``seqs``: packed sequences, at most that many (2^20 at most); B is 1, T the rows in all, and each call takes
    the offsets ``cu`` [seqs + 1] (int32, device).  Rows of no sequence are left as they were.

    ``word``: another plan's, so that its status() tells of this one's calls too, also when this one is gone.

    A plan may be used on any stream of its device and by several threads: the gradient's workspace is one for
    each of both, kept with the plan; graphs that were captured on one stream share it, so they are replayed
    one after another."""

    def __init__(self, B, T, Hq, H, d, seqs=None, io="bf16", scale=None, window=0, device="cuda", word=None):
        self._at(device)
        e = DrPromptDesc()
        e.B, e.T, e.Hq, e.H, e.d, e.window = B, T, Hq, H, d, window
        e.scale = d ** -0.5 if scale is None else float(scale)
        e.ld_q = e.ld_dq = Hq * d
        e.ld_k = e.ld_v = e.ld_dk = e.ld_dv = H * d
        self._plan(e, seqs, io, word)
        self._q, self._k, self._lse = (B, T, Hq, d), (B, T, H, d), (B, T, Hq)
        self._fwd, self._bwd = self._lib.dr_prompt_attn_fwd, self._lib.dr_prompt_attn_bwd
        self._ws_bytes = int(self._lib.dr_prompt_attn_workspace_bytes(ctypes.byref(e)))
        if self._ws_bytes == 0:
            raise DrError(DR_ERR_UNSUPPORTED, "dr_prompt_attn_workspace_bytes")

    def forward(self, q, k, v, cu=None, o=None, lse=None, want_lse=False):
        """o [B, T, Hq, d] and lse [B, T, Hq] fp32 (or None)."""
        e, index = self.desc, self._index
        (ld_q, qp), (ld_k, kp), (ld_v, vp) = self._in(q, self._q, "q"), self._in(k, self._k, "k"), self._in(v, self._k, "v")
        o = self._empty(self._q, self.io_dtype) if o is None else o
        lse = self._empty(self._lse, self._f32) if lse is None and want_lse else lse
        rc = self._fwd(self._ref((ld_q, ld_k, ld_v, e.ld_dq, e.ld_dk, e.ld_dv)), qp, kp, vp, self._offsets(cu),
                       _address(o, self.io_dtype, self._q, "o", index),
                       _address(lse, self._f32, self._lse, "lse", index), self._stream())
        if rc:
            raise DrError(rc, "dr_prompt_attn_fwd")
        return o, lse

    def backward(self, q, k, v, o, lse, dO, cu=None, out=None):
        """{dq, dk, dv} for the incoming gradient dO, with the forward's inputs and results.  ``out``: tensors to
        write to, also head ranges of one packed gradient."""
        index, given = self._index, out or {}
        (ld_q, qp), (ld_k, kp), (ld_v, vp) = self._in(q, self._q, "q"), self._in(k, self._k, "k"), self._in(v, self._k, "v")
        dq, ld_dq, dqp = self._out(given.get("dq"), self._q, "dq")
        dk, ld_dk, dkp = self._out(given.get("dk"), self._k, "dk")
        dv, ld_dv, dvp = self._out(given.get("dv"), self._k, "dv")
        if lse is None:
            raise ValueError("lse: the gradient needs the forward's")
        stream = self._stream()
        rc = self._bwd(self._ref((ld_q, ld_k, ld_v, ld_dq, ld_dk, ld_dv)), qp, kp, vp,
                       _address(o, self.io_dtype, self._q, "o", index), _address(lse, self._f32, self._lse, "lse", index),
                       _address(dO, self.io_dtype, self._q, "dO", index), self._offsets(cu), dqp, dkp, dvp,
                       self._workspace(stream).data_ptr(), self._ws_bytes, stream)
        if rc:
            raise DrError(rc, "dr_prompt_attn_bwd")
        return {"dq": dq, "dk": dk, "dv": dv}


class LinearAttention(_Mixer):
    """Linear attention with a decay for each head, S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t: over
    whole prompts in chunks, its gradient, and the recurrent step (dr_linear_attn_fwd / _bwd / _step).

    q, k [B, T, H, dk] and v [B, T, H, dv] may be head ranges of one packed projection; g [H] fp32 is the
    log-decay of a step, a constant of the layer; states are [sequences, H, dk, dv] fp32.  ``seqs`` and ``cu``:
    packed sequences, as for PromptAttention, and so are ``word``, streams, threads and graphs."""

    def __init__(self, B, T, H, dk, dv, seqs=None, io="bf16", scale=1.0, device="cuda", word=None):
        self._at(device)
        e = DrLinearDesc()
        e.B, e.T, e.H, e.d_k, e.d_v = B, T, H, dk, dv
        e.scale = float(scale)
        e.ld_q = e.ld_k = e.ld_dq = e.ld_dk = H * dk
        e.ld_v = e.ld_dv = H * dv
        self._plan(e, seqs, io, word)
        self._k, self._v, self._g = (B, T, H, dk), (B, T, H, dv), (H,)
        self._h = (e.num_seqs, H, dk, dv)
        self._fwd, self._bwd, self._step = (getattr(self._lib, "dr_linear_attn_" + n) for n in ("fwd", "bwd", "step"))
        self._ws_bytes = int(self._lib.dr_linear_attn_workspace_bytes(ctypes.byref(e)))
        # sizes that only the recurrent step takes: the library refuses the other calls itself
        if self._ws_bytes == 0 and not (dk in (16, 32, 64, 128) and dv in (16, 32, 64, 128) and seqs is None):
            raise DrError(DR_ERR_UNSUPPORTED, "dr_linear_attn_workspace_bytes")

    def _inputs(self, q, k, v):
        return (*self._in(q, self._k, "q"), *self._in(k, self._k, "k"), *self._in(v, self._v, "v"))

    def _state(self, t, what):
        return _address(t, self._f32, self._h, what, self._index)

    def _decays(self, g):
        if g is None:
            raise ValueError("g: the log-decays of the heads are missing")
        return _address(g, self._f32, self._g, "g", self._index)

    def forward(self, q, k, v, g, h0=None, cu=None, o=None, hT=None, want_hT=True):
        """o [B, T, H, dv] and the states after the last tokens (or None); h0 None: empty states before."""
        e = self.desc
        ld_q, qp, ld_k, kp, ld_v, vp = self._inputs(q, k, v)
        o = self._empty(self._v, self.io_dtype) if o is None else o
        hT = self._empty(self._h, self._f32) if hT is None and want_hT else hT
        stream = self._stream()
        rc = self._fwd(self._ref((ld_q, ld_k, ld_v, e.ld_dq, e.ld_dk, e.ld_dv)), qp, kp, vp, self._decays(g),
                       self._state(h0, "h0"), self._offsets(cu), _address(o, self.io_dtype, self._v, "o", self._index),
                       self._state(hT, "hT"), self._workspace(stream).data_ptr(), self._ws_bytes, stream)
        if rc:
            raise DrError(rc, "dr_linear_attn_fwd")
        return o, hT

    def backward(self, q, k, v, g, dO, h0=None, dhT=None, cu=None, out=None, want_dh0=None):
        """{dq, dk, dv, dh0} for the incoming gradients dO and dhT (None: zero).  dh0 is None unless it is wanted
        (default: where h0 or dhT is given).  ``out``: tensors to write to, also head ranges of one packed
        gradient."""
        given = out or {}
        ld_q, qp, ld_k, kp, ld_v, vp = self._inputs(q, k, v)
        dq, ld_dq, dqp = self._out(given.get("dq"), self._k, "dq")
        dk, ld_dk, dkp = self._out(given.get("dk"), self._k, "dk")
        dv, ld_dv, dvp = self._out(given.get("dv"), self._v, "dv")
        dh0 = given.get("dh0")
        if want_dh0 is None:
            want_dh0 = h0 is not None or dhT is not None
        if dh0 is None and want_dh0:
            dh0 = self._empty(self._h, self._f32)
        stream = self._stream()
        rc = self._bwd(self._ref((ld_q, ld_k, ld_v, ld_dq, ld_dk, ld_dv)), qp, kp, vp, self._decays(g),
                       self._state(h0, "h0"), _address(dO, self.io_dtype, self._v, "dO", self._index),
                       self._state(dhT, "dhT"), self._offsets(cu), dqp, dkp, dvp, self._state(dh0, "dh0"),
                       self._workspace(stream).data_ptr(), self._ws_bytes, stream)
        if rc:
            raise DrError(rc, "dr_linear_attn_bwd")
        return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh0}

    def step(self, q, k, v, g, state, o=None):
        """o [B, T, H, dv] of the T next tokens of every sequence; ``state`` [B, H, dk, dv] is updated in place."""
        if self._cu is not None:
            raise ValueError("the recurrent step takes dense batches")
        if state is None:
            raise ValueError("state: missing")
        e = self.desc
        ld_q, qp, ld_k, kp, ld_v, vp = self._inputs(q, k, v)
        o = self._empty(self._v, self.io_dtype) if o is None else o
        rc = self._step(self._ref((ld_q, ld_k, ld_v, e.ld_dq, e.ld_dk, e.ld_dv)), qp, kp, vp, self._decays(g),
                        self._state(state, "state"), _address(o, self.io_dtype, self._v, "o", self._index),
                        self._stream())
        if rc:
            raise DrError(rc, "dr_linear_attn_step")
        return o
