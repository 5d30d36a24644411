"""Host-side checks of the attention layer's entry points (no GPU: nothing is launched)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from delta_rule_recurrent_gated_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000  # a 16-byte aligned address that no call may touch


@pytest.fixture(scope="module")
def lib():
    from delta_rule_recurrent_gated_gb300 import build
    build.build()
    return B.load()


@pytest.mark.parametrize("cname,cls", [("dr_rope_desc", B.DrRopeDesc), ("dr_cache", B.DrCache),
                                       ("dr_cache_seqs", B.DrCacheSeqs), ("dr_attn_desc", B.DrAttnDesc)])
def test_struct_layouts_match_the_header(tmp_path, cname, cls):
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    names = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dr.h"\nint main(void){' +
                   "".join(f'printf("%zu\\n", offsetof({cname}, {n}));' for n in names) +
                   f'printf("%zu\\n", sizeof({cname}));return 0;}}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "a")], check=True)
    out = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [getattr(cls, n).offset for n in names] + [ctypes.sizeof(cls)]


def rope(**kw):
    e = B.DrRopeDesc()
    e.B, e.T, e.Hq, e.Hk, e.d, e.rot = 2, 3, 4, 2, 128, 64
    e.style, e.io_dtype, e.out_dtype, e.grad_dtype, e.table_rows, e.eps = 0, 0, 0, 0, 10, 1e-6
    e.ld_q, e.ld_k, e.ld_oq, e.ld_ok = 512, 256, 512, 256
    for k, v in kw.items():
        setattr(e, k, v)
    return e


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), B.DR_ERR_INVALID_ARG), (dict(T=-1), B.DR_ERR_INVALID_ARG),
    (dict(Hq=0, Hk=0), B.DR_ERR_INVALID_ARG), (dict(d=0), B.DR_ERR_INVALID_ARG),
    (dict(rot=144), B.DR_ERR_INVALID_ARG), (dict(rot=-16), B.DR_ERR_INVALID_ARG),
    (dict(style=2), B.DR_ERR_INVALID_ARG), (dict(io_dtype=3), B.DR_ERR_INVALID_ARG),
    (dict(eps=-1.0), B.DR_ERR_INVALID_ARG), (dict(eps=float("nan")), B.DR_ERR_INVALID_ARG),
    (dict(ld_q=511), B.DR_ERR_INVALID_ARG), (dict(ld_ok=0), B.DR_ERR_INVALID_ARG),
    (dict(table_rows=-1), B.DR_ERR_INVALID_ARG), (dict(ld_k=260), B.DR_ERR_ALIGNMENT),
    (dict(d=100, rot=0), B.DR_ERR_UNSUPPORTED), (dict(d=264, ld_q=2000, ld_k=2000), B.DR_ERR_UNSUPPORTED),
    (dict(rot=24), B.DR_ERR_UNSUPPORTED),
])
def test_norm_rope_refuses(lib, kw, code):
    e = rope(**kw)
    p = [PTR] * 2 + [None, None] + [PTR] * 2 + [None, None] + [PTR] * 2
    assert lib.dr_norm_rope_fwd(ctypes.byref(e), *p, None) == code
    p = [PTR] * 2 + [None, None] + [PTR] * 2 + [None, None] + [PTR] * 4 + [None, None]
    assert lib.dr_norm_rope_bwd(ctypes.byref(e), *p, PTR, 1 << 30, None) == code
    assert lib.dr_norm_rope_workspace_bytes(ctypes.byref(e)) == 0


def test_norm_rope_refuses_pointers(lib):
    e = rope()
    ok = [PTR] * 4 + [PTR] * 2 + [None, None] + [PTR] * 2  # q k wq wk cos sin positions start yq yk
    for i, bad, code in ((0, None, B.DR_ERR_INVALID_ARG), (1, None, B.DR_ERR_INVALID_ARG),
                         (4, None, B.DR_ERR_INVALID_ARG), (5, None, B.DR_ERR_INVALID_ARG),
                         (8, None, B.DR_ERR_INVALID_ARG), (9, PTR + 8, B.DR_ERR_ALIGNMENT),
                         (2, PTR + 4, B.DR_ERR_ALIGNMENT)):
        p = list(ok)
        p[i] = bad
        assert lib.dr_norm_rope_fwd(ctypes.byref(e), *p, None) == code, i
    bwd = [PTR] * 4 + [PTR] * 2 + [None, None] + [PTR] * 4 + [PTR] * 2  # .. dyq dyk dq dk dwq dwk
    need = lib.dr_norm_rope_workspace_bytes(ctypes.byref(e))
    assert need > 0
    assert lib.dr_norm_rope_bwd(ctypes.byref(e), *bwd, PTR, need - 1, None) == B.DR_ERR_WORKSPACE
    assert lib.dr_norm_rope_bwd(ctypes.byref(e), *bwd, None, need, None) == B.DR_ERR_WORKSPACE
    bwd[2] = None  # dwq of a weight that is not there
    assert lib.dr_norm_rope_bwd(ctypes.byref(e), *bwd, PTR, need, None) == B.DR_ERR_INVALID_ARG
    # no tokens: nothing to do, whatever the pointers
    e = rope(B=0)
    assert lib.dr_norm_rope_fwd(ctypes.byref(e), *([None] * 10), None) == B.DR_OK


def cache(**kw):
    c = B.DrCache()
    c.num_pages, c.H, c.d, c.page, c.code = 8, 2, 128, 64, 0
    c.k = c.v = c.k_scale = c.v_scale = c.status = PTR
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs(**kw):
    s = B.DrCacheSeqs()
    s.B, s.T, s.table_stride = 2, 3, 4
    s.page_table = s.lens = PTR
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def attn(**kw):
    a = B.DrAttnDesc()
    a.Hq, a.io_dtype, a.out_dtype, a.window, a.scale, a.ld_q = 8, 0, 0, 0, 0.1, 1024
    for k, v in kw.items():
        setattr(a, k, v)
    return a


CALL_REFUSALS = [
    (dict(H=0), {}, B.DR_ERR_INVALID_ARG), (dict(num_pages=-1), {}, B.DR_ERR_INVALID_ARG),
    (dict(code=2), {}, B.DR_ERR_INVALID_ARG), (dict(d=96), {}, B.DR_ERR_UNSUPPORTED),
    (dict(page=48), {}, B.DR_ERR_UNSUPPORTED), (dict(page=256), {}, B.DR_ERR_UNSUPPORTED),
    (dict(k=None), {}, B.DR_ERR_INVALID_ARG), (dict(v_scale=None), {}, B.DR_ERR_INVALID_ARG),
    (dict(v=PTR + 8), {}, B.DR_ERR_ALIGNMENT), (dict(status=PTR + 2), {}, B.DR_ERR_ALIGNMENT),
    ({}, dict(B=-1), B.DR_ERR_INVALID_ARG), ({}, dict(T=-2), B.DR_ERR_INVALID_ARG),
    ({}, dict(lens=None), B.DR_ERR_INVALID_ARG), ({}, dict(page_table=None), B.DR_ERR_INVALID_ARG),
    ({}, dict(table_stride=-1), B.DR_ERR_INVALID_ARG), ({}, dict(lens=PTR + 4), B.DR_ERR_ALIGNMENT),
    ({}, dict(B=1 << 20, T=1 << 12), B.DR_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("ckw,skw,code", CALL_REFUSALS)
def test_cache_calls_refuse(lib, ckw, skw, code):
    c, s, a = cache(**ckw), seqs(**skw), attn()
    by = ctypes.byref
    assert lib.dr_cache_write(by(c), by(s), PTR, 1024, PTR, 1024, 0, None) == code
    assert lib.dr_cache_read(by(c), by(s), PTR, PTR, 0, None) == code
    assert lib.dr_cache_attn(by(c), by(s), by(a), PTR, PTR, None, PTR, 1 << 40, None) == code


def test_cache_write_and_read_refuse_their_own(lib):
    c, s, by = cache(), seqs(), ctypes.byref
    assert lib.dr_cache_write(by(c), by(s), None, 256, PTR, 256, 0, None) == B.DR_ERR_INVALID_ARG
    assert lib.dr_cache_write(by(c), by(s), PTR, 255, PTR, 256, 0, None) == B.DR_ERR_INVALID_ARG
    assert lib.dr_cache_write(by(c), by(s), PTR, 256, PTR, 260, 0, None) == B.DR_ERR_ALIGNMENT
    assert lib.dr_cache_write(by(c), by(s), PTR + 2, 256, PTR, 256, 0, None) == B.DR_ERR_ALIGNMENT
    assert lib.dr_cache_write(by(c), by(s), PTR, 256, PTR, 256, 7, None) == B.DR_ERR_INVALID_ARG
    assert lib.dr_cache_read(by(c), by(s), PTR, PTR + 8, 0, None) == B.DR_ERR_ALIGNMENT
    assert lib.dr_cache_read(by(c), by(s), PTR, PTR, 5, None) == B.DR_ERR_INVALID_ARG
    s = seqs(T=0)
    assert lib.dr_cache_write(by(c), by(s), None, 256, None, 256, 0, None) == B.DR_OK
    assert lib.dr_cache_read(by(c), by(s), None, None, 0, None) == B.DR_OK


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=0), B.DR_ERR_INVALID_ARG), (dict(Hq=7), B.DR_ERR_INVALID_ARG),
    (dict(window=-1), B.DR_ERR_INVALID_ARG), (dict(scale=float("inf")), B.DR_ERR_INVALID_ARG),
    (dict(io_dtype=9), B.DR_ERR_INVALID_ARG), (dict(ld_q=1023), B.DR_ERR_INVALID_ARG),
    (dict(ld_q=1028), B.DR_ERR_ALIGNMENT),
])
def test_attention_refuses(lib, kw, code):
    c, s, a, by = cache(), seqs(), attn(**kw), ctypes.byref
    assert lib.dr_cache_attn(by(c), by(s), by(a), PTR, PTR, None, PTR, 1 << 40, None) == code
    assert lib.dr_cache_attn_workspace_bytes(by(c), by(a), 2, 3) == 0


def test_attention_refuses_workspace_and_pointers(lib):
    c, s, a, by = cache(), seqs(), attn(), ctypes.byref
    need = lib.dr_cache_attn_workspace_bytes(by(c), by(a), 2, 3)
    assert need > 0
    assert lib.dr_cache_attn(by(c), by(s), by(a), PTR, PTR, None, PTR, need - 1, None) == B.DR_ERR_WORKSPACE
    assert lib.dr_cache_attn(by(c), by(s), by(a), PTR, PTR, None, None, need, None) == B.DR_ERR_WORKSPACE
    assert lib.dr_cache_attn(by(c), by(s), by(a), None, PTR, None, PTR, need, None) == B.DR_ERR_INVALID_ARG
    assert lib.dr_cache_attn(by(c), by(s), by(a), PTR, PTR + 8, None, PTR, need, None) == B.DR_ERR_ALIGNMENT
    s = seqs(B=0)
    assert lib.dr_cache_attn(by(c), by(s), by(a), None, None, None, None, 0, None) == B.DR_OK


def test_the_new_code_has_a_name(lib):
    assert B.error_string(B.DR_ERR_INDEX).startswith("DR_ERR_INDEX")
