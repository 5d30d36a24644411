"""Host-side checks of PromptAttention, LinearAttention and their entry points (no GPU: nothing is launched)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000  # a 16-byte aligned address that no call may touch


@pytest.fixture(scope="module")
def lib():
    from delta_rule_recurrent_gated_gb300 import build
    build.build()
    return B.load()


@pytest.mark.parametrize("cname,cls", [("dr_prompt_desc", B.DrPromptDesc), ("dr_linear_desc", B.DrLinearDesc)])
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


def prompt(**kw):
    d = B.DrPromptDesc(2, 3, 4, 2, 128, 2, B.DR_BF16, 0, 0.1, 512, 256, 256, 512, 256, 256)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def linear(**kw):
    d = B.DrLinearDesc(2, 3, 4, 64, 128, 2, B.DR_BF16, 0.1, 256, 256, 512, 256, 256, 512)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD = [(dict(B=-1), B.DR_ERR_INVALID_ARG), (dict(T=-1), B.DR_ERR_INVALID_ARG), (dict(num_seqs=-1), B.DR_ERR_INVALID_ARG),
       (dict(num_seqs=3), B.DR_ERR_INVALID_ARG), (dict(H=0), B.DR_ERR_INVALID_ARG), (dict(io_dtype=2), B.DR_ERR_INVALID_ARG),
       (dict(scale=float("nan")), B.DR_ERR_INVALID_ARG), (dict(ld_q=8), B.DR_ERR_INVALID_ARG), (dict(ld_v=516), B.DR_ERR_ALIGNMENT),
       (dict(B=1 << 20, T=1 << 12, num_seqs=1 << 20), B.DR_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(Hq=5, ld_q=640), B.DR_ERR_INVALID_ARG), (dict(window=-1), B.DR_ERR_INVALID_ARG), (dict(d=96), B.DR_ERR_UNSUPPORTED),
    (dict(d=0), B.DR_ERR_INVALID_ARG)])
def test_prompt_attn_refuses(lib, kw, code):
    d = prompt(**kw)
    assert lib.dr_prompt_attn_fwd(ctypes.byref(d), PTR, PTR, PTR, None, PTR, PTR, None) == code
    assert lib.dr_prompt_attn_bwd(ctypes.byref(d), *[PTR] * 6, None, *[PTR] * 4, 1 << 40, None) == code
    if "num_seqs" not in kw or kw["num_seqs"] < 0:
        assert lib.dr_prompt_attn_workspace_bytes(ctypes.byref(d)) == 0


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(d_k=96, ld_q=384, ld_k=384), B.DR_ERR_UNSUPPORTED), (dict(d_v=0), B.DR_ERR_INVALID_ARG), (dict(H=70000), B.DR_ERR_UNSUPPORTED),
    (dict(d_k=32), B.DR_ERR_UNSUPPORTED)])
def test_linear_attn_refuses(lib, kw, code):
    d = linear(**kw)
    assert lib.dr_linear_attn_fwd(ctypes.byref(d), *[PTR] * 5, None, PTR, PTR, PTR, 1 << 40, None) == code
    assert lib.dr_linear_attn_bwd(ctypes.byref(d), *[PTR] * 7, None, *[PTR] * 5, 1 << 40, None) == code
    if kw != dict(d_k=32):  # the step takes this size
        assert lib.dr_linear_attn_step(ctypes.byref(d), *[PTR] * 6, None) == code
    if "num_seqs" not in kw or kw["num_seqs"] < 0:
        assert lib.dr_linear_attn_workspace_bytes(ctypes.byref(d)) == 0


def test_calls_refuse_pointers_and_workspaces(lib):
    d, r = prompt(), ctypes.byref
    fwd = lambda *a, d=d: lib.dr_prompt_attn_fwd(r(d), *a, None)  # noqa: E731
    assert lib.dr_prompt_attn_fwd(None, *[PTR] * 3, None, PTR, PTR, None) == B.DR_ERR_INVALID_ARG
    for i in range(4):
        a = [PTR] * 3 + [None, PTR, None]
        a[i if i < 3 else 4] = None
        assert fwd(*a) == B.DR_ERR_INVALID_ARG
        a[i if i < 3 else 4] = PTR + 8
        assert fwd(*a) == B.DR_ERR_ALIGNMENT
    assert fwd(PTR, PTR, PTR, None, PTR, PTR + 4) == B.DR_ERR_ALIGNMENT
    assert fwd(PTR, PTR, PTR, PTR, PTR, None) == B.DR_ERR_INVALID_ARG  # offsets, and B = 2
    one = prompt(B=1, num_seqs=5)
    assert fwd(PTR, PTR, PTR, None, PTR, None, d=one) == B.DR_ERR_INVALID_ARG  # no offsets, and five sequences
    assert fwd(PTR, PTR, PTR, PTR + 2, PTR, None, d=one) == B.DR_ERR_ALIGNMENT
    n = lib.dr_prompt_attn_workspace_bytes(r(d))
    assert n >= 2 * 3 * 4 * 4
    bwd = lambda *a: lib.dr_prompt_attn_bwd(r(d), *a, None)  # noqa: E731
    assert bwd(*[PTR] * 6, None, *[PTR] * 4, n - 1) == B.DR_ERR_WORKSPACE
    assert bwd(*[PTR] * 6, None, *[PTR] * 3, None, n) == B.DR_ERR_WORKSPACE
    assert bwd(*[PTR] * 4, None, PTR, None, *[PTR] * 4, n) == B.DR_ERR_INVALID_ARG  # no lse
    e = linear()
    n = lib.dr_linear_attn_workspace_bytes(r(e))
    assert n > 0
    lfwd = lambda *a: lib.dr_linear_attn_fwd(r(e), *a, None)  # noqa: E731
    assert lfwd(*[PTR] * 5, None, PTR, PTR, PTR, n - 1) == B.DR_ERR_WORKSPACE
    assert lfwd(*[PTR] * 3, None, PTR, None, PTR, PTR, PTR, n) == B.DR_ERR_INVALID_ARG  # no g
    assert lfwd(*[PTR] * 4, PTR + 4, None, PTR, PTR, PTR, n) == B.DR_ERR_ALIGNMENT
    assert lib.dr_linear_attn_step(r(e), *[PTR] * 4, None, PTR, None) == B.DR_ERR_INVALID_ARG
    # nothing to do is no error, whatever the pointers are
    z = prompt(T=0)
    assert lib.dr_prompt_attn_fwd(r(z), *[None] * 6, None) == B.DR_OK
    z = linear(B=0, num_seqs=0)
    assert lib.dr_linear_attn_fwd(r(z), *[None] * 8, None, 0, None) == B.DR_OK
    assert lib.dr_linear_attn_step(r(z), *[None] * 6, None) == B.DR_OK


def test_plans_refuse_tensors(lib):
    """Shapes, types, layouts and devices are refused before anything is launched (plans and tensors on the CPU)."""
    p = B.PromptAttention(1, 6, 4, 2, 64, seqs=2, device="cpu")
    p._index = -1  # where get_device() puts CPU tensors
    p._current, p._raw = lambda: -1, lambda _: 0
    q, k, cu = torch.zeros(1, 6, 4, 64).bfloat16(), torch.zeros(1, 6, 2, 64).bfloat16(), torch.zeros(3, dtype=torch.int32)
    for bad, what in (((q.float(), k, k), "q"), ((q, k[:, :5], k), "k"), ((q, k, k.transpose(1, 2)), "v"),
                      ((q[..., ::2], k, k), "q")):
        with pytest.raises(ValueError, match=what):
            p.forward(*bad, cu=cu)
    for bad in (None, cu.long(), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError, match="cu"):
            p.forward(q, k, k, cu=bad)
    with pytest.raises(ValueError, match="lse"):
        p.backward(q, k, k, q, None, q, cu=cu)
    with pytest.raises(ValueError, match="B has to be 1"):
        B.PromptAttention(2, 6, 4, 2, 64, seqs=2, device="cpu")
    with pytest.raises(B.DrError):
        B.PromptAttention(1, 6, 4, 3, 64, device="cpu")
    with pytest.raises(B.DrError):
        B.LinearAttention(1, 6, 4, 48, 64, device="cpu")
    x = B.LinearAttention(1, 6, 4, 64, 64, device="cpu")
    x._index, x._current, x._raw = -1, lambda: -1, lambda _: 0
    g = torch.zeros(4)
    with pytest.raises(ValueError, match="cu"):
        x.forward(q, q, q, g, cu=cu)
    for bad in (None, g.double(), torch.zeros(3)):
        with pytest.raises(ValueError, match="g"):
            x.step(q, q, q, bad, torch.zeros(1, 4, 64, 64))
    with pytest.raises(ValueError, match="state"):
        x.step(q, q, q, g, None)
    with pytest.raises(ValueError, match="state"):
        x.step(q, q, q, g, torch.zeros(1, 4, 64, 32))
