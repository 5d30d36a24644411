"""Host-side: a descriptor of linear attention that only the forward pass uses (no GPU: nothing is launched)."""
import ctypes

import pytest

from delta_rule_recurrent_gated_gb300 import binding as B

PTR = 0x10000  # a 16-byte aligned address that no call may touch


@pytest.fixture(scope="module")
def lib():
    from delta_rule_recurrent_gated_gb300 import build
    build.build()
    return B.load()


@pytest.mark.parametrize("io", [B.DR_BF16, B.DR_F32])
@pytest.mark.parametrize("batch,tokens", [(2, 3), (1, 16411)])  # the second one is split into segments
def test_workspace_of_a_forward_call(lib, io, batch, tokens):
    """The gradients' row distances are the backward call's: a forward caller may leave them zero."""
    d = B.DrLinearDesc(batch, tokens, 4, 64, 128, batch, io, 0.1, 256, 256, 512, 256, 256, 512)
    both = lib.dr_linear_attn_workspace_bytes(ctypes.byref(d))
    d.ld_dq = d.ld_dk = d.ld_dv = 0
    assert both > 0 and lib.dr_linear_attn_workspace_bytes(ctypes.byref(d)) == both
    # the size that it names is the size that the call asks for
    assert lib.dr_linear_attn_fwd(ctypes.byref(d), *[PTR] * 5, None, PTR, PTR, PTR, both - 1, None) == B.DR_ERR_WORKSPACE
    # the gradient still wants them
    assert lib.dr_linear_attn_bwd(ctypes.byref(d), *[PTR] * 7, None, *[PTR] * 5, 1 << 40, None) == B.DR_ERR_INVALID_ARG
