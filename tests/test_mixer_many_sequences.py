"""Host-side: how many packed sequences a call may have (no GPU: nothing is launched)."""
import ctypes

import pytest

from delta_rule_recurrent_gated_gb300 import binding as B

PTR = 0x10000  # a 16-byte aligned address that no call may touch
MOST = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from delta_rule_recurrent_gated_gb300 import build
    build.build()
    return B.load()


def prompt(seqs, T=4096):
    return B.DrPromptDesc(1, T, 4, 2, 128, seqs, B.DR_BF16, 0, 0.1, 512, 256, 256, 512, 256, 256)


def linear(seqs, T=4096):
    return B.DrLinearDesc(1, T, 4, 64, 128, seqs, B.DR_F32, 0.1, 256, 256, 512, 256, 256, 512)


@pytest.mark.parametrize("seqs", [MOST + 1, 1 << 27, 2 ** 31 - 1])
def test_more_packed_sequences_are_refused(lib, seqs):
    """A block walks over the offsets to find its tile: it has to be through within the limit of its waits, and
    the walk's counters within their 32 bits."""
    r = ctypes.byref
    d, e = prompt(seqs), linear(seqs)
    assert lib.dr_prompt_attn_workspace_bytes(r(d)) == lib.dr_linear_attn_workspace_bytes(r(e)) == 0
    assert lib.dr_prompt_attn_fwd(r(d), *[PTR] * 3, PTR, PTR, PTR + 8, None) == B.DR_ERR_UNSUPPORTED  # nor the address
    assert lib.dr_prompt_attn_bwd(r(d), *[PTR] * 6, PTR, *[PTR] * 3, PTR + 8, 1 << 40, None) == B.DR_ERR_UNSUPPORTED
    assert lib.dr_linear_attn_fwd(r(e), *[PTR] * 5, PTR, PTR, PTR, PTR + 8, 1 << 40, None) == B.DR_ERR_UNSUPPORTED
    assert lib.dr_linear_attn_bwd(r(e), *[PTR] * 7, PTR, *[PTR] * 4, PTR + 8, 1 << 40, None) == B.DR_ERR_UNSUPPORTED


def test_as_many_and_dense_batches_are_taken(lib):
    r = ctypes.byref
    assert lib.dr_prompt_attn_workspace_bytes(r(prompt(MOST))) > 0
    assert lib.dr_linear_attn_workspace_bytes(r(linear(MOST))) > 0
    d, e = prompt(4 * MOST, 2), linear(4 * MOST, 2)  # a dense batch has no offsets to walk over
    d.B = e.B = 4 * MOST
    assert lib.dr_prompt_attn_workspace_bytes(r(d)) > 0 and lib.dr_linear_attn_workspace_bytes(r(e)) > 0
    with pytest.raises(B.DrError):
        B.PromptAttention(1, 64, 4, 2, 64, seqs=MOST + 1, device="cpu")
