"""fp32 linear attention on rows far behind the start of large tensors, more than 2^31 values in."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from mixers import ULP, check, np64
from oracle import mixers as M
import numpy as np

pytestmark = pytest.mark.gpu

ROWS, USED = 1_060_000, 331  # of 16 heads of 128: 2.17e9 values


def far(small):
    """A tensor of ROWS rows whose last ones are those of `small` [1, USED, ...]."""
    t = torch.empty(1, ROWS, *small.shape[2:], dtype=small.dtype, device="cuda")
    t[:, -USED:] = small
    return t


def test_linear_attention():
    """The last two sequences of such tensors against the fp64 restatement, with the bounds of mixers.py (the number of
    rows decides where sequences are split, so the bits may differ from those of small tensors)."""
    g = torch.Generator().manual_seed(1)
    q, k, v, dO = (torch.randn(1, USED, 16, 128, generator=g).cuda() for _ in range(4))
    h0 = torch.randn(2, 16, 128, 128, generator=g).cuda()
    rates = -0.02 * torch.arange(1, 17).float().cuda()
    plan = binding.LinearAttention(1, ROWS, 16, 128, 128, seqs=2, io="f32", scale=0.1)
    cu = torch.tensor([ROWS - USED, ROWS - 100, ROWS], dtype=torch.int32).cuda()
    x = [far(t) for t in (q, k, v)]
    o, hT = plan.forward(*x, rates, h0=h0, cu=cu)
    got = dict(o=o, hT=hT, **plan.backward(*x, rates, far(dO), h0=h0, dhT=h0, cu=cu))
    spans = [(0, USED - 100), (USED - 100, USED)]
    ref, size = M.linear(*(np64(t[0]) for t in (q, k, v)), np64(rates), spans, 0.1, np64(h0), np64(dO[0]), np64(h0))
    fine = 2.0 ** -16 + (USED + 128) * 2.0 ** -24
    for n, t in got.items():
        if n in ("hT", "dh0"):
            check(np64(t), ref[n], fine * size[n], n)
        else:
            check(np64(t[0, -USED:]), ref[n], fine * size[n] + ULP["f32"] * np.abs(ref[n]), n)
