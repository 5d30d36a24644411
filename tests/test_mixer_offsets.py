"""Rows far behind the start of large tensors, more than 2^31 values in: the same bits as in small ones."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding

pytestmark = pytest.mark.gpu

ROWS, USED = 1_060_000, 331  # of 16 heads of 128: 2.17e9 values


def far(small):
    """A tensor of ROWS rows whose last ones are those of `small` [1, USED, ...]."""
    t = torch.empty(1, ROWS, *small.shape[2:], dtype=small.dtype, device="cuda")
    t[:, -USED:] = small
    return t


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention(io):
    kind = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator().manual_seed(0)
    q, dO = (torch.randn(1, USED, 16, 128, generator=g).to(kind).cuda() for _ in range(2))
    k, v = (torch.randn(1, USED, 2, 128, generator=g).to(kind).cuda() for _ in range(2))
    results = []
    for rows, place in ((USED, lambda t: t), (ROWS, far)):
        plan = binding.PromptAttention(1, rows, 16, 2, 128, seqs=2, io=io)
        cu = torch.tensor([rows - USED, rows - 100, rows], dtype=torch.int32).cuda()
        x = [place(t) for t in (q, k, v)]
        o, lse = plan.forward(*x, cu=cu, want_lse=True)
        grads = plan.backward(*x, o, lse, place(dO), cu=cu)
        results.append([t[:, -USED:].clone() for t in (o, lse, *grads.values())])
    if io == "bf16":
        assert all(torch.equal(a, b) for a, b in zip(*results))
    else:
        # Shared key heads are summed in a block or after it, as the number of rows has it: up to 8 x 331 terms
        # in another order. Independent roundings of 2^-24 add up to sqrt(2648) x 2^-24 = 2^-18.3 of the partial
        # sums; the bound leaves a factor of four for partial sums larger than the largest result.
        assert all(torch.allclose(a, b, rtol=2 ** -16, atol=2 ** -16 * float(a.abs().max())) for a, b in zip(*results))


def test_linear_attention():
    g = torch.Generator().manual_seed(1)
    q, k, v, dO = (torch.randn(1, USED, 16, 128, generator=g).bfloat16().cuda() for _ in range(4))
    h0 = torch.randn(2, 16, 128, 128, generator=g).cuda()
    rates = -0.02 * torch.arange(1, 17).float().cuda()
    results = []
    for rows, place in ((USED, lambda t: t), (ROWS, far)):
        plan = binding.LinearAttention(1, rows, 16, 128, 128, seqs=2)
        cu = torch.tensor([rows - USED, rows - 100, rows], dtype=torch.int32).cuda()
        x = [place(t) for t in (q, k, v)]
        o, hT = plan.forward(*x, rates, h0=h0, cu=cu)
        grads = plan.backward(*x, rates, place(dO), h0=h0, dhT=h0, cu=cu)
        results.append([hT, grads.pop("dh0"), *(t[:, -USED:].clone() for t in (o, *grads.values()))])
    assert all(torch.equal(a, b) for a, b in zip(*results))
