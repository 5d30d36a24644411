"""What the tests of PromptAttention and LinearAttention share: inputs in the layouts that the calls take, and
the comparison with the fp64 restatement (oracle/mixers.py).

Bounds, fixed before the first run, relative to the sums of the terms' sizes that the restatement returns.
Rounding to bf16 is off by at most 2^-8 of the value (fp32: 2^-24), `ULP`.
fp32 work.  A score is a sum of d <= 128 products: off by at most 2^-17 of the sum of their sizes, `top`, and the
  weight that is its power by as much relatively, twice (the row's sum too).  Sums over n tokens add n 2^-24 at most:
  fine = 2^-16 (1 + top) + n 2^-24.  Decays and their products over the chunks: 2^-17 and n 2^-24.
bf16 operands.  o and dv: softmax weights (decayed scores, the state) once, 2^-8.  dq and dk of softmax attention: ds
  once, and D = dO.o from an o that was rounded and whose weights were: 3 times 2^-8.  States: decayed keys (queries)
  in two bf16 parts, 2^-16.
Weights below 2^-126, the smallest normal number, may be taken as none (the power flushes them): an error of up to
  n |dO| |V| |Q| 2^-126 with fewer than 2^11 tokens and factors (rows of 128 values below 32) of 2^25 in all, `FLUSH`;
  the sizes hold such weights too, so without it a result made of them alone has no bound to meet.
"""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ULP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
OPERAND = {"bf16": 2.0 ** -8, "f32": 0.0}
SPLIT = {"bf16": 2.0 ** -16, "f32": 0.0}
FLUSH = 2.0 ** -90


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Layout:
    """Sequences of the given lengths: packed rows with `rest` more behind the last, or dense."""

    def __init__(self, lens, packed, rest=0):
        assert packed or len(set(lens)) == 1
        self.lens, self.packed = list(lens), packed
        at = np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.spans = [(int(a), int(b)) for a, b in zip(at, at[1:])]
        self.used = int(at[-1])
        self.B, self.T = (1, self.used + rest) if packed else (len(lens), lens[0])
        self.seqs = len(lens) if packed else None
        self.cu = torch.tensor(at, dtype=torch.int32).cuda() if packed else None

    def rows(self, t):
        """A tensor [B, T, ...] as rows of used tokens, numpy fp64."""
        return np64(t).reshape(self.B * self.T, *t.shape[2:])[:self.used]


def tensors(lay, heads, dims, io, seed, inside=False, spread=1.0):
    """q, k, v ... [B, T, heads[i], dims[i]]: their own tensors, or (inside) ranges of one wider tensor with more
    columns around them."""
    g = torch.Generator().manual_seed(seed)
    parts = [(spread * torch.randn(lay.B, lay.T, h, d, generator=g)).to(TYPES[io]) for h, d in zip(heads, dims)]
    if not inside:
        return [x.cuda() for x in parts]
    pad = torch.full((lay.B, lay.T, 16), float("nan"), dtype=TYPES[io])
    wide = torch.cat([y for x in parts for y in (pad, x.flatten(2))] + [pad], 2).cuda()
    out, at = [], 0
    for h, d in zip(heads, dims):
        at += 16
        out.append(wide[:, :, at:at + h * d].unflatten(2, (h, d)))
        at += h * d
    return out


def check(got, ref, bound, what):
    assert got.shape == ref.shape, what
    err = np.abs(got - ref)
    assert np.isfinite(err).all(), what
    assert (err <= bound + FLUSH).all(), f"{what}: error {err.max():.3e}, up to {np.max(err / np.maximum(bound, 1e-300)):.3g} of its bound"
