"""GPU parity of the attention over the paged 8-bit cache at the ends of the range of fp32: value scales,
gaps between scores, and scores that are infinite.  The bounds are those of tests/test_cache_attn.py and, for
outputs below the smallest normal number 2^-126, the spacing there: half of 2^-133 for a bf16 output and half of
2^-149 for each of the two last operations (a division and a power of two)."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding

from test_cache_attn import Case

pytestmark = pytest.mark.gpu

KINDS = [  # lens, T, Hq, H, d, page, code, io, out
    ([200, 37], 1, 8, 2, 128, 16, "i8", "bf16", "bf16"),
    ([300], 3, 8, 1, 64, 64, "e4m3", "bf16", "bf16"),      # 24 rows
    ([150, 64], 2, 4, 2, 128, 32, "e4m3", "f32", "f32"),
    ([99], 2, 4, 1, 64, 16, "i8", "bf16", "f32"),
    ([200, 37], 70, 8, 2, 128, 16, "i8", "bf16", "bf16"),  # on the tensor cores
    ([130], 40, 4, 2, 64, 128, "e4m3", "bf16", "bf16"),
]
LAST = {"bf16": 2.0 ** -134 + 2.0 ** -149, "f32": 2.0 ** -149}


def check(c, o, lse):
    assert c.cache.status() == binding.DR_OK
    ro, rl, mag, top, floor = c.oracle()
    prec = c.io == "f32" or c.out == "f32"
    weights = (2.0 ** -20 if prec else 2.0 ** -11) + 2 * 2.0 ** -20 * (1 + top[..., None])
    bound = weights * mag + 2.0 ** -37 * floor + (2.0 ** -8 if c.out == "bf16" else 2.0 ** -24) * np.abs(ro) + LAST[c.out]
    err = np.abs(o.double().cpu().numpy() - ro)
    assert np.isfinite(err).all()
    assert (err <= bound).all(), f"o: worst {(err / bound).max():.2f} of its bound"
    el = np.abs(lse.double().cpu().numpy() - rl)
    assert (el <= 2.0 ** -20 * (2 + top + np.abs(rl))).all(), f"lse: {el.max()}"


def set_scales(c, i, scale):
    """Scales of the keys (i = 0) or values (i = 1)."""
    c.scale[i] = np.asarray(scale, np.float32)
    (c.cache.k_scale, c.cache.v_scale)[i].copy_(torch.from_numpy(c.scale[i]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", [-100, -110, -118, -126, -136, None])
def test_value_scales_down_to_the_smallest_numbers(kind, power):
    """All value scales near 2^power, or (None) each page and head with a power of its own from -140 to -90."""
    c = Case(*kind, seed=41)
    p = np.random.default_rng(0).integers(-140, -90, c.scale[1].shape) if power is None else power
    set_scales(c, 1, c.scale[1] * np.exp2(np.asarray(p, np.float64)))
    o, lse = c.run()
    check(c, o, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gap", [30, 60, 80, 85, 95, 200])
@pytest.mark.parametrize("order", ["first", "last", "middle"])
def test_pages_without_values_that_hold_the_top_score(kind, gap, order):
    """The scores of one page exceed the others by gap to 2 gap, its values are all zero (scale 0); the
    others' value scales are 4 to 10^4.  So the result is that of the others, e^-gap of their size."""
    c = Case(*kind, seed=42)
    page = c.cache.desc.page
    rng = np.random.default_rng(1)
    # a query's channel 0 alone, and the keys' codes there, make the score: top 0, others -gap .. -2 gap
    c.q.zero_()
    c.q[..., 0] = 1
    c.softmax_scale = gap / 32.0
    set_scales(c, 0, np.ones_like(c.scale[0]))
    set_scales(c, 1, rng.uniform(4, 1e4, c.scale[1].shape))
    codes, vs = c.codes[0], c.scale[1].copy()
    if c.code == "i8":
        codes[..., 0] = (-rng.integers(32, 64, codes.shape[:-1])).astype(np.int8).view(np.uint8)
    else:  # e4m3: -32 .. -60
        codes[..., 0] = 0xe0 + rng.integers(0, 8, codes.shape[:-1])
    for b in range(c.B):
        pages = -(-int(c.lens[b] + c.n[b]) // page)
        at = c.table[b, {"first": 0, "last": (int(c.lens[b])) // page, "middle": pages // 2}[order]]
        codes[at, ..., 0] = 0
        vs[at] = 0
    set_scales(c, 1, vs)
    kind_of = torch.int8 if c.code == "i8" else torch.float8_e4m3fn
    c.cache.k.view(torch.int8).copy_(torch.from_numpy(codes.view(np.int8)))
    assert c.cache.k.dtype == kind_of
    check(c, *c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_a_row_whose_every_score_is_minus_infinity_is_not_a_number(kind):
    """e^-inf / e^-inf: an infinite query is no row without positions, and must not come out as zeros."""
    c = Case(*kind, seed=43)
    codes = c.codes[0]
    codes[..., 0] = 0xff if c.code == "i8" else 0xb8  # -1
    c.cache.k.view(torch.int8).copy_(torch.from_numpy(codes.view(np.int8)))
    good, lse = c.run()
    q = c.q.clone()
    q[0, 0, 1, 0] = float("inf")
    o, b = c.run(q)
    assert o[0, 0, 1].isnan().all() and b[0, 0, 1].isneginf()
    o[0, 0, 1], b[0, 0, 1] = good[0, 0, 1], lse[0, 0, 1]
    assert torch.equal(o, good) and torch.equal(b, lse)
