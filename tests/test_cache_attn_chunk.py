"""GPU parity of the attention over the paged 8-bit cache where a sequence and cache head have many
rows (query tokens times query heads): tiles of 128 rows on the tensor cores.  Bounds: those of
tests/test_cache_attn.py, whose helper this uses."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding

from test_cache_attn import Case

pytestmark = pytest.mark.gpu

SHAPES = [  # lens, T, Hq, H, d, page, window, counts
    ([0], 128, 1, 1, 64, 16, 0, None),
    ([0, 0], 129, 4, 4, 128, 128, 0, None),            # a second tile of one row
    ([5], 64, 2, 2, 128, 32, 0, None),                 # half a tile
    ([300, 63, 64], 100, 8, 2, 128, 64, 0, None),      # tiles that begin inside a sequence's tokens
    ([77], 50, 5, 1, 64, 16, 0, None),                 # five heads to a cache head: tokens across tiles
    ([200, 0], 33, 128, 2, 64, 32, 0, None),           # 64 heads to a cache head
    ([700], 90, 4, 2, 128, 16, 100, None),             # windows: tiles that see the end only
    ([500, 20], 130, 2, 1, 64, 64, 1, None),
    ([400, 90, 0, 7], 96, 4, 2, 128, 64, 0, [96, 0, 1, 50]),
    ([1500, 2, 900], 70, 4, 1, 128, 128, 333, [70, 70, 3]),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_parity(shape, code):
    lens, T, Hq, H, d, page, window, counts = shape
    c = Case(lens, T, Hq, H, d, page, code, "bf16", "bf16", window=window, counts=counts, seed=21)
    c.check(*c.run())


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_even_scales_and_unit_queries(code):
    """What a trained model's cache looks like: many positions share the weight."""
    c = Case([900, 333], 64, 8, 2, 128, 64, code, "bf16", "bf16", seed=22, spread=0.1)
    for i in (0, 1):
        c.scale[i] *= 0.05
    c.cache.k_scale.mul_(0.05), c.cache.v_scale.mul_(0.05)
    c.check(*c.run())


def test_tiles_shared_by_blocks():
    """Few tiles over a long axis: each is joined from many blocks' parts; and many tiles."""
    c = Case([9000], 64, 2, 2, 64, 64, "i8", "bf16", "bf16", seed=23)
    c.check(*c.run())
    c = Case([0, 10, 500] * 4, 64, 16, 16, 64, 64, "e4m3", "bf16", "bf16", seed=24)
    c.check(*c.run())


def test_scales_far_apart():
    c = Case([900, 77], 70, 8, 2, 128, 16, "i8", "bf16", "bf16", seed=25)
    c.scale[1][:] = (c.scale[1] * 10.0 ** np.random.default_rng(0).uniform(-6, 6, c.scale[1].shape)).astype(np.float32)
    c.scale[1][::5] = 0
    c.cache.v_scale.copy_(torch.from_numpy(c.scale[1]))
    c.check(*c.run())
    c.scale[1][:] = 0
    c.cache.v_scale.zero_()
    c.check(*c.run())


def test_queries_of_any_size():
    c = Case([130], 64, 8, 4, 64, 16, "e4m3", "bf16", "bf16", seed=26)
    c.q[0, 0, 0] = 0
    c.q[0, :32] *= 1e30
    c.q[0, 32:] *= 1e-30
    c.softmax_scale = 1e-30
    c.check(*c.run())


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_marked_pages_reach_only_the_rows_that_see_them(code):
    c = Case([200, 100], 64, 4, 2, 64, 16, code, "bf16", "bf16", window=50, seed=27)
    o, lse = c.run()
    c.check(o, lse)
    for i in (0, 1):
        s = (c.cache.k_scale, c.cache.v_scale)[i]
        keep = s.clone()
        s[int(c.table[0, 14]), 1] = float("nan")  # positions 224 .. 239 of sequence 0, head 1
        a, b = c.run()
        # query t is position 200 + t and sees 151 + t .. 200 + t
        sees = torch.tensor([t + 200 >= 224 and t + 151 <= 239 for t in range(64)], device="cuda")
        assert a[0, sees][:, 2:].isnan().all()
        assert torch.equal(a[0, ~sees], o[0, ~sees]) and torch.equal(a[0, :, :2], o[0, :, :2])
        assert torch.equal(a[1], o[1])
        s.copy_(keep)


def test_a_query_that_is_not_finite_stays_in_its_row():
    c = Case([100], 80, 4, 2, 64, 16, "i8", "bf16", "bf16", seed=28)
    o, _ = c.run()
    q = c.q.clone()
    q[0, 41, 3, 7] = float("nan")
    a, _ = c.run(q)
    assert a[0, 41, 3].isnan().all() and a.isnan().sum() == 64
    keep = ~a.isnan()
    assert torch.equal(a[keep], o[keep])


def test_packed_queries_other_streams_and_repeats():
    c = Case([300, 77, 0], 70, 8, 2, 128, 64, "i8", "bf16", "bf16", seed=29)
    o, lse = c.run()
    big = torch.randn(3, 70, 12, 128, device="cuda").bfloat16()
    big[:, :, 2:10] = c.q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = c.run(big[:, :, 2:10])
    side.synchronize()
    assert torch.equal(a, o) and torch.equal(b, lse)


def test_out_of_range_is_recorded_and_marked():
    base = dict(T=70, Hq=4, H=2, d=64, page=16, code="i8", io="bf16", out="bf16")
    for what in ("page", "negative length", "past the table", "count"):
        c = Case([40, 30], counts=[70, 70], **base)
        if what == "page":
            c.table[0, 0] = 10 ** 6
        elif what == "negative length":
            c.lens[0] = -5
        elif what == "past the table":
            c.lens[0] = 47
        else:
            c.counts[0] = 71
        a, b = c.run()
        assert c.cache.status() == binding.DR_ERR_INDEX
        assert a[0].isnan().all() and b[0].isnan().all()
        assert a[1].isfinite().all() and b[1].isfinite().all()


def test_the_same_tokens_one_at_a_time():
    """A chunk equals the steps it stands for (the other kernel), to the rounding of both."""
    c = Case([500], 64, 4, 2, 128, 64, "i8", "bf16", "bf16", seed=30)
    o, lse = c.run()
    p = binding.CacheAttention(c.cache, 1, 1, 4, scale=c.softmax_scale)
    table = torch.from_numpy(c.table).cuda()
    for t in (0, 1, 31, 63):
        a, b = p.forward(c.q[:, t:t + 1], table, torch.tensor([500 + t], dtype=torch.int32, device="cuda"),
                         want_lse=True)
        assert (b[:, 0] - lse[:, t]).abs().max() < 2.0 ** -18 * (1 + lse.abs().max())
        assert (a[:, 0].float() - o[:, t].float()).abs().max() <= 2.0 ** -7 * o[:, t].float().abs().max()
