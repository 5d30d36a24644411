"""GPU parity of the attention over the paged 8-bit cache against the fp64 restatement
(oracle/attention.py) on the same codes and scales.

Bounds, fixed before the first run, with A = sum_j softmax_j |v_j| and S = max_j scale sum_c |q_c k_jc|:
  weights rounded to 11 bits: 2^-11 A (fp32 types: 2^-20 A), and to no less than half the spacing
  2^-24 of the smallest 16-bit operands: an operand is the weight over its row's largest (within a
  factor of 4) times 2^14, so 2^-37 (largest weight with its value scale) sum_j |code_j|;
  an error e in a score changes the result by at most 2 e A: scores are fp32 sums of 128 products and
  a few fp32 products more, e = 2^-20 (1 + S);
  half a unit of the output type: 2^-8 |o| (bf16), 2^-24 |o|.
lse: 2^-20 (1 + S) + 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from oracle import attention as A

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Case:
    def __init__(self, lens, T, Hq, H, d, page, code, io, out, window=0, counts=None, seed=0, spread=1.0,
                 junk=True):
        rng = np.random.default_rng(seed)
        self.B, self.T, self.Hq, self.H, self.d, self.code, self.window = len(lens), T, Hq, H, d, code, window
        self.lens = np.array(lens, np.int32)
        self.counts = None if counts is None else np.array(counts, np.int32)
        n = self.n = np.array(counts if counts is not None else [T] * self.B)
        per = max(1, -(-int((self.lens + n).max()) // page))
        P = self.B * per + 2
        # table entries behind a sequence's last page are never read: out of range here
        self.table = rng.permutation(P)[:self.B * per].reshape(self.B, per).astype(np.int32)
        for b in range(self.B):
            self.table[b, -(-int(self.lens[b] + n[b]) // page):] = 1 << 30
        top = 0x7f if code == "e4m3" else 256
        self.codes = [rng.integers(0, top, (P, H, page, d)).astype(np.uint8) for _ in range(2)]
        if code == "e4m3":
            for c in self.codes:
                c |= (rng.integers(0, 2, c.shape) << 7).astype(np.uint8)
        else:
            for c in self.codes:
                c[c == 128] = 0
        unit = 1 / 64.0 if code == "i8" else 1 / 128.0
        self.scale = [(unit * np.exp(spread * rng.standard_normal((P, H)))).astype(np.float32) for _ in range(2)]
        if junk:  # behind the last position: codes that are no numbers
            for b in range(self.B):
                e = int(self.lens[b] + n[b])
                if e % page:
                    for c in self.codes:
                        c[self.table[b, e // page], :, e % page:] = 0x7f
        self.io, self.out = io, out
        # 1 / sqrt(d) of unit scores for unit queries: a lively softmax
        self.q = torch.from_numpy(rng.standard_normal((self.B, T, Hq, d))).to(TYPES[io]).cuda()
        self.softmax_scale = d ** -0.5
        kind = torch.int8 if code == "i8" else torch.float8_e4m3fn
        self.cache = binding.KvCache(P, H, d, page=page, code=code, buffers=[
            *(torch.from_numpy(c).cuda().view(kind) for c in self.codes),
            *(torch.from_numpy(s).cuda() for s in self.scale)])

    def run(self, q=None, want_lse=True):
        p = binding.CacheAttention(self.cache, self.B, self.T, self.Hq, io=self.io, out=self.out,
                                   scale=self.softmax_scale, window=self.window)
        p.ws.fill_(0xff)  # whatever a workspace held
        return p.forward(self.q if q is None else q, up(self.table), up(self.lens),
                         None if self.counts is None else up(self.counts), want_lse=want_lse)

    def oracle(self):
        return A.attention(self.q.double().cpu().numpy(), self.codes[0], self.scale[0], self.codes[1],
                           self.scale[1], self.table, self.lens, self.n, self.code, self.softmax_scale,
                           self.window)

    def check(self, o, lse):
        assert self.cache.status() == binding.DR_OK
        ro, rl, mag, top, floor = self.oracle()
        prec = self.io == "f32" or self.out == "f32"
        weights = (2.0 ** -20 if prec else 2.0 ** -11) + 2 * 2.0 ** -20 * (1 + top[..., None])
        bound = weights * mag + 2.0 ** -37 * floor + (2.0 ** -8 if self.out == "bf16" else 2.0 ** -24) * np.abs(ro)
        err = np.abs(o.double().cpu().numpy() - ro)
        assert np.isfinite(err).all()
        assert (err <= bound).all(), f"o: worst {(err / np.maximum(bound, 1e-30)).max():.2f} of its bound"
        gl = lse.double().cpu().numpy()
        none = np.isneginf(rl)
        assert (np.isneginf(gl) == none).all()
        el = np.abs(gl[~none] - rl[~none])
        assert (el <= 2.0 ** -20 * (2 + top[~none] + np.abs(rl[~none]))).all(), f"lse: {el.max()}"
        assert (o[torch.from_numpy(none).cuda()] == 0).all()


SHAPES = [  # lens, T, Hq, H, d, page, window
    ([0], 1, 1, 1, 64, 16, 0),
    ([0, 1, 15, 16, 17], 1, 4, 4, 64, 16, 0),
    ([63, 64, 65, 127, 0], 1, 16, 4, 128, 64, 0),
    ([1000], 1, 16, 4, 128, 64, 0),
    ([700, 3, 129], 1, 8, 8, 128, 128, 0),
    ([500, 31], 1, 20, 2, 64, 32, 0),       # ten query heads of each cache head: two row groups
    ([333], 1, 17, 1, 128, 16, 0),          # 17 rows
    ([90, 0, 250], 5, 8, 8, 64, 16, 0),
    ([64, 7], 6, 12, 4, 128, 64, 0),        # 18 rows that begin inside a token
    ([300, 100], 1, 16, 4, 128, 64, 1),     # a window of the token itself
    ([300, 100, 5], 3, 8, 4, 64, 32, 40),   # windows that begin inside a page
    ([300, 130], 40, 8, 2, 128, 64, 64),    # windows that leave pages unseen by a part of the rows
    ([0, 33], 70, 8, 4, 128, 64, 0),        # a prompt
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_parity(shape, code, io, out):
    lens, T, Hq, H, d, page, window = shape
    c = Case(lens, T, Hq, H, d, page, code, io, out, window=window)
    c.check(*c.run())


@pytest.mark.parametrize("T,counts", [(4, [0, 1, 4, 2, 0]), (1, [0, 0, 1, 0, 1]), (40, [40, 0, 17, 1, 39])])
def test_sequences_with_fewer_tokens(T, counts):
    c = Case([10, 200, 0, 64, 333], T, 8, 2, 128, 64, "e4m3", "bf16", "bf16", counts=counts, seed=1)
    c.check(*c.run())
    assert all(t is None or t.shape[0] == 5 for t in c.run(want_lse=False))


def test_all_sequences_idle():
    c = Case([10, 20], 2, 8, 2, 64, 16, "i8", "bf16", "bf16", counts=[0, 0])
    o, lse = c.run()
    assert (o == 0).all() and torch.isneginf(lse).all() and c.cache.status() == binding.DR_OK


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_a_long_axis_over_every_block(code):
    """A single sequence that all blocks share, beside many short ones."""
    c = Case([40003], 1, 4, 2, 64, 64, code, "f32", "f32", seed=2)
    c.check(*c.run())
    c = Case([20000] + list(range(70)), 1, 4, 2, 64, 16, code, "bf16", "bf16", seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_scales_far_apart(out):
    """Value and key scales over twelve orders of magnitude: no weight may be lost to them."""
    c = Case([900, 77], 2, 8, 2, 128, 16, "i8", "bf16", out, seed=4, spread=1.0)
    c.scale[1][:] = (c.scale[1] * 10.0 ** np.random.default_rng(0).uniform(-6, 6, c.scale[1].shape)).astype(np.float32)
    c.scale[1][::5] = 0
    c.cache.v_scale.copy_(torch.from_numpy(c.scale[1]))
    c.check(*c.run())
    c.scale[1][:] = 0
    c.cache.v_scale.zero_()
    c.check(*c.run())


def test_queries_of_any_size():
    c = Case([130, 40], 1, 8, 4, 64, 16, "i8", "bf16", "bf16", seed=5)
    q = c.q
    q[0, 0, 0] = 0                      # a uniform softmax
    q[0, 0, 1] *= 1e30
    c.softmax_scale = 1e-30
    q[0, 0, 2:] *= 1e29
    q[1] *= 1e-30
    c.check(*c.run())


def test_scores_far_apart():
    """One position that takes all the weight, and scores of several hundred."""
    c = Case([600], 1, 8, 2, 128, 64, "i8", "bf16", "bf16", seed=6)
    c.softmax_scale = 20.0
    c.check(*c.run())


def test_marked_pages_reach_only_the_rows_that_see_them():
    for code in ("i8", "e4m3"):
        c = Case([200, 100], 4, 8, 2, 64, 16, code, "bf16", "bf16", window=50, seed=7)
        o, lse = c.run()
        c.check(o, lse)
        for i in (0, 1):
            s = (c.cache.k_scale, c.cache.v_scale)[i]
            keep = s.clone()
            # sequence 0: tokens 200 .. 203 see positions 151 .. 203; page 9 holds 144 .. 159
            s[int(c.table[0, 9]), 1] = float("nan")
            a, b = c.run()
            assert a[0, :, 4:].isnan().all() and b[0, :, 4:].isnan().all() == (i == 0)
            assert torch.equal(a[0, :, :4], o[0, :, :4]) and torch.equal(a[1], o[1])
            s.copy_(keep)
            s[int(c.table[0, 8])] = float("nan")  # 128 .. 143: seen by nobody
            a, b = c.run()
            assert torch.equal(a, o) and torch.equal(b, lse)
            s.copy_(keep)
            # page 9 of sequence 1 (its tokens are 100 .. 103) lies behind its end
    # the first rows of a tile see a page that the later ones do not
    c = Case([64], 8, 1, 1, 64, 16, "i8", "bf16", "bf16", window=50, seed=8)
    o, _ = c.run()
    c.cache.v_scale[int(c.table[0, 0])] = float("nan")  # positions 0 .. 15, seen while p - 50 < 15
    a, _ = c.run()
    assert a[0, 0].isnan().all() and torch.equal(a[0, 1:], o[0, 1:])


def test_a_query_that_is_not_finite_stays_in_its_row():
    c = Case([100], 3, 8, 2, 64, 16, "i8", "bf16", "bf16", seed=9)
    o, _ = c.run()
    q = c.q.clone()
    q[0, 1, 3, 7] = float("nan")
    a, _ = c.run(q)
    assert a[0, 1, 3].isnan().all() and a.isnan().sum() == 64
    keep = ~a.isnan()
    assert torch.equal(a[keep], o[keep])


def test_packed_queries_other_streams_and_repeats():
    c = Case([300, 77, 0], 2, 8, 2, 128, 64, "i8", "bf16", "bf16", seed=10)
    o, lse = c.run()
    big = torch.randn(3, 2, 12, 128, device="cuda").bfloat16()
    big[:, :, :8] = c.q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = c.run(big[:, :, :8])
    side.synchronize()
    assert torch.equal(a, o) and torch.equal(b, lse)


def test_out_of_range_is_recorded_and_marked():
    base = dict(T=2, Hq=4, H=2, d=64, page=16, code="i8", io="bf16", out="bf16")
    good = Case([40, 30], **base)
    o, lse = good.run()
    for what in ("page", "negative page", "negative length", "past the table"):
        c = Case([40, 30], **base)
        if what == "page":
            c.table[0, 1] = 10 ** 6
        elif what == "negative page":
            c.table[0, 2] = -3
        elif what == "negative length":
            c.lens[0] = -5
        else:
            c.lens[0] = 47
        a, b = c.run()
        assert c.cache.status() == binding.DR_ERR_INDEX
        assert a[0].isnan().all() and b[0].isnan().all()
        assert torch.equal(a[1], o[1]) and torch.equal(b[1], lse[1])
    c = Case([40, 30], counts=[2, 2], **base)
    c.counts[0] = 3
    a, _ = c.run()
    assert c.cache.status() == binding.DR_ERR_INDEX and a[0].isnan().all() and torch.equal(a[1], o[1])


def test_written_then_read_by_the_attention():
    """Tokens appended one call after another; at each step the attention over the cache equals the
    softmax over the values that were written, to the size of a code's step."""
    H, d, page, B = 2, 64, 16, 2
    g = torch.Generator().manual_seed(0)
    cache = binding.KvCache(20, H, d, page=page, code="i8")
    table = torch.randperm(20, generator=g)[:2 * 8].reshape(2, 8).int().cuda()
    ks, vs = [], []
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for T in (30, 1, 1, 7):
        k, v, q = (torch.randn(B, T, n, d, generator=g).cuda() for n in (H, H, 4))
        cache.write(k, v, table, lens)
        ks.append(k), vs.append(v)
        o, _ = binding.CacheAttention(cache, B, T, 4, io="f32", out="f32").forward(q, table, lens)
        K, V = torch.cat(ks, 1).double(), torch.cat(vs, 1).double()
        s = torch.einsum("bthgd,bjhd->bhgtj", q.double().view(B, T, H, 2, d), K) / 8
        j = torch.arange(K.shape[1], device="cuda")
        s = s.masked_fill(j > j[-T:, None], float("-inf"))
        ref = torch.einsum("bhgtj,bjhd->bthgd", s.softmax(-1), V).reshape(B, T, 4, d)
        # codes are within one step (a page's scale may have grown once) = max|x| / 127 of k and of v:
        # e^(score error) with score error <= 8 * 4 / 127 in the worst case, 0.1 in practice
        assert (o.double() - ref).abs().max() < 0.1
        lens += T
    assert cache.status() == binding.DR_OK


def test_a_pool_whose_offsets_pass_32_bits():
    """Pages behind the first 4 GiB of a pool: 36,000 pages of 8 heads x 128 x 128 bytes."""
    P, H, page, d = 36000, 8, 128, 128
    codes = [torch.zeros(P, H, page, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.full((P, H), 1 / 64, device="cuda") for _ in range(2)]
    cache = binding.KvCache(P, H, d, page=page, code="i8", buffers=[*codes, *scale])
    small = Case([200, 300], 1, 16, H, d, page, "i8", "bf16", "bf16", seed=11)
    table = small.table.copy()
    for b in range(2):
        for i in range(-(-int(small.lens[b] + 1) // page)):
            at = P - 1 - (b * 8 + i)
            for j in range(2):
                codes[j][at] = torch.from_numpy(small.codes[j][table[b, i]]).cuda().view(torch.int8)
                scale[j][at] = torch.from_numpy(small.scale[j][table[b, i]]).cuda()
            table[b, i] = at
    o, lse = small.run()
    p = binding.CacheAttention(cache, 2, 1, 16, scale=small.softmax_scale)
    a, b = p.forward(small.q, up(table), up(small.lens), want_lse=True)
    assert cache.status() == binding.DR_OK and torch.equal(a, o) and torch.equal(b, lse)
    x = torch.ones(2, 1, H, d, device="cuda")
    cache.write(x, x, up(table), up(small.lens))
    k, _ = cache.read(up(table), up(small.lens), None, 1, out="f32")
    assert ((k - 1).abs() <= scale[0].max() * 0.5 + 0.01).all() and cache.status() == binding.DR_OK


def test_arguments_are_refused_before_a_launch():
    c = Case([10], 1, 8, 2, 64, 16, "i8", "bf16", "bf16")
    p = binding.CacheAttention(c.cache, 1, 1, 8)
    with pytest.raises(ValueError):
        p.forward(c.q.float(), up(c.table), up(c.lens))
    with pytest.raises(ValueError):
        p.forward(c.q[:, :, :4], up(c.table), up(c.lens))
    with pytest.raises(ValueError):
        p.forward(c.q, up(c.table), up([1, 2]))
    with pytest.raises(binding.DrError):
        binding.CacheAttention(c.cache, 1, 1, 7)
