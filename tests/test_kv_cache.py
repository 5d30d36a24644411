"""GPU tests of the paged 8-bit cache against its restatement (oracle/attention.py): codes and
scales bit for bit, values read back to half a unit of the output type."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from oracle import attention as A

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class Pair:
    """A cache on the GPU, its restatement, and a table that shares out the pages at random."""

    def __init__(self, B, positions, H, d, page, code, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        self.B, self.H, self.d, self.page, self.code = B, H, d, page, code
        per = -(-positions // page)
        P = B * per + spare
        self.table = rng.permutation(P)[:B * per].reshape(B, per).astype(np.int32)
        # what pages held before: anything, the codes that are no numbers among it
        self.codes = [rng.integers(0, 256, (P, H, page, d)).astype(np.uint8) for _ in range(2)]
        self.scale = [rng.uniform(0, 5, (P, H)).astype(np.float32) for _ in range(2)]
        kind = torch.int8 if code == "i8" else torch.float8_e4m3fn
        self.gpu = binding.KvCache(P, H, d, page=page, code=code, buffers=[
            *(torch.from_numpy(c.copy()).cuda().view(kind) for c in self.codes),
            *(torch.from_numpy(s.copy()).cuda() for s in self.scale)])
        self.lens = np.zeros(B, np.int32)
        self.rng = rng

    def put(self, k, v, counts):
        """Append on both sides; k, v: torch tensors [B, T, H, d]."""
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.gpu.write(k, v, up(self.table), up(self.lens), None if counts is None else up(counts))
        n = [k.shape[1]] * self.B if counts is None else counts
        for i, x in enumerate((k, v)):
            A.cache_write(self.codes[i], self.scale[i], x.float().cpu().numpy(), self.table, self.lens, n, self.code)
        self.lens = self.lens + np.asarray(n, np.int32)

    def same(self):
        assert self.gpu.status() == binding.DR_OK
        for i, (c, s) in enumerate(((self.gpu.k, self.gpu.k_scale), (self.gpu.v, self.gpu.v_scale))):
            assert (c.view(torch.uint8).cpu().numpy() == self.codes[i]).all()
            assert np.array_equal(s.cpu().numpy(), self.scale[i], equal_nan=True)

    def draw(self, T, io, loud=1.0):
        x = self.rng.standard_normal((2, self.B, T, self.H, self.d)) * loud
        return [torch.from_numpy(a).to(TYPES[io]).cuda() for a in x]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("H,d,io", [(1, 64, "f32"), (3, 128, "bf16")])
def test_codes_and_scales_bit_for_bit(page, code, H, d, io):
    """Calls of one token, of a few, of a page's rest and of several pages, growing in size so that
    the scales of started pages grow as well."""
    p = Pair(3, 400, H, d, page, code)
    for i, T in enumerate((1, 1, 5, page - 7, 2 * page + 3, 1, 17)):
        counts = [T, max(0, T - 1), T // 2]
        p.put(*p.draw(T, io, loud=1 + i), counts=counts)
        p.same()


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_read_back(code, out):
    p = Pair(3, 300, 2, 128, 32, code, seed=5)
    p.put(*p.draw(200, "bf16"), counts=[200, 131, 0])
    up = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    first, n, T = [0, 40, 0], [200, 91, 0], 203
    k, v = p.gpu.read(up(p.table.tolist()), up(first), up(n), T, out=out)
    for i, x in enumerate((k, v)):
        for b in range(3):
            ref = A.cache_values(p.codes[i], p.scale[i], p.table[b], first[b] + n[b], code)[first[b]:]
            # fp32: the product of a code and a scale rounded once
            ref = torch.from_numpy(ref).float().to(TYPES[out])
            assert torch.equal(x[b, :n[b]].cpu(), ref)
            assert (x[b, n[b]:] == 0).all()


def test_out_of_a_packed_projection_and_on_another_stream():
    p = Pair(2, 100, 4, 128, 64, "i8", seed=6)
    side = torch.cuda.Stream()
    big = torch.from_numpy(p.rng.standard_normal((2, 33, 24, 128))).bfloat16().cuda()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.put(big[:, :, 16:20], big[:, :, 20:], counts=None)
    side.synchronize()
    p.same()


def test_odd_values():
    """Zeros, one large value, values too small for a scale, and values that are not finite."""
    for code in ("i8", "e4m3"):
        p = Pair(1, 200, 2, 64, 16, code, seed=7)
        k, v = p.draw(80, "f32")
        k[0, :16] = 0
        k[0, 16:32] *= 1e-42
        k[0, 32, 0, 3] = 3e38
        k[0, 50, 1, 60] = float("nan")
        v[0, 3, 0, 0] = -float("inf")
        v[0, 64:] = 0
        p.put(k, v, counts=None)
        p.same()
        assert np.isnan(p.scale[0][p.table[0, 3], 1]) and not np.isnan(p.scale[0][p.table[0, 3], 0])
        p.put(*p.draw(20, "f32"), counts=None)  # the marked pages that were full stay marked
        p.same()
        k, v = p.draw(3, "f32")
        k[0, 0, 0, 0] = float("inf")            # a started page is marked by a later token
        p.put(k, v, counts=None)
        p.put(*p.draw(2, "f32"), counts=None)   # and stays so
        p.same()


def test_out_of_range_is_recorded_and_touches_nothing():
    up = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for table, lens, counts in (([[0, 9]], [0], [20]), ([[0, -1]], [20], [5]), ([[0, 1]], [-1], [2]),
                                ([[0, 1]], [30], [5]), ([[0, 1]], [0], [-1]), ([[0, 1]], [0], [26]),
                                ([[0, 1]], [2147483647], [25])):
        cache = binding.KvCache(4, 1, 64, page=16, code="i8")
        x = torch.ones(1, 25, 1, 64, device="cuda")
        cache.write(x, x, up(table), up(lens), up(counts))
        assert cache.status() == binding.DR_ERR_INDEX
        wrote = cache.k.view(4, -1).ne(0).any(1).tolist()
        assert wrote == [table[0][1] == 9, False, False, False]  # the page before the bad one is in order
        cache.clear_status()
        assert cache.status() == binding.DR_OK
        k, _ = cache.read(up(table), up(lens), up(counts), 25, out="f32")
        assert cache.status() == binding.DR_ERR_INDEX
        assert k.isnan().any()
    cache = binding.KvCache(0, 1, 64, page=16)
    cache.write(x, x, up([[0, 0]]), up([0]), up([1]))
    assert cache.status() == binding.DR_ERR_INDEX


def test_nothing_to_do():
    p = Pair(2, 64, 2, 64, 16, "i8", seed=8)
    p.put(*p.draw(0, "bf16"), counts=None)
    p.put(*p.draw(4, "bf16"), counts=[0, 0])
    p.same()
    with pytest.raises(ValueError):
        p.gpu.write(*p.draw(2, "bf16"), torch.zeros(2, 4, device="cuda"), torch.zeros(2, device="cuda"))
