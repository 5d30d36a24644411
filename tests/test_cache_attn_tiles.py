"""GPU parity of the attention over the paged 8-bit cache at the edges of its tiles of 256 rows (query tokens
times query heads) on the tensor cores, and over several tiles of a sequence.  Bounds: those of
tests/test_cache_attn.py, whose helper this uses."""
import pytest

from test_cache_attn import Case

pytestmark = pytest.mark.gpu

SHAPES = [  # lens, T, Hq, H, d, page, window, counts
    ([40], 128, 2, 2, 64, 16, 0, None),                # the first half of a tile, filled
    ([0, 9], 129, 2, 2, 128, 64, 0, None),             # one row in the second half
    ([70], 255, 1, 1, 128, 32, 0, None),
    ([0, 130], 256, 1, 1, 64, 64, 0, None),            # a tile, filled
    ([0, 130], 257, 1, 1, 128, 128, 0, None),          # a second tile of one row
    ([33], 171, 3, 1, 64, 16, 0, None),                # 513 rows: tokens across tiles, a third tile of one row
    ([200, 3], 300, 8, 2, 128, 64, 0, [300, 65]),      # five tiles, and two
    ([600], 400, 4, 2, 64, 64, 150, None),             # tiles whose windows share no position
    ([0], 700, 2, 1, 128, 16, 90, None),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_parity(shape, code):
    lens, T, Hq, H, d, page, window, counts = shape
    c = Case(lens, T, Hq, H, d, page, code, "bf16", "bf16", window=window, counts=counts, seed=31)
    c.check(*c.run())
