"""The few-row attention over the 4-bit cache where its tiles go to pairs of
warps: tables of more than two and at most eight tiles a CTA, at both ends of
that range.  Tolerances: see check_attn."""
import pytest

from test_gpu_kv4 import BF16, check_attn, filled, queries, sp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("lens,Hq,Hkv,Lq,width", [
    ([148 * 128 - 5], 8, 8, 1, 148),              # every part of every CTA has a tile
    ([148 * 128 - 5], 8, 8, 1, 149),              # one more a head: no pairs
    ([37 * 128 + 1], 16, 8, 3, 38),               # just over two a CTA; six rows
    ([37 * 128], 8, 8, 1, 37),                    # two a CTA: no pairs
    ([9000, 1, 0, 4000, 130, 128, 77, 9472], 4, 2, 2, 74),   # ragged, some without a tile
    ([3], 1, 1, 1, 1184),                         # one tile, a wide table
])
def test_tiles_of_pairs(sp, D, lens, Hq, Hkv, Lq, width):
    cache = filled(sp, lens, Hkv, D, seed=sum(lens), max_pages=width)
    for causal in (False, True):
        check_attn(sp, cache, queries(len(lens), Hq, Lq, D, BF16), causal=causal)
