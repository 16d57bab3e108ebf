"""How the few-row attention over the 4-bit cache cuts its line of tiles
(csrc/kv4_attn_few.cu), checked on the host: a pair of warps may be given one
tile at most, as its two warps have no way to join what several would leave."""
import os
import random
import re

from conftest import ROOT

SOURCE = open(os.path.join(ROOT, "block_sparse_attention_18_b200", "csrc",
                           "kv4_attn_few.cu")).read()


def constant(name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, SOURCE).group(1))


def longest_part(total, ctas, parts):
    """Tiles of the longest part: the kernel's arithmetic for whole tiles."""
    share = -(-total // ctas)
    longest = 0
    for cta in range(ctas):
        c0 = min(share * cta, total)
        pieces = min(c0 + share, total) - c0
        each, rest = divmod(pieces, parts)
        longest = max(longest, each + (rest > 0))
    return longest


def test_a_pair_has_one_tile_at_most():
    ctas, pairs = constant("kCtas"), constant("kPairs")
    # The rule: the tables' widths give at most `pairs` tiles a CTA, and lengths
    # beyond a table are cut, so there are no more tiles than that.
    assert "most <= (double)kPairs * kCtas" in SOURCE
    launches = re.findall(r"launch<(?:128|64), \d, (?:true|false), (\w+), 2>", SOURCE)
    assert launches == ["kPairs"] * 2
    rng = random.Random(0)
    totals = [1, pairs, ctas - 1, ctas, ctas + 1, pairs * ctas - 1, pairs * ctas]
    for total in totals + [rng.randint(1, pairs * ctas) for _ in range(200)]:
        assert longest_part(total, ctas, pairs) <= 1, total
    assert longest_part(pairs * ctas + 1, ctas, pairs) > 1  # the rule is not looser


def test_a_pair_waits_for_nothing_but_its_copies():
    # The barriers of the kernel: one a stage, and none between the warps.
    assert re.findall(r"__shared__ uint64_t (.*);", SOURCE) == ["full[kParts][kStages]"]
