"""The pipelines of the many-row attention over the 4-bit cache, checked on the
host (csrc/kv4_attn_many.cu describes the roles).

With block lists its ring is that of the attention kernel over plain values,
which test_ring_protocol.py covers.  The two other forms:

shared    Without lists blocks A and B read one stream of tiles, the longer
          one's.  A stage is free after its last reader: B's product, or A's
          where B has no tile left.
in place  One query block, whose tiles are read by two softmax halves; a lane
          copies packed tiles into a ring of three, six warps unpack them from
          there into the ring of five, one warp issues whichever product is
          ready next.

As there, a test of slot e is exact when slot e - 2S has landed before it (two
full barriers a stage), and the waits must not form a cycle.
"""
import graphlib

import pytest

from test_ring_protocol import STAGES, producer_order, slot_k, slot_v

PACKED = 3


def copied(n):
    """The order of the copying lane: the blocks that its lookup ahead gives."""
    out, nxt, last, before = [], 0, 0, 0

    def key():
        nonlocal nxt, last, before
        before, last, nxt = last, nxt, nxt + 1
        return last

    if n > 0:
        out.append(("K", key()))
    for j in range(n):
        if j + 1 < n:
            out.append(("K", key()))
        out.append(("V", before if j + 1 < n else last))
    return out


@pytest.mark.parametrize("n", range(0, 20))
def test_one_stream_is_copied_unpacked_and_read_in_one_order(n):
    order = copied(n)
    assert order == [(t, j) for t, _, j in producer_order(n, 0)]
    kinds = [e > 0 and (e % 2 == 0 or e == 2 * n - 1) for e in range(2 * n)]
    assert kinds == [t == "V" for t, _ in order]
    for e, (t, j) in enumerate(order):
        assert e == (slot_v if t == "V" else slot_k)(0, j, n, 0)


def acyclic(g):
    return list(graphlib.TopologicalSorter(g).static_order())  # raises CycleError


def before(g):
    """Every event's predecessors."""
    out = {}
    for ev in acyclic(g):
        out[ev] = set()
        for q in g.get(ev, ()):
            out[ev] |= out[q] | {q}
    return out


def shared(nA, nB):
    """The waits of the shared form; LOAD(e): slot e has landed, in any order."""
    n, g = max(nA, nB), {}
    seq = [(x, j) for j in range(n) for x in range(2) if j < (nA, nB)[x]]
    order = copied(n)
    reader = {}
    for x, j in seq:  # the last reader of a slot stands
        reader[slot_k(0, j, n, 0)] = ("QK", x, j)
        reader[slot_v(0, j, n, 0)] = ("PV", x, j)
        frees = x == 1 or j >= nB
        assert frees == (x == max(y for y in range(2) if j < (nA, nB)[y]))

    def add(a, *bs):
        g.setdefault(a, set()).update(b for b in bs if b is not None)

    for e in range(len(order)):
        add(("ISSUE", e), ("ISSUE", e - 1) if e else None,
            reader[e - STAGES] if e >= STAGES else None)
        add(("LOAD", e), ("ISSUE", e))
    for i, (x, j) in enumerate(seq):
        prev = seq[i - 1] if i else None
        add(("QKtest", x, j), ("QK",) + prev if prev else None)
        add(("QK", x, j), ("QKtest", x, j), ("LOAD", slot_k(0, j, n, 0)),
            ("SREAD",) + prev if prev else None)
        add(("SREAD", x, j), ("QK", x, j), ("PSTORE", x, j - 1) if j else None)
        add(("PSTORE", x, j), ("SREAD", x, j), ("PV", x, j - 1) if j else None)
        add(("PVtest", x, j), ("PSTORE", x, j), ("PV",) + prev if prev else None)
        add(("PV", x, j), ("PVtest", x, j), ("LOAD", slot_v(0, j, n, 0)))
    return seq, g


@pytest.mark.parametrize("nA", list(range(0, 9)) + [23])
def test_shared_tiles(nA):
    for nB in list(range(0, 9)) + [22, 24]:
        n = max(nA, nB)
        seq, g = shared(nA, nB)
        known = before(g)
        for x, j in seq:
            for test, e in ((("QKtest", x, j), slot_k(0, j, n, 0)),
                            (("PVtest", x, j), slot_v(0, j, n, 0))):
                if e >= 2 * STAGES:
                    assert ("LOAD", e - 2 * STAGES) in known[test], (nA, nB, e)
                # Nobody tests a slot after its barrier's next use: that waits
                # for the stage's readers.
                nxt = ("ISSUE", e + 2 * STAGES)
                if nxt in g:
                    assert test in known[nxt]


def in_place(n):
    g, order = {}, copied(n)
    reader = {}
    for j in range(n):
        reader[slot_k(0, j, n, 0)] = ("QK", j)
        reader[slot_v(0, j, n, 0)] = ("PV", j, 1)

    def add(a, *bs):
        g.setdefault(a, set()).update(b for b in bs if b is not None)

    for e in range(len(order)):
        add(("COPY", e), ("COPY", e - 1) if e else None,
            *((("UNPACK", e - PACKED, w) for w in range(6)) if e >= PACKED else ()))
        for w in range(6):
            add(("UNPACK", e, w), ("COPY", e), ("UNPACK", e - 1, w) if e else None,
                reader[e - STAGES] if e >= STAGES else None)
        add(("LOAD", e), *(("UNPACK", e, w) for w in range(6)))
    for j in range(n):
        add(("QKtest", j), ("QK", j - 1) if j else None)
        add(("QK", j), ("QKtest", j), ("LOAD", slot_k(0, j, n, 0)),
            *((("SREAD", h, j - 1) for h in range(2)) if j else ()))
        for h in range(2):
            add(("SREAD", h, j), ("QK", j), ("PSTORE", h, j - 1) if j else None)
            add(("PSTORE", h, j), ("SREAD", h, j), ("PV", j - 1, h) if j else None)
            prev = ("PV", j, 0) if h else ("PV", j - 1, 1) if j else None
            add(("PVtest", j, h), ("PSTORE", h, j), prev)
            add(("PV", j, h), ("PVtest", j, h),
                ("LOAD", slot_v(0, j, n, 0)) if h == 0 else None)
    return g


@pytest.mark.parametrize("n", list(range(0, 14)) + [40])
def test_tiles_unpacked_in_place(n):
    g = in_place(n)
    known = before(g)
    for j in range(n):
        for test, e in ((("QKtest", j), slot_k(0, j, n, 0)),
                        (("PVtest", j, 0), slot_v(0, j, n, 0))):
            if e >= 2 * STAGES:
                assert ("LOAD", e - 2 * STAGES) in known[test], (n, e)
        if j + 1 < n:
            # One S, one P a half, one phase of each barrier at a time.
            for h in range(2):
                assert ("SREAD", h, j) in known[("QK", j + 1)]
                assert ("PVtest", j, h) in known[("PSTORE", h, j + 1)]
    for e in range(PACKED, 2 * n):
        assert all(("UNPACK", e - PACKED, w) in known[("COPY", e)] for w in range(6))
