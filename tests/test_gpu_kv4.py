"""The paged 4-bit key/value cache on the GPU against its 64-bit model
(tests/kv4_ref.py): every byte of the pages and tables, and attention."""
import numpy as np
import pytest
import torch

import kv4_ref
from kv4_ref import BAD_INDEX, BLOCK, CLAMPED, NO_PAGES, SHARED, Ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from block_sparse_attention_18_b200 import build
    build.build()
    from block_sparse_attention_18_b200 import sparstar
    return sparstar


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def model(cache):
    torch.cuda.synchronize()
    return Ref(*(t.cpu().numpy() for t in (cache.pages, cache.refs, cache.table, cache.lens)),
               cache.D)


def check_state(cache, ref, what=""):
    torch.cuda.synchronize()
    for name in ("lens", "refs", "table", "pages"):
        got, want = getattr(cache, name).cpu().numpy(), getattr(ref, name)
        bad = np.argwhere(got != want)
        assert len(bad) == 0, "%s %s differs at %s (%d places)" % (what, name, bad[0], len(bad))


def status_of(status):
    torch.cuda.synchronize()
    got = int(status.item())
    status.zero_()
    return got


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def filled(sp, lens, Hkv, D, max_pages=None, extra=2, seed=0, scramble=True):
    """A cache of sequences of these lengths with random page bytes."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-L // BLOCK) for L in lens]
    width = max_pages or max(1, max(counts))
    cache = sp.Kv4Cache.empty(max(1, sum(counts) + extra), len(lens), width, Hkv, D)
    # Scale codes 104..191 (2^-7 .. 2^3): scores and values of ordinary size.
    pages = torch.randint(0, 256, cache.pages.shape, generator=g, dtype=torch.uint8)
    a, b = BLOCK * D // 2, BLOCK * D // 32
    for at in (a, 2 * a + b):
        pages[..., at:at + b] = torch.randint(124, 160, pages[..., at:at + b].shape, generator=g,
                                              dtype=torch.uint8)
    order = torch.randperm(cache.n_pages, generator=g) if scramble else torch.arange(cache.n_pages)
    table, at = torch.full((len(lens), width), -1, dtype=torch.int32), 0
    refs = torch.zeros(cache.n_pages, dtype=torch.int32)
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c].int()
        refs[order[at:at + c]] = 1
        at += c
    cache.pages.copy_(pages)
    cache.table.copy_(table)
    cache.refs.copy_(refs)
    cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return cache


def tokens(n, H, T, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(n, H, T, D, generator=g).to(dtype).cuda() for _ in range(2))


BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- codec

@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32), (64, F32)])
@pytest.mark.parametrize("T,lens,starts", [
    (1, [1, 128, 129, 300], None),              # one token, first and last slots of pages
    (1, [9, 10, 11], [0, 5, 7]),                # inside a word of eight tokens
    (13, [40, 200, 141], [3, 120, 128]),        # odd, over a page border, at a page start
    (128, [128, 256], [0, 128]),                # whole pages
    (300, [300, 431], [0, 131]),                # several pages, ragged at both ends
])
def test_write_and_read_match_the_model(sp, D, dtype, T, lens, starts):
    cache = filled(sp, lens, 3, D, seed=T)
    ref = model(cache)
    k, v = tokens(len(lens), 3, T, D, dtype, seed=D + T)
    st = None if starts is None else ints(*starts)
    status = new_status()
    sp.sparstar_kv4_write(cache, k, v, starts=st, status=status)
    ref.write(k.float().cpu().numpy(), v.float().cpu().numpy(), starts=starts)
    check_state(cache, ref)  # also that every other byte stayed
    first = [L - T for L in lens] if starts is None else starts
    for out in (BF16, F32):
        ko, vo = sp.sparstar_kv4_read(cache, T, dtype=out, starts=ints(*first), status=status)
        kr, vr = ref.read(T, len(lens), starts=first)
        assert np.array_equal(ko.double().cpu().numpy(), kr)
        assert np.array_equal(vo.double().cpu().numpy(), vr)
    assert status_of(status) == 0


def test_quantisation_ties_and_extremes(sp):
    D = 64
    rows = []
    for s in (0.25, 0.28125, 0.46875, 2.0 ** -20, 3840.0):
        # half steps (ties) up to the largest, exactly representable in fp32
        half = (np.arange(32) - 16) * 0.5
        half[0] = 7.0
        rows.append(np.concatenate([half * s, np.nextafter(np.float32(half * s), np.float32(9e9))]))
    rng = np.random.RandomState(0)
    for e in (-140, -126, -30, -22, 0, 10, 14):
        rows.append(rng.randn(64) * 2.0 ** e)
    # magnitudes a whose a / 7 is on a border of two scales: 7 * (odd / 16)
    for m in (17, 19, 21, 31):
        rows.append(np.concatenate([np.full(32, 7 * m / 16.0),
                                    np.full(32, np.nextafter(np.float32(7 * m / 16.0), np.float32(0)))]))
    rows.append(np.zeros(64))
    x = torch.tensor(np.array(rows), dtype=torch.float32)[None, None].cuda()
    T = x.shape[2]
    cache = filled(sp, [T], 1, D)
    ref, status = model(cache), new_status()
    sp.sparstar_kv4_write(cache, x, -x, status=status)
    ref.write(x.cpu().numpy(), -x.cpu().numpy())
    check_state(cache, ref)
    # 7.5 * 3840 = 28800 is beyond the range, 26880.
    assert status_of(status) == ref.status == CLAMPED


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_tie_of_every_scale(sp, dtype):
    """Groups whose largest magnitude is 7 s, with all half steps of s: the
    multiples of s / 2 have at most 4 + 4 bits, so bf16 holds them."""
    codes = np.arange(256)
    half = np.clip((np.arange(32) - 15) * 0.5, -7, 7)
    x = (kv4_ref.scale_of(codes)[:, None] * half).reshape(1, 1, 128, 64)
    x = torch.tensor(x, dtype=dtype).cuda()
    cache = filled(sp, [128], 1, 64)
    ref, status = model(cache), new_status()
    sp.sparstar_kv4_write(cache, x, -x, status=status)
    ref.write(x.double().cpu().numpy(), -x.double().cpu().numpy())
    check_state(cache, ref)
    assert status_of(status) == 0
    a = 128 * 64 // 2
    assert cache.pages[int(cache.table[0, 0]), 0, a:a + 256].tolist() == list(range(256))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30, 26880.5])
def test_values_beyond_the_range_are_clamped_and_said(sp, bad):
    k, v = tokens(1, 2, 5, 64, F32, 0)
    v[0, 1, 3, 40] = bad
    cache = filled(sp, [5], 2, 64)
    ref, status = model(cache), new_status()
    sp.sparstar_kv4_write(cache, k, v, status=status)
    ref.write(k.cpu().numpy(), v.cpu().numpy())
    check_state(cache, ref)
    assert status_of(status) == ref.status == CLAMPED


def test_ragged_counts_and_entries_that_are_left_out(sp):
    cache = filled(sp, [50, 260, 7, 130, 129, 40, 40, 40], 2, 64)
    ref, status = model(cache), new_status()
    k, v = tokens(8, 2, 20, 64, BF16, 1)
    seqs = [1, 0, 2, 99, 1, -1, 3, 5]
    starts = [250, 31, 0, 0, 0, 0, 111, 25]      # entry 1: 31 + 20 > 50
    counts = [10, 20, 0, 3, 4, 1, 19, 21]        # entry 4 repeats slot 1, entry 7 has 21 > 20
    sp.sparstar_kv4_write(cache, k, v, seqs=ints(*seqs), starts=ints(*starts),
                          counts=ints(*counts), status=status)
    ref.write(k.float().cpu().numpy(), v.float().cpu().numpy(), seqs, starts, counts)
    check_state(cache, ref)
    assert status_of(status) == ref.status == BAD_INDEX
    ko = torch.full((8, 2, 20, 64), 77.0, device="cuda")
    vo = ko.clone()
    sp.sparstar_kv4_read(cache, 20, seqs=ints(*seqs), starts=ints(*starts), counts=ints(*counts),
                         k=ko, v=vo, status=status)
    kr, vr = ref.read(20, 8, seqs, starts, counts, fill=77.0)  # rows behind counts stay
    assert np.array_equal(ko.cpu().numpy(), kr) and np.array_equal(vo.cpu().numpy(), vr)
    assert status_of(status) == BAD_INDEX
    only = sp.sparstar_kv4_read(cache, 20, seqs=ints(1), v=vo[:1])
    assert only[0] is None and np.array_equal(
        vo[0].cpu().numpy(), ref.read(20, 1, [1])[1][0])


def test_writes_into_shared_pages_are_left_out(sp):
    cache = filled(sp, [200, 0], 1, 64, extra=4)
    sp.sparstar_kv4_fork(cache, ints(0), ints(1))
    ref, status = model(cache), new_status()
    k, v = tokens(1, 1, 10, 64, BF16, 0)
    sp.sparstar_kv4_write(cache, k, v, seqs=ints(1), status=status)
    check_state(cache, ref)
    assert status_of(status) == SHARED


# ---------------------------------------------------------------- pages

@pytest.mark.parametrize("seed", range(6))
def test_page_calls_match_the_model_over_random_runs(sp, seed):
    rng = np.random.RandomState(seed)
    n_seqs, width = 9, 5
    cache = sp.Kv4Cache.empty(23, n_seqs, width, 2, 64)
    cache.pages.copy_(torch.randint(0, 256, cache.pages.shape, dtype=torch.uint8))
    ref, status = model(cache), new_status()
    for step in range(40):
        n = rng.randint(1, n_seqs + 1)
        slots = rng.randint(-1, n_seqs + 1, n) if rng.rand() < 0.3 else rng.permutation(n_seqs)[:n]
        kind = rng.choice(["resize", "resize", "fork", "deep", "compact"])
        if kind == "resize":
            new = rng.randint(-1, width * BLOCK + 2, n)
            now = np.array([ref.lens[s] if 0 <= s < n_seqs else 0 for s in slots])
            new = np.where(rng.rand(n) < 0.5, np.minimum(now + rng.randint(0, 9, n), new), new)
            new = np.where(rng.rand(n) < 0.2, 0, new)
            seqs = None if rng.rand() < 0.2 else slots
            sp.sparstar_kv4_resize(cache, ints(*new), None if seqs is None else ints(*seqs),
                                   status=status)
            ref.resize(new, seqs)
        elif kind == "compact":
            n_live = sp.sparstar_kv4_compact(cache)
            assert int(n_live) == ref.compact()
        else:
            src = rng.randint(0, n_seqs, n)
            lens = None if rng.rand() < 0.5 else rng.randint(0, 300, n)
            sp.sparstar_kv4_fork(cache, ints(*src), ints(*slots),
                                 None if lens is None else ints(*lens), deep=kind == "deep",
                                 status=status)
            ref.fork(src, slots, lens, kind == "deep")
        check_state(cache, ref, "step %d %s" % (step, kind))
        assert status_of(status) == ref.status, (step, kind)
        ref.status = 0


def test_page_calls_over_a_pool_larger_than_one_pass(sp):
    # 9000 pages: several passes of the planning CTA over the counts, and a
    # scan whose first free page lies late.
    cache = sp.Kv4Cache.empty(9001, 3, 9001, 1, 64)
    status = new_status()
    ref = model(cache)
    for new in ([4500 * BLOCK, 0, 1], [4500 * BLOCK, 4400 * BLOCK + 5, 1], [0, 4400 * BLOCK + 5, 9],
                [3 * BLOCK, 4400 * BLOCK + 5, 9], [4700 * BLOCK, 1, 9]):
        sp.sparstar_kv4_resize(cache, ints(*new), status=status)
        ref.resize(new)
        check_state(cache, ref)
        assert status_of(status) == ref.status
        ref.status = 0
    assert int(sp.sparstar_kv4_compact(cache)) == ref.compact()
    check_state(cache, ref)


def test_too_few_pages_serves_the_entries_before(sp):
    cache = sp.Kv4Cache.empty(4, 4, 4, 1, 64)
    status = new_status()
    sp.sparstar_kv4_resize(cache, ints(2 * BLOCK, 3 * BLOCK, 1, 0), status=status)
    assert cache.lens.tolist() == [2 * BLOCK, 0, 0, 0]  # the third counts after the second
    assert status_of(status) == NO_PAGES
    assert cache.refs.tolist() == [1, 1, 0, 0]


# ------------------------------------------------------------- attention

def check_attn(sp, cache, q, expect=0, **kw):
    """Runs attention and holds it against the model.

    Tolerances.  u = finfo.eps / 2 of a type; e = 2^-24 for fp32.
    Scores: products of D terms summed in fp32, each partial sum rounded (or,
    in the tensor core, truncated: 2 e), and a scale and two roundings of the
    exponent's argument; |s| <= t, the row's largest sum of |terms|, so
    |ds| <= (2 D + 8) e t, and the weights are off by that relatively, plus
    8 e for the exponential.  Values: bf16 rounds the weights once (u of
    bf16); sums over all tokens add 4 e a page and 2 e a token of one.
    The output rounds once more.
    """
    D, pages = cache.D, max(1, -(-int(cache.lens.max()) // BLOCK))
    status = new_status()
    ref = model(cache)
    args = {k: (None if v is None else v.cpu().numpy() if torch.is_tensor(v) else v)
            for k, v in kw.items()}
    out = torch.full_like(q, float("nan"))  # every element has to be written
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    sp.sparstar_kv4_attn(cache, q, out=out, lse=lse, status=status, **kw)
    want, want_lse, size, terms = ref.attn(q.float().cpu().numpy(), **args)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    e, u = 2.0 ** -24, torch.finfo(q.dtype).eps / 2
    ds = (2 * D + 8) * e * terms
    dw = 2 * ds + (8 + 4 * pages + 2 * BLOCK) * e + (u if q.dtype == BF16 else 0.0)
    tol = (dw[..., None] * size + u * np.abs(want)) * 1.01 + 1e-30
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert len(bad) == 0, "out[%s] = %r, want %r (tol %.3g), %d off" % (
        bad[0], got[tuple(bad[0])], want[tuple(bad[0])], tol[tuple(bad[0])], len(bad))
    seen = np.isfinite(want_lse)
    assert np.array_equal(np.isneginf(got_lse), ~seen)
    err = np.abs(np.where(seen, got_lse, 0) - np.where(seen, want_lse, 0))
    lse_tol = ds + (8 + 4 * pages + 2 * BLOCK) * e + 4 * e * np.abs(np.where(seen, want_lse, 0))
    assert (err <= lse_tol).all(), "lse off by %.3g" % err.max()
    assert status_of(status) == ref.status == expect
    return out, lse


def queries(n, Hq, Lq, D, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 17)
    return (torch.randn(n, Hq, Lq, D, generator=g) * scale).to(dtype).cuda()


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32), (64, F32)])
@pytest.mark.parametrize("lens,Hq,Hkv,Lq", [
    ([1], 1, 1, 1),                       # one token
    ([127, 128, 129, 257], 2, 2, 1),      # around page borders
    ([700, 3, 0, 512, 90], 8, 2, 1),      # ragged, one empty; four heads share one
    ([300, 45], 6, 1, 3),                 # 18 rows a key head: two row tiles
    ([1500], 8, 8, 5),
    ([2100, 9], 16, 1, 2),                # 32 rows
])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("width", [None, 1300])  # wide tables: the split for long caches
def test_attention_of_few_rows(sp, D, dtype, lens, Hq, Hkv, Lq, causal, width):
    cache = filled(sp, lens, Hkv, D, seed=sum(lens), max_pages=width)
    check_attn(sp, cache, queries(len(lens), Hq, Lq, D, dtype), causal=causal)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (64, F32)])
@pytest.mark.parametrize("lens,Hq,Hkv,Lq", [
    ([640], 2, 2, 130),                   # rows past a tile of 128
    ([300, 1000, 40], 4, 2, 100),         # causal: rows before the first token (Lq > 40)
    ([513], 2, 1, 257),
    ([128, 1], 2, 2, 64),
])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_of_many_rows(sp, D, dtype, lens, Hq, Hkv, Lq, causal):
    cache = filled(sp, lens, Hkv, D, seed=sum(lens))
    check_attn(sp, cache, queries(len(lens), Hq, Lq, D, dtype), causal=causal)


@pytest.mark.parametrize("D,dtype,Lq,G,causal", [
    (128, BF16, 1, 1, False), (128, BF16, 300, 1, False), (128, BF16, 300, 2, True),
    (64, BF16, 140, 1, False), (64, F32, 140, 2, True), (128, F32, 5, 1, True)])
def test_attention_over_block_lists(sp, D, dtype, Lq, G, causal):
    lens = [1000, 390]
    cache = filled(sp, lens, 2, D, seed=Lq)
    rng = np.random.RandomState(Lq)
    nqb, max_sel = -(-Lq // BLOCK), 6
    idx = np.full((2, 2 * G, nqb, max_sel), -1, np.int32)
    cnt = rng.randint(0, max_sel + 1, idx.shape[:3]).astype(np.int32)
    for at in np.ndindex(*cnt.shape):
        blocks = -(-lens[at[0]] // BLOCK)
        cnt[at] = min(cnt[at], blocks)
        idx[at][:cnt[at]] = np.sort(rng.permutation(blocks)[:cnt[at]])
    cnt[0, 0, 0] = 0  # a row without blocks
    idx[0, 0, 0] = 0
    cnt[1, 1, 0], idx[1, 1, 0, :2] = 2, (3, 1)  # the last block first
    check_attn(sp, cache, queries(2, 2 * G, Lq, D, dtype), causal=causal,
               kv_idx=torch.tensor(idx).cuda(), kv_cnt=torch.tensor(cnt).cuda())


@pytest.mark.parametrize("Lq", [2, 200])
def test_bad_list_entries_and_slots_are_skipped_and_said(sp, Lq):
    cache = filled(sp, [500, 200], 1, 128)
    nqb = -(-Lq // BLOCK)
    idx = torch.tensor([-1, 1, 2, 4, 1 << 30], dtype=torch.int32).cuda()
    idx = idx.expand(2, 2, nqb, 5).contiguous()
    cnt = torch.full((2, 2, nqb), 9, dtype=torch.int32, device="cuda")  # over max_sel
    q = queries(2, 2, Lq, 128, BF16)
    check_attn(sp, cache, q, expect=BAD_INDEX, kv_idx=idx, kv_cnt=cnt)
    check_attn(sp, cache, q, expect=BAD_INDEX, seqs=ints(1, 7))
    check_attn(sp, cache, q, expect=BAD_INDEX, seqs=ints(-1, 0), causal=True)


@pytest.mark.parametrize("Lq", [1, 150])
def test_slots_in_any_order_and_twice(sp, Lq):
    cache = filled(sp, [90, 400, 129], 2, 128)
    check_attn(sp, cache, queries(5, 4, Lq, 128, BF16), seqs=ints(2, 0, 2, 1, 0), causal=True)


@pytest.mark.parametrize("scale", [0.0, 30.0])
@pytest.mark.parametrize("Lq,dtype", [(1, BF16), (150, BF16), (1, F32)])
def test_flat_and_peaked_scores(sp, scale, Lq, dtype):
    # Scores of several hundred: the running maximum moves, most weights vanish.
    cache = filled(sp, [1200], 1, 128)
    check_attn(sp, cache, queries(1, 2, Lq, 128, dtype, scale=scale))


@pytest.mark.parametrize("Lq", [1, 130])
def test_what_lies_behind_a_sequence_does_not_matter(sp, Lq):
    # The largest scales and codes behind the last token of the last page.
    cache = filled(sp, [200], 1, 128)
    q = queries(1, 1, Lq, 128, BF16)
    a = check_attn(sp, cache, q)
    page = cache.pages[int(cache.table[0, 1]), 0]
    keys, ks, vals, vs = page.split([8192, 512, 8192, 512])
    keys.view(128, 64)[72:] = 0
    ks.view(128, 4)[72:] = 255
    vs.view(4, 128)[:, 72:] = 255
    vals.view(128, 64)[:, 36:] = 0
    b = check_attn(sp, cache, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32)])
def test_attention_of_a_long_ragged_batch(sp, D, dtype):
    # Units that begin and end inside a warp's part, and ones over many CTAs.
    lens = [9000, 1, 130, 260, 4000, 0, 90, 129, 1000, 640, 17000, 300]
    cache = filled(sp, lens, 2, D, seed=5)
    check_attn(sp, cache, queries(len(lens), 4, 1, D, dtype))


@pytest.mark.parametrize("Lq", [1, 300])
def test_attention_is_the_same_twice(sp, Lq):
    cache = filled(sp, [5000, 77], 2, 128)
    q = queries(2, 8, Lq, 128, BF16)
    a, b = (sp.sparstar_kv4_attn(cache, q) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_behind_two_gibibytes(sp):
    # Byte offsets in the pool pass 2^32.
    Hkv, D = 16, 128
    n_pages = (1 << 32) // (Hkv * sp.sparstar_kv4_page_bytes(D)) + 40
    cache = sp.Kv4Cache.empty(n_pages, 2, 8, Hkv, D)
    cache.refs.fill_(1)
    cache.refs[-9:] = 0
    sp.sparstar_kv4_resize(cache, ints(300, 0))
    assert int(cache.table[0, 0]) == n_pages - 9
    k, v = tokens(1, Hkv, 300, D, BF16, 3)
    sp.sparstar_kv4_write(cache, k, v, seqs=ints(0))
    sp.sparstar_kv4_fork(cache, ints(0), ints(1), deep=True)
    small = sp.Kv4Cache.empty(3, 1, 3, Hkv, D)
    sp.sparstar_kv4_resize(small, ints(300))
    sp.sparstar_kv4_write(small, k, v)
    for Lq in (1, 200):
        q = queries(1, Hkv, Lq, D, BF16)
        want = sp.sparstar_kv4_attn(small, q)
        got = sp.sparstar_kv4_attn(cache, q, seqs=ints(1))
        # The tables' widths differ, so the pages may be split differently: each
        # result has its weights (which sum to 1) rounded to bf16 by 2^-8 at
        # most, and itself; |out| <= max |v|.  Sums and maxima are fp32.
        size = float(v.abs().max()) * (1 + 2.0 ** -4)  # a value read is within half a step
        assert float((got[0].float() - want[0].float()).abs().max()) <= 4 * size * 2.0 ** -8
        assert float((got[1] - want[1]).abs().max()) <= 1e-4
    for a, b in zip(sp.sparstar_kv4_read(cache, 300, seqs=ints(1)),
                    sp.sparstar_kv4_read(small, 300)):
        assert torch.equal(a, b)


# ------------------------------------------------------------- together

def test_cached_scale_gives_the_attention_of_its_values(sp):
    """The framework's own path over the cache: keys of text, reference and
    current scale go in, the block front-end selects from what comes back,
    and the listed attention over the cache equals sparstar_attn_fwd over the
    values read."""
    from block_sparse_attention_18_b200 import synth
    w = synth.custom(H=3, D=128, text=128, ref=600, cur=500, density=0.5, seed=5)
    q, k, v = (t.cuda() for t in synth.generate(w))
    cache = sp.Kv4Cache.empty(3 * w.nKB, 2, w.nKB, w.H, w.D)
    prefix = w.text + w.ref
    sp.sparstar_kv4_resize(cache, ints(prefix))
    sp.sparstar_kv4_write(cache, *(t[:, :, :prefix].contiguous() for t in (k, v)))
    sp.sparstar_kv4_fork(cache, ints(0), ints(1))  # the scale goes into its own sequence
    sp.sparstar_kv4_resize(cache, ints(w.Lk), seqs=ints(1))
    sp.sparstar_kv4_write(cache, *(t[:, :, prefix:].contiguous() for t in (k, v)), seqs=ints(1))
    kc, vc = sp.sparstar_kv4_read(cache, w.Lk, seqs=ints(1))
    out, lse, ws = sp.sparstar_forward_fused(q, kc, vc, w.text, 0, w.ref, w.cur, w.density)
    got, got_lse = sp.sparstar_kv4_attn(cache, q, seqs=ints(1), kv_idx=ws.kv_idx,
                                        kv_cnt=ws.kv_cnt)
    # The weights of both are rounded to bf16 once (2^-8 each, |v| < 6 here,
    # averaged with weights that sum to 1), and so are the outputs.
    size = float(vc.abs().max())
    assert float((got.float() - out.float()).abs().max()) <= 4 * size * 2.0 ** -8
    assert float((got_lse - lse).abs().max()) <= 1e-4
    ref = model(cache)
    assert ref.lens.tolist() == [prefix, w.Lk]
    sp.sparstar_kv4_resize(cache, ints(0), seqs=ints(1))
    assert int(sp.sparstar_kv4_compact(cache)) == -(-prefix // BLOCK)


def serve_step(sp, cache, st):
    sp.sparstar_kv4_resize(cache, st["lens"])
    sp.sparstar_kv4_write(cache, st["k"], st["v"])
    return sp.sparstar_kv4_attn(cache, st["q"], out=st["out"], lse=st["lse"], work=st["work"])


def serve_state(sp, n, Hq, Hkv, D, seed, max_pages=7):
    k, v = tokens(n, Hkv, 1, D, BF16, seed)
    need = sp.sparstar_kv4_attn_work_bytes(n, Hq, Hkv, 1, D, max_pages)
    return dict(k=k, v=v, q=queries(n, Hq, 1, D, BF16, seed),
                lens=torch.zeros(n, dtype=torch.int32, device="cuda"),
                out=torch.empty(n, Hq, 1, D, dtype=BF16, device="cuda"),
                lse=torch.empty(n, Hq, 1, device="cuda"),
                work=torch.zeros(need, dtype=torch.uint8, device="cuda"))


def test_a_serving_step_captured_into_graphs(sp):
    """resize, write and attention of one token in two graphs that share the
    scratch, replayed in turn with new inputs, against the same calls eager."""
    n, Hq, Hkv, D = 3, 4, 2, 128
    caches = [filled(sp, [126, 5, 700], Hkv, D, max_pages=7, extra=6) for _ in range(2)]
    st = serve_state(sp, n, Hq, Hkv, D, 0)
    eager = serve_state(sp, n, Hq, Hkv, D, 0)
    st["lens"].copy_(caches[0].lens)
    serve_step(sp, caches[0], st)  # first use outside the capture: nothing grows
    caches[0].pages.copy_(caches[1].pages)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            serve_step(sp, caches[0], st)
        graphs.append(g)
    for step in range(5):
        fresh = serve_state(sp, n, Hq, Hkv, D, 10 + step)
        for name in ("k", "v", "q"):
            st[name].copy_(fresh[name])
            eager[name].copy_(fresh[name])
        lens = torch.tensor([127 + step, 6 + step, 701 + step], dtype=torch.int32, device="cuda")
        st["lens"].copy_(lens)
        eager["lens"].copy_(lens)
        graphs[step % 2].replay()
        serve_step(sp, caches[1], eager)
        assert torch.equal(st["out"], eager["out"]) and torch.equal(st["lse"], eager["lse"])
    check_state(caches[0], model(caches[1]))


def test_calls_on_another_stream(sp):
    cache = filled(sp, [100, 900], 2, 128, max_pages=8, extra=3)
    twin = filled(sp, [100, 900], 2, 128, max_pages=8, extra=3)
    k, v = tokens(2, 2, 30, 128, BF16, 4)
    q = queries(2, 4, 3, 128, BF16)
    lens = ints(130, 930)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sp.sparstar_kv4_resize(cache, lens, stream=side)
    sp.sparstar_kv4_write(cache, k, v, stream=side)
    got = sp.sparstar_kv4_attn(cache, q, causal=True, stream=side)
    kv = sp.sparstar_kv4_read(cache, 40, counts=ints(40, 7), stream=side)
    side.synchronize()
    sp.sparstar_kv4_resize(twin, lens)
    sp.sparstar_kv4_write(twin, k, v)
    want = sp.sparstar_kv4_attn(twin, q, causal=True)
    kv2 = sp.sparstar_kv4_read(twin, 40, counts=ints(40, 7))
    for a, b in zip((*got, *kv), (*want, *kv2)):
        assert torch.equal(a, b)
