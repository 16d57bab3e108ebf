"""The paged 4-bit key/value cache on the GPU: the ways that its kernels cut
and order their work, the longest lists of sequences, scales of the scores of
every sign, values that are not numbers, several streams and captured forks.
Tolerances: see check_attn."""
import threading

import numpy as np
import pytest
import torch

from kv4_ref import BAD_INDEX, BLOCK
from test_gpu_kv4 import (BF16, F32, check_attn, check_state, filled, ints, model, new_status,
                          queries, sp, status_of, tokens)  # noqa: F401

pytestmark = pytest.mark.gpu


def lists_for(cache, lens, Hq, Lq, max_sel, seed, full=False):
    rng = np.random.RandomState(seed)
    nqb = -(-Lq // BLOCK)
    idx = np.full((len(lens), Hq, nqb, max_sel), -1, np.int32)
    cnt = np.zeros(idx.shape[:3], np.int32)
    for at in np.ndindex(*cnt.shape):
        blocks = -(-lens[at[0]] // BLOCK)
        cnt[at] = min(max_sel if full else rng.randint(0, max_sel + 1), blocks)
        idx[at][:cnt[at]] = np.sort(rng.permutation(blocks)[:cnt[at]])
    return dict(kv_idx=torch.tensor(idx).cuda(), kv_cnt=torch.tensor(cnt).cuda())


# ------------------------------------------------------ many sequences

@pytest.mark.parametrize("n,D,dtype,Lq", [(300, 128, BF16, 1), (1000, 64, BF16, 1),
                                          (257, 64, F32, 2), (520, 128, BF16, 12)])
def test_few_rows_of_many_sequences(sp, n, D, dtype, Lq):
    # More sequences than chunks of the line; a third of them empty.
    rng = np.random.RandomState(n)
    lens = (rng.randint(0, 400, n) * (rng.rand(n) < 0.67)).tolist()
    lens[n // 2] = 3000
    cache = filled(sp, lens, 1, D, seed=n)
    check_attn(sp, cache, queries(n, 2, Lq, D, dtype), causal=Lq > 1)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, BF16), (128, F32)])
@pytest.mark.parametrize("lens,Hq,Hkv,Lq", [
    ([20000], 8, 1, 1),          # one unit over every CTA
    ([20000], 8, 1, 2),          # sixteen rows
    ([9000, 20000, 77], 2, 1, 1),
    ([20000, 15000], 4, 2, 3),
    ([20000], 1, 1, 100),        # many rows: as many parts as a unit may have
    ([9000, 20000], 2, 1, 40),
])
def test_few_heads_over_long_caches(sp, D, dtype, lens, Hq, Hkv, Lq):
    cache = filled(sp, lens, Hkv, D, seed=Lq)
    q = queries(len(lens), Hq, Lq, D, dtype)
    for _ in range(2):  # the counters go back to zero
        check_attn(sp, cache, q, causal=Lq > 1)


@pytest.mark.parametrize("n,Lq", [(5, 40), (60, 20)])
def test_lists_longer_than_their_sequences(sp, n, Lq):
    # Rows of a stride far above the blocks that any of them names.
    lens = [(37 * i) % 600 for i in range(n)]
    cache = filled(sp, lens, 1, 128, seed=n)
    check_attn(sp, cache, queries(n, 2, Lq, 128, BF16),
               **lists_for(cache, lens, 2, Lq, 900 // n, seed=n))


@pytest.mark.parametrize("n,Lq", [(250, 129), (350, 129)])
def test_many_rows_of_many_sequences(sp, n, Lq):
    # Past the sequences that are put in order, past the units that are counted.
    lens = [(61 * i) % 300 for i in range(n)]
    lens[3] = 2000
    cache = filled(sp, lens, 1, 128, seed=n)
    check_attn(sp, cache, queries(n, 4, Lq, 128, BF16), causal=True)


@pytest.mark.parametrize("seed", range(2))
def test_page_calls_with_many_entries(sp, seed):
    # More entries than the planning CTA keeps in shared memory.
    rng = np.random.RandomState(seed)
    n_seqs = 1300
    cache = sp.Kv4Cache.empty(2600, n_seqs, 3, 1, 64)
    cache.pages.copy_(torch.randint(0, 256, cache.pages.shape, dtype=torch.uint8))
    ref, status = model(cache), new_status()
    for step, n in enumerate([1300, 513, 1024, 700, 1300]):
        slots = rng.randint(-1, n_seqs + 1, n) if step == 3 else rng.permutation(n_seqs)[:n]
        new = rng.randint(0, 3 * BLOCK + 1, n) * (rng.rand(n) < 0.8)
        sp.sparstar_kv4_resize(cache, ints(*new), ints(*slots), status=status)
        ref.resize(new, slots)
        check_state(cache, ref, "resize %d" % step)
        assert status_of(status) == ref.status
        ref.status = 0
        for deep in (False, True):
            half = rng.permutation(n_seqs)
            src, dst = half[:n_seqs // 2], half[n_seqs // 2:]
            sp.sparstar_kv4_fork(cache, ints(*src), ints(*dst), deep=deep, status=status)
            ref.fork(src, dst, None, deep)
            check_state(cache, ref, "fork %d" % step)
            assert status_of(status) == ref.status
            ref.status = 0
    assert int(sp.sparstar_kv4_compact(cache)) == ref.compact()
    check_state(cache, ref)


# ------------------------------------------------------ how many rows are cut

@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,Lq,width", [
    ([900, 40, 2000, 0, 300], 8, 2, 150, None),   # ragged, five query blocks: unpacked first
    ([6000, 20], 4, 1, 140, None),                # few units: the pages are split
    ([700], 4, 2, 300, 1300),                     # a wide table
    ([3000, 5], 2, 2, 257, None),                 # in place, three blocks, split
    ([500] * 20, 4, 4, 300, None),                # in place, more units than CTAs
    ([700], 16, 16, 2600, None),                  # unpacked first, more units than CTAs
    ([1], 1, 1, 700, None),                       # one token, many rows
])
def test_many_rows_cut_and_ordered(sp, lens, Hq, Hkv, Lq, width, causal):
    cache = filled(sp, lens, Hkv, 128, seed=sum(lens), max_pages=width)
    check_attn(sp, cache, queries(len(lens), Hq, Lq, 128, BF16), causal=causal)


@pytest.mark.parametrize("lens,Hq,Hkv,Lq,max_sel,causal", [
    ([2600, 100], 2, 2, 700, 20, False),     # unpacked first, split
    ([2600, 100], 2, 1, 700, 20, True),
    ([6000], 2, 2, 300, 40, False),          # in place, split
    ([1300], 16, 16, 2600, 8, False),        # more units than CTAs
    ([1000], 4, 1, 40, 8, True),             # one short block a head
])
def test_many_rows_over_lists_cut(sp, lens, Hq, Hkv, Lq, max_sel, causal):
    cache = filled(sp, lens, Hkv, 128, seed=Lq)
    check_attn(sp, cache, queries(len(lens), Hq, Lq, 128, BF16), causal=causal,
               **lists_for(cache, lens, Hq, Lq, max_sel, Lq))


@pytest.mark.parametrize("Lq", [200, 700])
def test_a_block_named_several_times_counts_as_often(sp, Lq):
    cache = filled(sp, [900], 1, 128)
    idx = torch.tensor([2, 2, 0, 7, 2], dtype=torch.int32).cuda()
    idx = idx.expand(1, 1, -(-Lq // BLOCK), 5).contiguous()
    cnt = torch.full(idx.shape[:3], 5, dtype=torch.int32, device="cuda")
    check_attn(sp, cache, queries(1, 1, Lq, 128, BF16), kv_idx=idx, kv_cnt=cnt)


# ------------------------------------------------------ scores

@pytest.mark.parametrize("tau", [-0.1, 0.0, 1e-32, 0.5])
@pytest.mark.parametrize("Lq,dtype", [(1, BF16), (150, BF16), (700, BF16), (3, F32)])
def test_scales_of_the_scores(sp, tau, Lq, dtype):
    cache = filled(sp, [700, 130], 1, 128)
    check_attn(sp, cache, queries(2, 2, Lq, 128, dtype), tau=tau, causal=True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("Lq,dtype", [(3, BF16), (150, BF16), (700, BF16), (3, F32)])
def test_queries_that_are_not_numbers_stay_in_their_rows(sp, bad, Lq, dtype):
    cache = filled(sp, [900], 2, 128)
    q = queries(1, 4, Lq, 128, dtype)
    want, want_lse = sp.sparstar_kv4_attn(cache, q)
    at = (0, 1, min(Lq - 1, 130))
    q[at][5] = bad
    out, lse = sp.sparstar_kv4_attn(cache, q)
    assert torch.isnan(out[at]).all() and not torch.isfinite(lse[at])
    out[at], lse[at] = want[at], want_lse[at]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# ------------------------------------------------------ streams and graphs

@pytest.mark.parametrize("Lq", [1, 150, 700])
def test_two_streams_read_one_cache(sp, Lq):
    cache = filled(sp, [5000, 900], 2, 128)
    qs = [queries(2, 4, Lq, 128, BF16, seed) for seed in range(4)]
    want = [sp.sparstar_kv4_attn(cache, q) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [sp.sparstar_kv4_attn(cache, q, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_threads_use_one_cache(sp):
    cache = filled(sp, [5000, 900], 2, 128)
    q = queries(2, 4, 1, 128, BF16)
    want = sp.sparstar_kv4_attn(cache, q)
    torch.cuda.synchronize()
    wrong = []

    def run():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                out, lse = sp.sparstar_kv4_attn(cache, q)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(out, want[0]) and torch.equal(lse, want[1])):
                    wrong.append(1)

    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("Lq", [1, 150, 700])
def test_a_captured_fork_of_streams(sp, Lq):
    """Write on one branch, attention over another cache on a second one, both
    read after the join; the captured calls follow several nodes at once."""
    caches = [filled(sp, [600, 90], 2, 128, seed=s) for s in range(2)]
    k, v = tokens(2, 2, 40, 128, BF16, 0)
    q = queries(2, 4, Lq, 128, BF16)
    twin = filled(sp, [600, 90], 2, 128, seed=0)
    sp.sparstar_kv4_write(twin, k, v)
    want = [sp.sparstar_kv4_attn(twin, q), sp.sparstar_kv4_attn(caches[1], q)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        other = sp.sparstar_kv4_attn(caches[1], q, stream=side)
        sp.sparstar_kv4_write(caches[0], k, v)
        main.wait_stream(side)
        mine = sp.sparstar_kv4_attn(caches[0], q)
        kv = sp.sparstar_kv4_read(caches[0], 90)
    for _ in range(3):
        for t in (*mine, *other, *kv):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got, w in ((mine, want[0]), (other, want[1]), (kv, sp.sparstar_kv4_read(twin, 90))):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


def test_a_run_of_calls_without_pauses(sp):
    """Each call reads what the one before it wrote, many times over: a kernel
    that starts before the last one's end must not see its work half done."""
    lens, n, Hkv = [100, 1, 640, 255], 4, 2
    cache = filled(sp, lens, Hkv, 128, max_pages=8, extra=12)
    ref, status = model(cache), new_status()
    outs, now = [], list(lens)
    for step in range(60):
        grow = 1 + step % 7
        now = [L + grow if L + grow <= 1000 else 5 for L in now]
        new = ints(*now)
        k, v = tokens(n, Hkv, 1, 128, BF16, step)
        sp.sparstar_kv4_resize(cache, new, status=status)
        sp.sparstar_kv4_write(cache, k, v, status=status)
        outs.append((queries(n, 4, 1, 128, BF16, step), k, v, list(now)))
        outs[-1] += (sp.sparstar_kv4_attn(cache, outs[-1][0], status=status),
                     sp.sparstar_kv4_read(cache, 1, starts=new - 1, status=status))
    torch.cuda.synchronize()
    for q, k, v, new, (out, lse), (ko, vo) in outs:
        ref.resize(new)
        ref.write(k.float().cpu().numpy(), v.float().cpu().numpy())
        kr, vr = ref.read(1, n, starts=[L - 1 for L in new])
        assert np.array_equal(ko.double().cpu().numpy(), kr)
        assert np.array_equal(vo.double().cpu().numpy(), vr)
        want = ref.attn(q.float().cpu().numpy())
        # check_attn's bounds for at most eight pages, in their plainest form
        dw = 2 * (2 * 128 + 8) * 2.0 ** -24 * want[3] + 400 * 2.0 ** -24 + 2.0 ** -8
        tol = dw[..., None] * want[2] + np.abs(want[0]) * 2.0 ** -8
        assert (np.abs(out.double().cpu().numpy() - want[0]) <= tol * 1.01).all()
    check_state(cache, ref)
    assert status_of(status) == ref.status == 0


def test_page_calls_captured_into_a_graph(sp):
    """Free, fork both ways, grow and compact, replayed over tables that the
    replay before changed, against the model."""
    cache = filled(sp, [700, 0, 0, 130], 1, 64, max_pages=8, extra=20)
    status, n_live = new_status(), ints(0)
    src, dst, deep = ints(0, 3), ints(1, 2), ints(1)
    lens = ints(650, 130)
    none, grown, first = ints(0, 0), ints(655, 135), ints(0)
    ref = model(cache)

    def calls(c):
        c("resize", none, dst)
        c("fork", src[1:], dst[:1], lens[1:], False)
        c("resize", first, deep)
        c("fork", src, dst, lens, False)
        c("resize", grown, dst)
        c("resize", none, dst)
        c("fork", src, dst, lens, True)
        c("compact")

    def on_gpu(name, *args):
        if name == "resize":
            sp.sparstar_kv4_resize(cache, *args, status=status)
        elif name == "fork":
            sp.sparstar_kv4_fork(cache, *args, status=status)
        else:
            sp.sparstar_kv4_compact(cache, n_live)

    def on_model(name, *args):
        args = [x.cpu().numpy() if torch.is_tensor(x) else x for x in args]
        if name == "compact":
            assert int(n_live) == ref.compact()
        else:
            getattr(ref, name)(*args)

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls(on_gpu)
    for step in range(4):
        g.replay()
        torch.cuda.synchronize()
        calls(on_model)
        check_state(cache, ref, "replay %d" % step)
        # 655 + 3 * 128 tokens are more than eight pages hold.
        assert status_of(status) == ref.status == (BAD_INDEX if step == 3 else 0)
        grown.add_(128)


def test_scratch_given_up_is_made_anew(sp):
    cache = filled(sp, [5000], 1, 128)
    q = queries(1, 2, 1, 128, BF16)
    want = sp.sparstar_kv4_attn(cache, q)
    torch.cuda.synchronize()
    for work in cache._work_of.values():
        work[:sp.KV4_WORK_ZEROS].fill_(1)  # as a call that gave up may leave it
    cache.drop_work()
    got = sp.sparstar_kv4_attn(cache, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
