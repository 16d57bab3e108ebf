"""Refusals of the 4-bit cache's calls that test_kv4_cpu.py does not make, on a
host without a GPU: every call below is refused before anything is launched."""
import types

import pytest

from test_kv4_cpu import A, MIS, cache, sp  # noqa: F401


def test_misaligned_lists_of_slots_are_refused(sp):
    L, c = sp.lib, cache(sp)
    assert L.sparstar_kv4_write(c, A, A, 0, 1, 1, MIS, 0, 0, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_read(c, A, A, 0, 1, 1, MIS, 0, 0, 0, 0) == sp.EINVAL


def test_misaligned_status_words_are_refused(sp):
    L, c = sp.lib, cache(sp)
    assert L.sparstar_kv4_resize(c, 0, A, 1, MIS, 0) == sp.EINVAL
    assert L.sparstar_kv4_fork(c, A, A, 0, 1, 0, MIS, 0) == sp.EINVAL
    assert L.sparstar_kv4_write(c, A, A, 0, 1, 1, 0, 0, 0, MIS, 0) == sp.EINVAL
    assert L.sparstar_kv4_read(c, A, A, 0, 1, 1, 0, 0, 0, MIS, 0) == sp.EINVAL
    assert L.sparstar_kv4_attn(c, A, 0, 1, 4, 1, 0, 0.1, 0, 0, 0, 0, A, 0, A, 1 << 40, MIS,
                               0) == sp.EINVAL


def test_the_compaction_hook_refuses_as_the_call_does(sp):
    L = sp.lib
    for call in (L.sparstar_kv4_compact, L.sparstar_test_kv4_compact_timeout):
        assert call(cache(sp), 0, 0) == sp.EINVAL
        assert call(cache(sp), MIS, 0) == sp.EINVAL
        assert call(cache(sp, work=0), A, 0) == sp.EINVAL
        assert call(None, A, 0) == sp.EINVAL


def test_a_stream_of_another_device_is_refused(sp):
    # The switch would go to that stream's device and from there back to the
    # cache's, on whatever stream is current there.
    here = types.SimpleNamespace(index=0, device="cuda:0")
    there = types.SimpleNamespace(device_index=1, cuda_stream=7)
    for call in (lambda: sp.sparstar_kv4_resize(here, None, stream=there),
                 lambda: sp.sparstar_kv4_fork(here, None, None, stream=there),
                 lambda: sp.sparstar_kv4_compact(here, stream=there),
                 lambda: sp.sparstar_kv4_write(here, None, None, stream=there),
                 lambda: sp.sparstar_kv4_read(here, 1, stream=there),
                 lambda: sp.sparstar_kv4_attn(here, None, stream=there)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_the_attention_hook_refuses_as_the_call_does(sp):
    c = cache(sp)

    def call(**kw):
        f = dict(q=A, dtype=0, n=1, Hq=4, Lq=1, tau=0.1, out=A, work=A, bytes=1 << 40, status=A,
                 stream=0)
        f.update(kw)
        return sp.lib.sparstar_test_kv4_attn_timeout(c, *f.values())
    assert call(dtype=2) == sp.EDTYPE
    for kw in (dict(q=0), dict(out=0), dict(work=0), dict(status=0), dict(status=MIS), dict(n=9),
               dict(Hq=3), dict(Lq=0), dict(tau=float("inf"))):
        assert call(**kw) == sp.EINVAL, kw
    assert call(bytes=100) == sp.ESIZE
