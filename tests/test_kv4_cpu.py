"""Argument checks of the paged 4-bit key/value cache on a host without a
GPU: every call below is refused before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref

A = 0x10000      # fake device addresses: never dereferenced
MIS = 0x10002


@pytest.fixture(scope="module")
def sp():
    from block_sparse_attention_18_b200 import build
    build.build()
    from block_sparse_attention_18_b200 import sparstar
    return sparstar


def cache(sp, **kw):
    f = dict(pages=A, refs=A, table=A, lens=A, work=A, n_pages=64, n_seqs=8, max_pages=16, Hkv=2,
             D=128)
    f.update(kw)
    return sp._Kv4Struct(*f.values())


BAD_CACHES = [dict(pages=0), dict(refs=0), dict(table=0), dict(lens=0), dict(pages=0x10008),
              dict(refs=0x10004), dict(table=MIS), dict(lens=MIS), dict(n_pages=0), dict(n_seqs=0),
              dict(max_pages=0), dict(Hkv=0), dict(D=96), dict(n_pages=(1 << 28) + 1),
              dict(n_seqs=(1 << 20) + 1), dict(max_pages=(1 << 23) + 1), dict(Hkv=65536)]


@pytest.mark.parametrize("kw", BAD_CACHES, ids=str)
def test_every_call_refuses_a_bad_cache(sp, kw):
    L, c = sp.lib, cache(sp, **kw)
    assert L.sparstar_kv4_resize(c, A, A, 1, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_fork(c, A, A, 0, 1, 0, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_compact(c, A, 0) == sp.EINVAL
    assert L.sparstar_kv4_write(c, A, A, 0, 1, 1, 0, 0, 0, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_read(c, A, A, 0, 1, 1, 0, 0, 0, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_attn(c, A, 0, 1, 2, 1, 0, 0.1, 0, 0, 0, 0, A, 0, A, 1 << 40, 0,
                               0) == sp.EINVAL


def test_page_calls_refuse_bad_arguments(sp):
    L, c = sp.lib, cache(sp)
    for n, seqs, lens in ((0, 0, A), (9, 0, A), (1, 0, 0), (1, MIS, A), (1, 0, MIS)):
        assert L.sparstar_kv4_resize(c, seqs, lens, n, 0, 0) == sp.EINVAL
    for src, dst, n, deep in ((0, A, 1, 0), (A, 0, 1, 0), (A, A, 0, 0), (A, A, 9, 0), (A, A, 1, 2),
                              (MIS, A, 1, 1)):
        assert L.sparstar_kv4_fork(c, src, dst, 0, n, deep, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_compact(c, 0, 0) == sp.EINVAL
    no_work = cache(sp, work=0)
    assert L.sparstar_kv4_resize(no_work, 0, A, 1, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_resize(None, 0, A, 1, 0, 0) == sp.EINVAL


def test_codec_calls_refuse_bad_arguments(sp):
    L, c = sp.lib, cache(sp)
    for call in (L.sparstar_kv4_write, L.sparstar_kv4_read):
        assert call(c, A, A, 7, 1, 1, 0, 0, 0, 0, 0) == sp.EDTYPE
        for k, n, T in ((A, 0, 1), (A, 9, 1), (A, 1, 0), (A, 1, 1 << 31), (0x10008, 1, 1)):
            assert call(c, k, A, 0, n, T, 0, 0, 0, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_write(c, A, 0, 0, 1, 1, 0, 0, 0, 0, 0) == sp.EINVAL
    assert L.sparstar_kv4_read(c, 0, 0, 0, 1, 1, 0, 0, 0, 0, 0) == sp.EINVAL
    many = cache(sp, n_seqs=1 << 20, Hkv=65535)
    assert L.sparstar_kv4_write(many, A, A, 0, 1 << 20, 1, 0, 0, 0, 0, 0) == sp.EINVAL  # grid


def test_attention_refuses_bad_arguments(sp):
    L, c = sp.lib, cache(sp)

    def call(**kw):
        f = dict(q=A, dtype=0, n=1, Hq=4, Lq=1, seqs=0, tau=0.1, causal=0, idx=0, cnt=0, sel=0,
                 out=A, lse=0, work=A, bytes=1 << 40, status=0, stream=0)
        f.update(kw)
        return L.sparstar_kv4_attn(c, *f.values())
    assert call(dtype=2) == sp.EDTYPE
    for kw in (dict(q=0), dict(out=0), dict(q=0x10008), dict(out=0x10008), dict(work=0x10008),
               dict(n=0), dict(n=9), dict(Hq=3), dict(Hq=0), dict(Lq=0), dict(Lq=1 << 31),
               dict(tau=float("nan")), dict(causal=2), dict(sel=1), dict(sel=-1),
               dict(idx=A, sel=3), dict(cnt=A, sel=3), dict(lse=MIS), dict(seqs=MIS),
               dict(n=1 << 20, seqs=A, Lq=1 << 12)):
        assert call(**kw) == sp.EINVAL, kw
    need = sp.sparstar_kv4_attn_work_bytes(1, 4, 2, 1, 128, 16)
    assert call(bytes=need - 1) == sp.ESIZE
    assert call(work=0) == sp.EINVAL


def test_sizes(sp):
    assert sp.sparstar_kv4_page_bytes(128) == 17408
    assert sp.sparstar_kv4_page_bytes(64) == 8704
    assert sp.sparstar_kv4_page_bytes(96) == -1
    assert sp.lib.sparstar_kv4_work_ints(0, 1) == -1
    assert sp.lib.sparstar_kv4_work_ints(10, 3) >= 13
    for bad in ((0, 4, 2, 1, 128, 9), (1, 3, 2, 1, 128, 9), (1, 4, 2, 1, 80, 9),
                (1, 4, 2, 0, 128, 9), (1, 4, 2, 1, 128, 0)):
        assert sp.sparstar_kv4_attn_work_bytes(*bad) == -1
    assert sp.sparstar_kv4_attn_work_bytes(1, 4, 2, 1, 128, 9, torch.float16) == -1
    assert sp.sparstar_kv4_attn_work_bytes(1, 4, 2, 1, 128, 9) >= sp.KV4_WORK_ZEROS


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_no_device_is_reported(sp):
    L, c = sp.lib, cache(sp)
    assert L.sparstar_kv4_resize(c, 0, A, 1, 0, 0) == sp.ENODEV
    assert L.sparstar_kv4_write(c, A, A, 0, 1, 1, 0, 0, 0, 0, 0) == sp.ENODEV
    assert L.sparstar_kv4_attn(c, A, 0, 1, 4, 1, 0, 0.1, 0, 0, 0, 0, A, 0, A, 1 << 40, 0,
                               0) == sp.ENODEV


def test_the_model_codec_round_trips():
    rng = np.random.RandomState(0)
    codes = rng.randint(0, 16, (5, 64))
    assert np.array_equal(kv4_ref.unpack(kv4_ref.pack(codes)), codes)
    x = rng.randn(100, 64) * 3
    c, s, clamped = kv4_ref.quantise(x)
    back = (c - 8) * kv4_ref.scale_of(s).repeat(32, -1)
    # The scale is within 2^-4 of a / 7, and a code within half a step.
    step = np.abs(x.reshape(100, 2, 32)).max(-1).repeat(32, -1) / 7 * (1 + 2.0 ** -4)
    assert not clamped and (np.abs(back - x) <= step / 2).all()
    assert (c >= 1).all() and (c <= 15).all()
