"""Failure detection of the 4-bit cache's calls on the GPU without a fault: waits
that run out.  The hooks withhold copies, so that what waits for them gives up,
says so and leaves; the context stays usable."""
import time

import pytest
import torch

from kv4_ref import BLOCK
from test_gpu_kv4 import (BF16, F32, check_attn, check_state, filled, ints, model, new_status,
                          queries, sp, status_of)  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 64])
def test_a_compaction_whose_copies_give_up_says_so(sp, D):
    cache = filled(sp, [40, 2 * BLOCK, 9], 2, D, extra=0, scramble=False)
    sp.sparstar_kv4_resize(cache, ints(0), seqs=ints(0))  # page 3 is to move to page 0
    n_live = ints(7)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    sp.sparstar_test_kv4_compact_timeout(cache, n_live)
    torch.cuda.synchronize()
    assert int(n_live) == -1
    assert 1.0 < time.monotonic() - t0 < 30.0

    # The same context compacts a cache that is whole.
    cache = filled(sp, [40, 2 * BLOCK, 9], 2, D, extra=0, scramble=False)
    sp.sparstar_kv4_resize(cache, ints(0), seqs=ints(0))
    ref = model(cache)
    assert int(sp.sparstar_kv4_compact(cache, n_live)) == ref.compact() == 3
    check_state(cache, ref)


def test_nothing_to_copy_does_not_wait(sp):
    cache = filled(sp, [40, 9], 1, 64, extra=2, scramble=False)
    n_live = ints(7)
    sp.sparstar_test_kv4_compact_timeout(cache, n_live)
    assert int(n_live) == 2


@pytest.mark.parametrize("lens,Hq,Hkv,Lq,width,dtype", [
    ([900, 40], 4, 2, 1, None, BF16),       # few rows: a warp a part
    ([900, 40], 4, 2, 1, 100, BF16),        # a pair of warps a tile
    ([900, 40], 4, 2, 3, None, F32),
    ([900, 40], 2, 2, 130, None, BF16),     # many rows, pages unpacked in place
    ([900, 40, 2000, 0, 300], 8, 2, 150, None, BF16),  # many rows, pages unpacked first
])
def test_attention_whose_copies_give_up_says_so(sp, lens, Hq, Hkv, Lq, width, dtype):
    cache = filled(sp, lens, Hkv, 128, max_pages=width)
    q = queries(len(lens), Hq, Lq, 128, dtype)
    need = sp.sparstar_kv4_attn_work_bytes(len(lens), Hq, Hkv, Lq, 128, cache.max_pages, dtype)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out, status = torch.zeros_like(q), new_status()
    torch.cuda.synchronize()
    t0 = time.monotonic()
    sp.sparstar_test_kv4_attn_timeout(cache, q, out, work, status)
    assert status_of(status) == sp.STATUS_TIMEOUT
    assert 1.0 < time.monotonic() - t0 < 60.0

    # The same context goes on, with scratch of its own.
    check_attn(sp, cache, q)
