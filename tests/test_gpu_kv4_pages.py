"""Page calls of the 4-bit cache that run out of pages, entry by entry, against
what the header says and the model."""
import pytest

from kv4_ref import BLOCK, NO_PAGES
from test_gpu_kv4 import check_state, filled, ints, model, new_status, sp, status_of  # noqa: F401

pytestmark = pytest.mark.gpu


def test_entries_that_need_no_page_are_served_behind_a_refused_one(sp):
    cache = filled(sp, [5, 5, BLOCK, 300, 60], 1, 64, max_pages=4, extra=1)
    ref, status = model(cache), new_status()
    # Entry 0 needs two pages of one; 1 grows within its page; 2 needs the page
    # that is there, but comes behind entry 0; 3 shrinks; 4 stays.
    new = [2 * BLOCK + 5, 6, BLOCK + 1, 10, 60]
    sp.sparstar_kv4_resize(cache, ints(*new), status=status)
    assert cache.lens.tolist() == [5, 6, BLOCK, 10, 60]
    assert status_of(status) == NO_PAGES
    ref.resize(new)
    check_state(cache, ref)


def test_a_shared_page_needs_its_copy_first(sp):
    # Growing by one token within a page that two sequences hold takes a page:
    # with none free it is refused, with one it is served, first come first.
    cache = filled(sp, [5, 0, 0], 2, 64, max_pages=2, extra=0)
    sp.sparstar_kv4_fork(cache, ints(0, 0), ints(1, 2))
    ref, status = model(cache), new_status()
    sp.sparstar_kv4_resize(cache, ints(6, 6, 5), status=status)
    assert cache.lens.tolist() == [5, 5, 5] and status_of(status) == NO_PAGES
    ref.resize([6, 6, 5])
    check_state(cache, ref)

    cache = filled(sp, [5, 0, 0], 2, 64, max_pages=2, extra=1)
    sp.sparstar_kv4_fork(cache, ints(0, 0), ints(1, 2))
    ref = model(cache)
    sp.sparstar_kv4_resize(cache, ints(6, 6, 5), status=status)
    assert cache.lens.tolist() == [6, 5, 5] and status_of(status) == NO_PAGES
    ref.resize([6, 6, 5])
    check_state(cache, ref)
