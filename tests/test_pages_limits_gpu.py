"""gdn_pages_* where the pool is full: what needs a page is refused whole, what needs none is done."""
import pytest

from test_pages_gpu import Both

pytestmark = pytest.mark.gpu


def full():
    """12 pages in use, sequence 0's first one held by sequence 3 too."""
    b = Both(12, 16, 6, 4)
    b.extend([0, 1, 2], [20, 64, 5])
    assert b.fork([0], [3])
    assert b.extend([4], [48]) and b.extend([5], [16])
    assert min(b.m.refs) > 0 and b.m.refs[b.m.table[0][0]] == 2
    return b


def test_a_trim_into_a_shared_page_needs_a_free_one():
    b = full()
    assert not b.trim([0], [3])
    # pages that the call itself gives back do not count, whoever gives them
    assert not b.trim([1, 0], [0, 3]) and not b.trim([0, 3], [3, 3])
    assert b.trim([1], [60])                   # its own page: no copy
    assert b.trim([0], [16])                   # the shared page whole, the one behind it given back
    assert b.trim([3], [3])                    # which now takes the copy
    assert b.m.refs[b.m.table[0][0]] == 1 and b.m.table[3][0] != b.m.table[0][0]


def test_a_full_pool_still_frees_and_grows_within_pages():
    b = full()
    assert not b.extend([5], [1])
    assert b.extend([2], [11]) == [[b.m.table[2][0] * 16 + j for j in range(5, 16)]]
    b.free([1, 3])
    assert b.extend([5], [1])
    b.compact()
