"""Forks whose parent's partly filled page has a table entry outside the pool: the
child holds no page for it, so that it never shows rows of a sequence that held
such a page before."""
import pytest
import torch

import decode_attention_static_gb300 as da

pytestmark = pytest.mark.gpu

NONE = -1


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def parents(pages):
    """Three sequences of 20, 24 and 40 rows in pages of 16, three slots for children, `pages` free pages."""
    table = i32([[0, 1, NONE], [2, 3, NONE], [4, 5, 6]] + [[NONE] * 3] * 3)
    pool = da.alloc_page_pool(7 + pages)
    free, counts, order = da.page_pool_views(pool)
    free.fill_(pages)
    counts[:7] = 1
    order[:pages] = torch.arange(7, 7 + pages, dtype=torch.int32, device="cuda")
    return table, i32([20, 24, 40, 0, 0, 0]), pool


@pytest.mark.parametrize("bad", [-1, -7, 9, 1 << 30])
def test_no_page_for_an_entry_outside_the_pool(bad):
    """Two pages are free and two forks can use one: the fork between them takes none."""
    table, lens, pool = parents(2)
    table[1, 1] = bad
    err = i32([0])
    copies = da.kvcache_fork_paged(table, lens, i32([0, 1, 2]), i32([3, 4, 5]), pool, 16, err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_PAGE
    assert table[3:].tolist() == [[0, 8, NONE], [2, NONE, NONE], [4, 5, 7]]
    assert copies.tolist() == [[1, NONE, 6], [8, NONE, 7], [4, 0, 8]]
    assert lens.tolist() == [20, 24, 40, 20, 24, 40]
    free, counts, _ = da.page_pool_views(pool)
    assert free.tolist() == [0] and counts.tolist() == [2, 1, 2, 1, 2, 2, 1, 1, 1]


def test_no_page_needed_where_none_is_free():
    table, lens, pool = parents(0)
    table[0, 1] = 77
    err = i32([0])
    copies = da.kvcache_fork_paged(table, lens, i32([0]), i32([3]), pool, 16, err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_PAGE and copies.tolist() == [[NONE], [NONE], [0]]
    assert table[3].tolist() == [0, NONE, NONE] and lens[3].item() == 20


def test_attention_on_the_child_reports_the_page():
    """The child gives NaN and the error bit, as its parent does, not somebody else's rows."""
    table, lens, pool = parents(3)
    table[1, 1] = NONE
    k, v = (torch.randn(10, 1, 16, 64, device="cuda").half() for _ in range(2))
    da.kvcache_copy_pages(k, v, da.kvcache_fork_paged(table, lens, i32([1]), i32([3]), pool, 16))
    err = i32([0])
    both = table[[1, 3]].contiguous()
    out = da.decode_attn_paged_fwd(torch.randn(2, 1, 64, device="cuda").half(), k, v, both, i32([24, 24]), err_flag=err)
    assert out.isnan().all() and int(err.item()) == da.DA_DEVERR_PAGE
