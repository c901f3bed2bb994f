"""More calls around the paged cache that the host answers: tables without
pages (CPU only)."""

import pytest
import torch

import block_decoding_gb300 as bd
from test_cache_ops_host import _evict, _move, world  # noqa: F401
from test_paged_host import FAKE


def test_no_pages_to_go_to_is_not_in_place(world):  # noqa: F811
    # a table of no columns has no memory, so its pointer is that of no table
    i32, p = world.i32, world.pages
    table, none, n, m = i32(0, 1)[None], torch.empty((1, 0), dtype=torch.int32), i32(17), world.zeros(3, 2, 16, t=torch.float32)
    with pytest.raises(ValueError):
        bd.kv_move(p, i32(3, 4)[None, None], i32(2), None, table, dst_table=none)
    with pytest.raises(ValueError):
        bd.kv_evict(p, m, n, table, 8, 17, dst_table=none)
    assert not world.w.launched
    bd.kv_move(p, i32(3, 4)[None, None], i32(2), None, none, dst_table=table)     # none to come from is for the device to report
    bd.kv_evict(p, m, n, none, 8, 17)                                             # the cache's own table, without pages
    assert len(world.w.launched) == 2


def test_pages_of_no_table_are_refused():
    assert _move(dst_table=None, dst_pages=2) == 1 and _evict(dst_table=None, dst_pages=2) == 1
    assert _move(dst_table=None, dst_pages=2, B=0) == 0 and _evict(dst_table=None, dst_pages=2, B=0) == 0
    assert _move(dst_table=FAKE + 64, dst_pages=2) != 1 and _evict(dst_table=FAKE + 64, dst_pages=2) != 1
