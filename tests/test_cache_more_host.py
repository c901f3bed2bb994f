"""More calls around the paged cache that the host answers: tables without pages,
axes without pairs, frequencies from any sequence (CPU only)."""

import array

import numpy as np
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


@pytest.mark.parametrize("sections,interleaved", [([32, 0], False), ([16, 16, 0], True), ([0, 32, 0, 0], False), ([0, 0, 32], False)])
def test_sections_without_pairs_are_axes(world, sections, interleaved):  # noqa: F811
    i32, zeros, p = world.i32, world.zeros, world.pages
    r = bd.Rope.standard(64, sections=sections, interleaved=interleaved)
    assert r.axes == len(sections)
    off, table, n, k = i32(0, 5), i32(0, 1)[None], i32(17), zeros(5, 2, 64)
    used = max(a for a, m in enumerate(sections) if m) + 1
    for axes in range(used, len(sections) + 1):         # rows that no pair turns by may be left out
        bd.rope_kv_write(p, r, torch.zeros((axes, 5), dtype=torch.int32), None, k, k, off, n, table)
    assert len(world.w.launched) == len(sections) - used + 1
    for axes in (used - 1, len(sections) + 1):
        with pytest.raises(ValueError):
            bd.rope_kv_write(p, r, torch.zeros((axes, 5), dtype=torch.int32), None, k, k, off, n, table)


@pytest.mark.parametrize("make", [list, tuple, bytes, lambda x: np.array(x), lambda x: np.array(x, np.int16), lambda x: torch.tensor(x),
                                  lambda x: array.array("i", x)])
def test_axes_and_frequencies_of_any_sequence(make):
    axis, freq = [0, 1, 2, 0, 1, 2, 2, 1], [1.0, 0.5, 0.25, 2.0, 3.0, -1.0, 0.0, 8.0]
    r = bd.Rope(64, make(axis), np.array(freq, np.float32))
    assert r.axes == 3 and list(r.desc.axis)[:9] == axis + [0] and list(r.desc.freq)[:9] == freq + [0.0]
    with pytest.raises(ValueError):
        bd.Rope(64, make([0] * 7 + [4]), freq)
