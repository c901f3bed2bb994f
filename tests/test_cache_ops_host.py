"""The entry points around the paged cache refuse bad arguments on the host,
before anything is launched, and take their memory from the stream they are
given (CPU only)."""

import ctypes
import types

import pytest
import torch

import block_decoding_gb300 as bd
from test_paged_host import BAD_PAGES, FAKE, _pages
from test_streams_host import World

B = bd._binding
ref = ctypes.byref


def _rope(rot=64, axes=3, axis=(0, 1, 2), freq=None):
    n = 32
    return B.RopeDesc(rot, axes, (ctypes.c_uint8 * 64)(*[axis[j % len(axis)] for j in range(n)]),
                      (ctypes.c_double * 64)(*(freq or [0.5] * n)))


ROPE = dict(pos=FAKE, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_stride=256, k_stride=128, v_stride=128, q_out_stride=256, off=FAKE,
            pos0=FAKE, page_table=FAKE, max_pages=2, B=1, Hq=4, rows=4)


def _write(pages=None, rope=None, **kw):
    a = B.RopeWriteArgs(*dict(ROPE, **kw).values())
    return bd.LIB.dllm_rope_kv_write(ref(pages or _pages()), ref(rope or _rope()), ref(a), None)


TREE = dict(q=FAKE, q_stride=256, out=FAKE, out_fp32=0, lse=None, q_off=FAKE, kv_len=FAKE, q_pos=None, page_table=FAKE,
            max_pages=2, B=1, Hq=4, max_q=40, max_kv=32, q_rows=40, scale=0.1, left=-1, right=-1, sinks=0)


def _tree(pages=None, mask=FAKE, stride=2, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = B.PagedAttnArgs(*dict(TREE, **kw).values())
    return bd.LIB.dllm_tree_attn(ref(pages or _pages()), ref(a), mask, stride, ws, ws_bytes, None)


def _mask(parent=FAKE, off=FAKE, rows=8, max_q=40, n=1, mask=FAKE, stride=2, depth=None):
    return bd.LIB.dllm_tree_mask(parent, off, rows, max_q, n, mask, stride, depth, None)


MASS = dict(q=FAKE, q_stride=256, lse=FAKE, mass=FAKE, q_off=FAKE, kv_len=FAKE, q_pos=None, fresh=None, page_table=FAKE,
            max_pages=2, B=1, Hq=4, max_q=4, max_kv=32, q_rows=4, scale=0.1, right=-1, decay=1.0)


def _mass(pages=None, **kw):
    return bd.LIB.dllm_attn_mass(ref(pages or _pages()), ref(B.AttnMassArgs(*dict(MASS, **kw).values())), None)


MOVE = dict(src=FAKE, count=FAKE, first=None, page_table=FAKE, dst_table=None, src_heads=2, max_n=4, max_pages=2, dst_pages=0,
            B=1, mass=None)


def _move(pages=None, **kw):
    return bd.LIB.dllm_kv_move(ref(pages or _pages()), ref(B.KvMoveArgs(*dict(MOVE, **kw).values())), None)


EVICT = dict(mass=FAKE, kv_len=FAKE, page_table=FAKE, dst_table=None, max_pages=2, dst_pages=0, B=1, budget=8, max_kv=32,
             sinks=2, recent=2, move_mass=1, new_len=FAKE, keep=FAKE)


def _evict(pages=None, **kw):
    return bd.LIB.dllm_kv_evict(ref(pages or _pages()), ref(B.KvEvictArgs(*dict(EVICT, **kw).values())), None)


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_bad_pages_are_refused(kw, code):
    p = _pages(**kw)
    rot = _rope(rot=32) if p.dh < 64 else None
    assert _write(p, rot) == code and _tree(p) == code and _mass(p) == code and _move(p) == code and _evict(p) == code


def test_rope_refuses_bad_arguments():
    p, r, a = _pages(), _rope(), B.RopeWriteArgs(*ROPE.values())
    assert bd.LIB.dllm_rope_kv_write(None, ref(r), ref(a), None) == 1
    assert bd.LIB.dllm_rope_kv_write(ref(p), None, ref(a), None) == 1
    assert bd.LIB.dllm_rope_kv_write(ref(p), ref(r), None, None) == 1
    for name in ("rows", "B", "max_pages", "Hq"):
        assert _write(**{name: -1}) == 1
    for name in ("pos", "q", "k", "v", "q_out", "off", "pos0", "page_table"):
        assert _write(**{name: None}) == 1
    for name in ("q", "k", "v", "q_out"):
        assert _write(**{name: FAKE + 8}) == 1
    for name, least in (("q_stride", 256), ("k_stride", 128), ("v_stride", 128), ("q_out_stride", 256)):
        assert _write(**{name: least - 8}) == 1 and _write(**{name: least + 4}) == 1
    assert _write(B=4097) == 2 and _write(rows=(1 << 31) - 1) == 2 and _write(Hq=16385, q_stride=1 << 21, q_out_stride=1 << 21) == 2
    assert _write(rope=_rope(rot=-16)) == 1 and _write(rope=_rope(rot=80)) == 1 and _write(rope=_rope(rot=24)) == 2
    assert _write(rope=_rope(axes=0)) == 1 and _write(rope=_rope(axes=5)) == 2 and _write(rope=_rope(axes=2)) == 1
    for bad in (float("nan"), float("inf"), 1025.0, -1025.0):
        assert _write(rope=_rope(freq=[0.5] * 31 + [bad])) == 1
    assert _write(rows=0, k=None) == 0 and _write(B=0, off=None) == 0
    assert _write(page_table=None, max_pages=0) != 1


def test_tree_refuses_bad_arguments():
    for f, names in ((_mask, ("rows", "max_q", "n", "stride")), (_tree, ("B", "max_q", "max_kv", "q_rows", "max_pages", "sinks"))):
        for name in names:
            assert f(**{name: -1}) == 1
    for name in ("parent", "off", "mask"):
        assert _mask(**{name: None}) == 1
    assert _mask(max_q=1025, stride=64) == 2 and _mask(n=4097) == 2 and _mask(stride=1) == 1
    assert _mask(rows=0, parent=None) == 0 and _mask(max_q=0, parent=None) == 0 and _mask(n=0, parent=None) == 0
    for name in ("q", "out", "q_off", "kv_len", "page_table", "mask"):
        assert _tree(**{name: None}) == 1
    assert _tree(stride=1) == 1 and _tree(max_q=1025, q_rows=1025, stride=64) == 2
    assert _tree(q_pos=FAKE) == 1 and _tree(left=0) == 1 and _tree(right=0) == 1     # a tree is the order
    assert _tree(Hq=3) == 2 and _tree(B=4097) == 2 and _tree(q=FAKE + 8) == 1 and _tree(q_stride=248) == 1
    assert _tree(B=0, q=None, mask=None) == 0 and _tree(max_q=0, q=None, mask=None) == 0
    big = dict(max_kv=9000, max_pages=600)
    a = B.PagedAttnArgs(*dict(TREE, **big).values())
    need = bd.LIB.dllm_paged_attn_workspace(ref(_pages()), ref(a))
    assert need > 0 and _tree(ws=None, ws_bytes=0, **big) == 3 and _tree(ws_bytes=need - 1, **big) == 3


def test_mass_refuses_bad_arguments():
    assert bd.LIB.dllm_attn_mass(ref(_pages()), None, None) == 1
    for name in ("B", "max_q", "max_kv", "q_rows", "max_pages"):
        assert _mass(**{name: -1}) == 1
    for name in ("q", "lse", "mass", "q_off", "kv_len", "page_table"):
        assert _mass(**{name: None}) == 1
    assert _mass(Hq=0) == 1 and _mass(Hq=3) == 2 and _mass(Hq=130, q_stride=130 * 64) == 2 and _mass(B=4097) == 2
    assert _mass(q=FAKE + 8) == 1 and _mass(mass=FAKE + 4) == 1 and _mass(q_stride=248) == 1 and _mass(q_stride=260) == 1
    for name in ("right", "max_kv"):
        assert _mass(**{name: 1 << 30}) == 2
    assert _mass(q_rows=1 << 28) == 2 and _mass(max_q=1 << 28) == 2
    for bad in (float("nan"), float("inf")):
        assert _mass(decay=bad) == 1
    for name in ("B", "max_q", "q_rows", "max_kv"):
        assert _mass(**{name: 0, "q": None}) == 0
    assert _mass(max_pages=0, page_table=None) == 0


def test_moves_refuse_bad_arguments():
    assert bd.LIB.dllm_kv_move(ref(_pages()), None, None) == 1 and bd.LIB.dllm_kv_evict(ref(_pages()), None, None) == 1
    for name in ("B", "max_n", "max_pages", "dst_pages"):
        assert _move(**{name: -1}) == 1
    for name in ("src", "count", "page_table"):
        assert _move(**{name: None}) == 1
    assert _move(src_heads=3) == 1 and _move(src_heads=0) == 1 and _move(B=4097) == 2 and _move(max_n=1 << 30) == 2
    assert _move(dst_table=FAKE, dst_pages=1) == 1             # the same table with other pages
    assert _move(B=0, src=None) == 0 and _move(max_n=0, src=None) == 0
    for name in ("B", "max_kv", "sinks", "recent", "max_pages", "dst_pages"):
        assert _evict(**{name: -1}) == 1
    for name in ("mass", "kv_len", "page_table", "new_len", "keep"):
        assert _evict(**{name: None}) == 1
    assert _evict(budget=0) == 1 and _evict(sinks=5, recent=4) == 1 and _evict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1) == 1
    assert _evict(B=4097) == 2 and _evict(max_kv=1 << 30) == 2 and _evict(budget=1 << 30) == 2
    assert _evict(dst_table=FAKE, dst_pages=1) == 1 and _evict(B=0, mass=None) == 0


def test_rope_tables():
    r = bd.Rope.standard(128, 1e6, sections=[16, 24, 24])
    assert r.axes == 3 and list(r.desc.axis)[:64] == [0] * 16 + [1] * 24 + [2] * 24 and r.desc.rot == 128
    assert r.desc.freq[0] == 1.0 and abs(r.desc.freq[32] - 1e-3) < 1e-18
    r = bd.Rope.standard(64, rot=32, sections=[4, 8, 4], interleaved=True)
    assert list(r.desc.axis)[:16] == [0, 1, 2] * 4 + [1] * 4 and r.desc.rot == 32
    assert bd.Rope.standard(64).axes == 1 and bd.Rope(64, [], []).desc.rot == 0
    for bad in (lambda: bd.Rope(64, [0] * 8, [1.0] * 7), lambda: bd.Rope(64, [0] * 12, [1.0] * 12), lambda: bd.Rope(64, [0] * 40, [1.0] * 40),
                lambda: bd.Rope(64, [4] * 8, [1.0] * 8), lambda: bd.Rope(64, [-1] * 8, [1.0] * 8),
                lambda: bd.Rope.standard(64, sections=[16, 8])):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("rot", [17, 24, 31, -16, 80])
def test_rope_of_uncommon_sizes_is_refused(rot):
    with pytest.raises(ValueError):
        bd.Rope.standard(64, rot=rot)


@pytest.fixture
def world(monkeypatch):
    w = types.SimpleNamespace(i32=lambda *v: torch.tensor(v, dtype=torch.int32), zeros=lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t))
    w.pages = types.SimpleNamespace(index=0, device=torch.device("cpu"), heads=2, dh=64, desc=B.KvPagesDesc(), _need={},
                                    k=torch.zeros((3, 2, 16, 64)))
    w.w = World(monkeypatch)
    return w


@pytest.mark.parametrize("side", [False, True])
def test_calls_allocate_on_their_stream(world, side):
    s = world.w.side if side else None
    i32, zeros, p = world.i32, world.zeros, world.pages
    off, table, n = i32(0, 5), i32(0, 1)[None], i32(17)
    got = bd.rope_kv_write(p, bd.Rope.standard(64), i32(0, 1, 2, 3, 4), zeros(5, 4, 64), zeros(5, 2, 64), zeros(5, 2, 64), off, n, table, stream=s)
    world.w.check([got], s, 0)
    world.w.blocks.clear(), world.w.recorded.clear()
    mask, depth = bd.tree_mask(i32(-1, 0, 1, 1, 0), off, 5, stream=s)
    world.w.check([mask, depth], s, 0)
    world.w.blocks.clear(), world.w.recorded.clear()
    out, lse = bd.tree_attn(zeros(5, 4, 64), p, off, n, table, mask, 5, 17, return_lse=True, stream=s)
    world.w.check([out, lse], s, 1)
    world.w.blocks.clear(), world.w.recorded.clear()
    new, keep = bd.kv_evict(p, zeros(3, 2, 16, t=torch.float32), n, table, 8, 17, stream=s)
    world.w.check([new, keep], s, 0)
    m = zeros(3, 2, 16, t=torch.float32)
    bd.attn_mass(zeros(5, 4, 64), zeros(5, 4, t=torch.float32), p, m, off, n, table, 5, 17, stream=s)
    bd.kv_move(p, i32(3, 4)[None, None], i32(2), None, table, mass=m, stream=s)
    assert [x[0] for x in world.w.launched] == ["dllm_rope_kv_write", "dllm_tree_mask", "dllm_tree_attn", "dllm_kv_evict",
                                                "dllm_attn_mass", "dllm_kv_move"]
    assert all(x[1] is s for x in world.w.launched)


def test_binding_refuses_what_does_not_fit(world):
    i32, zeros, p = world.i32, world.zeros, world.pages
    off, table, n, m = i32(0, 5), i32(0, 1)[None], i32(17), world.zeros(3, 2, 16, t=torch.float32)
    q, k, r = zeros(5, 4, 64), zeros(5, 2, 64), bd.Rope.standard(64)
    pos, mask = i32(0, 1, 2, 3, 4), i32(1, 3, 7, 15, 31)[:, None]
    bad = [
        lambda: bd.rope_kv_write(p, bd.Rope.standard(128), pos, q, k, k, off, n, table),
        lambda: bd.rope_kv_write(p, r, pos[:4], q, k, k, off, n, table),
        lambda: bd.rope_kv_write(p, bd.Rope.standard(64, sections=[16, 16]), pos, q, k, k, off, n, table),
        lambda: bd.rope_kv_write(p, r, pos, q[:4], k, k, off, n, table),
        lambda: bd.rope_kv_write(p, r, pos, q, k, k[:4], off, n, table),
        lambda: bd.rope_kv_write(p, r, pos, None, k, k, off, n, table, q_out=q),
        lambda: bd.rope_kv_write(p, r, pos, q, k, k, off, n, table, q_out=q[:3]),
        lambda: bd.tree_mask(pos, off, 5, mask=i32(0, 0, 0, 0)[:, None]),
        lambda: bd.tree_mask(pos, off, 40, mask=mask),
        lambda: bd.tree_mask(pos, off, -1),
        lambda: bd.tree_mask(pos, off, 5, depth=pos[:3]),
        lambda: bd.tree_attn(q, p, off, n, table, mask[:4], 5, 17),
        lambda: bd.tree_attn(q, p, off, n, table, mask, 33, 17),
        lambda: bd.tree_attn(q, p, off, n, table, mask, 5, 1 << 32),
        lambda: bd.attn_mass(q, zeros(5, 3, t=torch.float32), p, m, off, n, table, 5, 17),
        lambda: bd.attn_mass(q, zeros(5, 4, t=torch.float32), p, m[:2], off, n, table, 5, 17),
        lambda: bd.attn_mass(q, zeros(5, 4, t=torch.float32), p, m, off, n, table, 5, 17, fresh=pos),
        lambda: bd.attn_mass(q, zeros(5, 4, t=torch.float32), p, m, off, n, table, 5, 17, right=1 << 31),
        lambda: bd.kv_move(p, pos[None, None], i32(2, 2), None, table),
        lambda: bd.kv_move(p, pos[None, None].expand(1, 3, 5).contiguous(), n, None, table),
        lambda: bd.kv_move(p, pos[None, None], n, pos, table),
        lambda: bd.kv_move(p, pos[None, None], n, None, table[0]),
        lambda: bd.kv_move(p, pos[None, None], n, None, table, dst_table=table[0]),
        lambda: bd.kv_evict(p, m, n, table, 1 << 31, 17),
        lambda: bd.kv_evict(p, m, n, table, 8, 17, sinks=-1),
        lambda: bd.kv_evict(p, m, n, table, 8, 17, keep=pos),
        lambda: bd.kv_evict(p, m, n, table, 8, 17, new_len=pos),
        lambda: bd.kv_evict(p, m[:1], n, table, 8, 17),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    assert not world.w.launched
