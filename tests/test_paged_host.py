"""The paged-cache entry points refuse bad arguments on the host, before
anything is launched (CPU only)."""

import ctypes
import os

import pytest
import torch

import block_decoding_gb300 as bd

P = ctypes.c_void_p
FAKE = 256


def _pages(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, type=0, num_pages=8, page_size=16, heads=2, dh=64)
    a.update(kw)
    return bd._binding.KvPagesDesc(*a.values())


def _write(pages=None, k=FAKE, v=FAKE, ks=128, vs=128, rows=4, off=FAKE, pos0=FAKE, table=FAKE, n=2, B=1):
    return bd.LIB.dllm_kv_write(ctypes.byref(pages or _pages()), k, v, ks, vs, rows, off, pos0, table, n, B, None)


def _read(pages=None, k=FAKE, v=FAKE, rows=4, off=FAKE, pos0=FAKE, table=FAKE, n=2, B=1):
    return bd.LIB.dllm_kv_read(ctypes.byref(pages or _pages()), k, v, rows, off, pos0, table, n, B, None)


BAD_PAGES = [(dict(type=2), 2), (dict(dh=96), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(heads=0), 1),
             (dict(heads=257), 2), (dict(num_pages=0), 1), (dict(num_pages=1 << 27), 2), (dict(k=None), 1),
             (dict(v=None), 1), (dict(k=264), 1), (dict(v=FAKE + 2), 1), (dict(type=1), 1),
             (dict(type=1, k_scale=FAKE), 1)]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_bad_pages_are_refused(kw, code):
    p = _pages(**kw)
    assert _write(p) == code and _read(p) == code and _attn(p) == code


def test_moves_refuse_bad_arguments():
    assert bd.LIB.dllm_kv_write(None, FAKE, FAKE, 128, 128, 4, FAKE, FAKE, FAKE, 2, 1, None) == 1
    for f in (_write, _read):
        assert f(rows=-1) == 1 and f(B=-1) == 1 and f(n=-1) == 1
        assert f(B=4097) == 2
        for name in ("k", "v", "off", "pos0", "table"):
            assert f(**{name: None}) == 1
        assert f(k=FAKE + 8) == 1 and f(v=FAKE + 8) == 1
        assert f(rows=0, k=None) == 0 and f(B=0, off=None) == 0         # nothing to do
    assert _write(ks=120) == 1 and _write(vs=120) == 1                  # rows overlap
    assert _write(ks=132) == 1 and _write(vs=132) == 1                  # misaligned rows


ATTN = dict(q=FAKE, q_stride=256, out=FAKE, out_fp32=0, lse=None, q_off=FAKE, kv_len=FAKE, q_pos=None, page_table=FAKE,
            max_pages=2, B=1, Hq=4, max_q=4, max_kv=32, q_rows=4, scale=0.1, left=-1, right=-1, sinks=0)


def _attn(pages=None, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = bd._binding.PagedAttnArgs(*dict(ATTN, **kw).values())
    return bd.LIB.dllm_paged_attn(ctypes.byref(pages or _pages()), ctypes.byref(a), ws, ws_bytes, None)


def test_attention_refuses_bad_arguments():
    for name in ("B", "max_q", "max_kv", "q_rows", "max_pages", "sinks"):
        assert _attn(**{name: -1}) == 1
    for name in ("q", "out", "q_off", "kv_len", "page_table"):
        assert _attn(**{name: None}) == 1
    assert _attn(Hq=0) == 1 and _attn(Hq=3) == 2 and _attn(Hq=130, q_stride=130 * 64) == 2
    assert _attn(B=4097) == 2
    assert _attn(q=FAKE + 8) == 1 and _attn(out=FAKE + 8) == 1
    assert _attn(q_stride=248) == 1 and _attn(q_stride=260) == 1
    for name in ("left", "right", "sinks", "max_kv"):
        assert _attn(**{name: 1 << 30}) == 2
    assert _attn(q_rows=1 << 28) == 2 and _attn(max_q=1 << 28) == 2
    assert _attn(B=0, q=None) == 0 and _attn(max_q=0, q=None) == 0 and _attn(q_rows=0, q=None) == 0
    assert bd.LIB.dllm_paged_attn(ctypes.byref(_pages()), None, None, 0, None) == 1


def test_attention_workspace():
    def need(pages=None, **kw):
        a = bd._binding.PagedAttnArgs(*dict(ATTN, **kw).values())
        return bd.LIB.dllm_paged_attn_workspace(ctypes.byref(pages or _pages()), ctypes.byref(a))

    assert need(_pages(dh=96)) == 0 and need(Hq=3) == 0
    big = dict(B=16, Hq=32, max_q=96, max_kv=9000, q_stride=32 * 64)
    n = need(**big)
    assert n % 256 == 0
    for kw in (dict(B=1), dict(max_q=1), dict(max_kv=200), dict(B=3, max_q=33, max_kv=5000)):
        assert need(**dict(big, **kw)) <= n
    if n:
        assert _attn(ws=None, ws_bytes=0, **big) == 3
        assert _attn(ws_bytes=n - 1, **big) == 3 and _attn(ws=FAKE + 16, ws_bytes=n, **big) == 3


def test_binding_refuses_what_is_not_a_cache():
    k = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bd.KVPages(k, k)                                    # not on a GPU
    with pytest.raises(TypeError):
        bd.KVPages(k.float(), k.float())
    with pytest.raises(ValueError):
        bd.KVPages(k[0], k[0])
    with pytest.raises(ValueError):
        bd.KVPages(k, k[:1])
    with pytest.raises(ValueError):
        bd.KVPages(k, k, k[..., 0], k[..., 0])              # scales beside bf16 pages
    f = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        bd.KVPages(f, f)                                    # 8-bit pages without scales


def test_no_piece_is_read_after_a_wait_that_gave_up():
    """A piece's slot holds anything until the piece is published, and its
    numbers become addresses: every wait for one decides what happens next."""
    here = os.path.join(os.path.dirname(bd.__file__), "csrc")
    for name in ("paged_attn.cu", "paged_rows.cu"):
        with open(os.path.join(here, name)) as f:
            lines = [x.strip() for x in f if "_wait(&piece_full[" in x]
        assert len(lines) >= 4
        for x in lines:
            assert x.startswith(("ok = ", "if (")), f"{name}: result dropped: {x}"
        # what a stage found is voted on before its rows are used
        assert any(x.startswith("if (bar_any(") and "||" in x for x in lines), name


def test_a_table_without_pages_is_no_null_argument():
    # what an empty tensor's address is: requests without any cached row
    assert _attn(page_table=None, max_pages=0) != 1
    assert _write(table=None, n=0) != 1 and _read(table=None, n=0) != 1
    assert _attn(page_table=None, max_pages=1) == 1 and _write(table=None, n=1) == 1 and _read(table=None, n=1) == 1


@pytest.mark.parametrize("heads,dh", [(1, 64), (2, 128), (3, 64)])
def test_moves_refuse_rows_whose_numbers_pass_32_bits(heads, dh):
    # the last block's rows are numbered beyond `rows`, by less than a block of threads
    p, stride = _pages(heads=heads, dh=dh), heads * dh
    for rows in ((1 << 31) - 1, (1 << 31) - 127):
        assert _write(p, ks=stride, vs=stride, rows=rows) == 2 and _read(p, rows=rows) == 2
