"""GPU: calls on a given stream beside calls on the current one, nothing
synchronised in between, give what they give one after the other."""

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV = torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def _status_clear():
    bd.device_status()
    yield
    torch.cuda.synchronize()
    assert bd.device_status() == 0


@pytest.fixture
def blocks(monkeypatch):
    """Addresses of the byte buffers (workspaces) allocated since."""
    empty, seen = torch.empty, []

    def new(*a, **kw):
        t = empty(*a, **kw)
        if t.dtype == torch.uint8 and t.is_cuda:
            seen.append(t.data_ptr())
        return t

    monkeypatch.setattr(torch, "empty", new)
    return seen


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _cache(seed, lens, heads=2, dh=128, page=64, dtype=torch.bfloat16):
    """(pages, table, offsets) of a cache that holds random rows."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = bd.KVPages.empty(sum(need), page, heads, dh, dtype, DEV)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    for i, at in enumerate(np.cumsum([0] + need)[:-1]):
        table[i, :need[i]] = torch.arange(at, at + need[i])
    table = table.to(DEV)
    off = i32(np.cumsum([0] + lens))
    k, v = (torch.randn((sum(lens), heads, dh), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    bd.kv_write(pages, k, v, off, i32([0] * len(lens)), table)
    return pages, table, off


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("w", [1, 130])
def test_attention_beside_a_call_without_a_stream(w, dtype, blocks):
    lens = [60000, 9000]
    caches = [_cache(i, lens, dtype=dtype) for i in range(2)]
    gen = torch.Generator(device=DEV).manual_seed(9)
    q = [torch.randn((2 * w, 8, 128), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2)]
    off, n = i32([0, w, 2 * w]), i32(lens)
    side = torch.cuda.Stream()

    def call(i, stream):
        pages, table, _ = caches[i]
        return bd.paged_attn(q[i], pages, off, n, table, w, max(lens), right=0, return_lse=True, stream=stream)

    want = [call(i, None) for i in range(2)]
    torch.cuda.synchronize()
    del blocks[:]
    got = []
    for _ in range(8):      # the first of each pair gives its workspace back while its kernels run
        got += [call(0, None), call(1, side)]
    torch.cuda.synchronize()
    assert len(blocks) == 16 and not set(blocks[::2]) & set(blocks[1::2])
    for k, (out, lse) in enumerate(got):
        assert torch.equal(out, want[k % 2][0]) and torch.equal(lse, want[k % 2][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_reading_beside_work_whose_memory_was_given_back(dtype):
    """Buffers of the size of the read rows, given back while a long chain of
    work of the current stream still goes through them."""
    lens = [8000, 3001]
    pages, table, off = _cache(3, lens, dtype=dtype)
    zero = i32([0, 0])
    want = bd.kv_read(pages, off, zero, table, sum(lens))
    x = torch.randn((sum(lens), 2, 128), device=DEV).to(torch.bfloat16)
    side = torch.cuda.Stream()

    def chain():
        y = x
        for _ in range(60):
            y = y * 0.99 + x
        return y

    ref = chain()
    torch.cuda.synchronize()
    for _ in range(4):
        mine = chain()
        k, v = bd.kv_read(pages, off, zero, table, sum(lens), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and torch.equal(mine, ref)


def test_a_cache_filled_and_read_on_a_stream():
    pages, table, off = _cache(4, [500, 77], dtype=torch.float8_e4m3fn)
    want = bd.kv_read(pages, off, i32([0, 0]), table, 577)
    pages2 = bd.KVPages.empty(pages.num_pages, 64, 2, 128, torch.float8_e4m3fn, DEV)
    zero, side = i32([0, 0]), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bd.kv_write(pages2, *want, off, zero, table, stream=side)
    got = bd.kv_read(pages2, off, zero, table, 577, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_product_and_head_beside_work_whose_memory_was_given_back():
    gen = torch.Generator(device=DEV).manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    a, w, x = rnd(1024, 512), rnd(768, 512), rnd(1024, 768)
    hidden, head, emb = rnd(32, 512), rnd(1000, 512), rnd(1000, 512)
    want = bd.gemm_bf16(a, w)
    stats = bd.head_confidence(hidden, head, emb)
    side = torch.cuda.Stream()

    def chain():
        y = x
        for _ in range(100):
            y = y * 0.99 + x
        return y

    ref = chain()
    torch.cuda.synchronize()
    for _ in range(4):
        mine = chain()
        got = bd.gemm_bf16(a, w, stream=side)
        s = bd.head_confidence(hidden, head, emb, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(mine, ref)
        assert all(torch.equal(p, q) for p, q in zip(s, stats))


def test_served_steps_on_a_busy_stream():
    from test_gpu_serve import _server
    side = torch.cuda.Stream()
    x = torch.randn((4096, 4096), device=DEV)
    results = []
    for stream in (None, side):
        _, srv = _server()
        for rid, (prompt, resp) in enumerate([(20, 16), (60, 8), (5, 16)]):
            assert srv.submit(rid, prompt, resp)
        steps = []
        for _ in range(200):
            if stream is not None:
                with torch.cuda.stream(stream):
                    for _ in range(20):        # the step waits behind this
                        x.mul_(1.0)
            ents = srv.step(stream)
            if ents is None:
                break
            steps.append([(e["req"], e["block"], e["kind"], e["n_commit"]) for e in ents])
        torch.cuda.synchronize()
        results.append((steps, srv.tokens.cpu(), srv.mask.cpu()))
    (a, tok_a, mask_a), (b, tok_b, mask_b) = results
    assert a == b and torch.equal(tok_a, tok_b) and torch.equal(mask_a, mask_b) and not mask_a.any()
