"""GPU: attention over the paged cache where the batch passes the host bounds,
and at the ends of the ranges of its arguments, against the float64 oracle."""

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd
from oracle import paged
from test_gpu_paged import DEV_OFFSETS, DEV_PAGE, LARGE, Batch, f64, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _status_clear():
    bd.device_status()
    yield
    torch.cuda.synchronize()
    assert bd.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [9, 40, 150])
def test_rows_of_clipped_requests_keep_their_positions(w, fp8):
    """Rows beyond max_q or q, and keys beyond max_kv, are left out; the others
    are where q_off and kv_len say."""
    b = Batch(50, [500, 300], 2, 64, 16, fp8)
    b.queries([w, w], 2)
    off = i32(b.q_off)
    cut = w - 5
    mark = torch.full_like(b.q, 3.0)
    out, lse = bd.paged_attn(b.q, b.pages, off, i32(b.lens), b.table, cut, 500, right=0, out=mark, return_lse=True)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    pos = [n - w for n in b.lens]
    kept = [np.arange(cut) + i * w for i in range(2)]
    assert (out[cut:w] == 3).all() and (out[w + cut:] == 3).all()
    c = Batch.__new__(Batch)
    c.__dict__.update(b.__dict__)
    c.w, c.q_off, c.q = [cut, cut], np.array([0, cut, 2 * cut]), torch.cat([b.q[k] for k in kept])
    c.check(torch.cat([out[k] for k in kept]), torch.cat([lse[k] for k in kept]), pos=pos, right=0)
    # q ends before the last request's rows do
    out, lse = bd.paged_attn(b.q[:2 * w - 5], b.pages, off, i32(b.lens), b.table, w, 500, left=60, right=0, return_lse=True)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    c.w, c.q_off, c.q = [w, cut], np.array([0, w, w + cut]), b.q[:w + cut]
    c.check(out, lse, pos=pos, left=60, right=0)
    # keys beyond max_kv are not there for any row
    out, lse = bd.paged_attn(b.q, b.pages, off, i32(b.lens), b.table, w, 400, left=110, right=0, return_lse=True)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    c.w, c.q_off, c.q, c.lens = b.w, b.q_off, b.q, [400, 300]
    c.k, c.v = [x[:400] for x in b.k], [x[:400] for x in b.v]
    c.check(out, lse, pos=pos, left=110, right=0)


FAR = (1 << 30) - 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [1, 40, 150])
@pytest.mark.parametrize("left,right", [(FAR, 0), (FAR - 20, 5), (-1, FAR), (FAR, FAR), (3, FAR)])
def test_far_positions_under_the_widest_masks(w, fp8, left, right):
    b = Batch(51, [200, 200, 200, 64], 1, 64, 32, fp8)
    b.queries([w] * 4, 2)
    for pos in ([FAR + 51, FAR + 130, -FAR - 60, -FAR + 30], [FAR - 20, (1 << 31) - 1, -(1 << 31), -FAR - 1 - w]):
        b.check(*b.run(pos=pos, left=left, right=right, sinks=7), pos=pos, left=left, right=right, sinks=7)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [1, 40, 150])
def test_requests_without_a_cache_at_all(w, fp8):
    b = Batch(52, [20, 30], 2, 64, 16, fp8)
    b.queries([w, w], 2)
    none = torch.empty((2, 0), dtype=torch.int32, device=b.table.device)
    for max_kv in (0, 5000):
        out, lse = bd.paged_attn(b.q, b.pages, i32(b.q_off), i32([0, 0]), none, w, max_kv, right=0, return_lse=True)
        assert not out.any() and torch.isneginf(lse).all()
    rows = torch.ones((2, 2, 64), dtype=torch.bfloat16, device=b.table.device)
    before = b.pages.k.view(torch.uint8).clone()
    bd.kv_write(b.pages, rows, rows, i32([0, 0, 0]), i32([0, 0]), none)          # no row belongs to a request
    k, v = bd.kv_read(b.pages, i32([0, 0, 0]), i32([0, 0]), none, 2, k=rows.clone(), v=rows.clone())
    assert torch.equal(k, rows) and torch.equal(v, rows)
    torch.cuda.synchronize()
    assert bd.device_status() == 0
    bd.kv_write(b.pages, rows, rows, i32([0, 1, 2]), i32([0, 0]), none)          # rows without a place
    k, v = bd.kv_read(b.pages, i32([0, 1, 2]), i32([0, 0]), none, 2)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    assert not k.any() and not v.any() and torch.equal(before, b.pages.k.view(torch.uint8))


@pytest.mark.parametrize("w", [1, 30, 40, 150, 300])
def test_small_queries_over_very_large_keys(w):
    """e4m3: keys of 2^121 and queries of 2^-108. Scores are some 2^13, so that
    products on the way to them pass fp32 unless the small factor comes first;
    nearly every row has one key that takes all the weight."""
    b = Batch(53, [700, 260], 2, 128, 32, True, spread=0.1, k_size=2.0 ** 121)
    assert all(np.isfinite(k).all() for k in b.k)
    b.queries([w, w], 2, q_size=2.0 ** -108)
    for max_kv in (None, LARGE):
        out, lse = b.run(right=0, max_kv=max_kv)
        b.check(out, lse, right=0)
        alone = 0
        for i, n in enumerate(b.lens):
            q, got = f64(b.q[i * w:(i + 1) * w]), f64(out[i * w:(i + 1) * w])
            see = paged.visible(np.arange(n - w, n), n, -1, 0, 0)
            for h in range(4):
                s = np.where(see, q[:, h] @ b.k[i][:, h // 2].T / np.sqrt(128), -np.inf)
                top = np.sort(s, axis=1)
                clear = top[:, -1] - top[:, -2] > 60       # scores are off by less than 1
                alone += clear.sum()
                want = b.v[i][s.argmax(axis=1)[clear], h // 2]
                # the weight's rounding and the output's, half a step of bf16 each
                assert (np.abs(got[clear, h] - want) <= 2.01 * 2.0 ** -8 * np.abs(want)).all()
        assert alone > 4 * w


@pytest.mark.parametrize("w", [1, 13, 30, 40, 200])
def test_small_weights_beside_a_dominant_scale(w):
    """e4m3: one key has by far the largest V scale and nothing in the columns
    that are looked at; weight times V scale of the others, 2^-4 to 2^-35 of
    it, a size to a column, keeps the bits that are promised."""
    L, dh = 640, 64
    b = Batch(54, [L], 1, dh, 32, True, spread=0.0, k_size=0.3)
    b.queries([w], 1)
    v = torch.zeros((L, 1, dh))
    size = torch.exp2(-4.0 - torch.arange(L) % 32) * (1 + torch.from_numpy(b.rng.random(L)).float())
    v[torch.arange(L), 0, 32 + torch.arange(L) % 32] = size
    v[17] = 0
    v[17, 0, 0] = 1.0
    v = v.to(torch.bfloat16)
    bd.kv_write(b.pages, b.k_in, v.to(b.table.device), b.off, i32([0]), b.table)
    codes, scale = paged.quantise(f64(v))
    b.v = [paged.restore(codes, scale)]
    out, _ = b.run(out_fp32=True)
    want, lse, absv, mag = paged.attention(f64(b.q), b.k[0], b.v[0], np.arange(w), dh ** -0.5)
    s = f64(b.q)[:, 0] @ b.k[0][:, 0].T * dh ** -0.5
    p = np.exp(s - lse)                                                     # [w][L]
    value = np.abs(paged.restore(codes, np.full(scale.shape, 127)))[:, 0]   # the codes' own values
    vs = 2.0 ** (scale[:, 0].astype(float) - 127)
    if w <= 32:
        # (l, the sum of exp(score - reference), is at least this: the reference is no score's superior)
        floor = 2.0 ** -41.6 * vs.max() * np.exp(s.max(axis=1, keepdims=True) - lse)
        tol = np.maximum(2.0 ** -8.8 * p * vs, floor) @ value
    else:
        tol = 2.0 ** -8 * (p * vs) @ value
    d = (dh + 8) * 2.0 ** -23 * mag[..., None]
    tol = tol + absv[:, 0] * (2 * d[:, 0] + 2.0 ** -20 + (L + 8) * 2.0 ** -23) + 1e-38
    err = np.abs(f64(out) - want)[:, 0]
    assert (err <= tol).all(), f"{(err / tol)[:, 32:].max(axis=0)} of the tolerance"
