"""GPU parity of the paged K/V cache: writing, reading and attention against
the float64 oracle.

Writing and reading are exact: codes, scales and restored values equal the
oracle's bit for bit. Attention is held element by element to what its
roundings allow, with A = sum_u w_u |v_u| of the element:
  * a weight is rounded to bf16, 2^-8 of it: 2^-8 A
  * a score is an fp32 sum of dh products whose magnitudes add up to at most
    `mag`, plus a few more operations: d = (dh + 8) 2^-23 mag off, so a weight
    and the sum it is divided by are each off by a factor of up to 1 + d
    beside the 2^-20 of the exponential: (2 d + 2^-20) A
  * the fp32 sums over L keys: (L + 8) 2^-23 A
  * a bf16 output is rounded once more: 2^-8 of the result
and lse by d, the sum over L keys and its own size.
"""

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd
from oracle import paged

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV = torch.device("cuda", 0)
DEV_OFFSETS, DEV_PAGE = 0x20, 0x40


@pytest.fixture(autouse=True)
def _status_clear():
    bd.device_status()
    yield
    torch.cuda.synchronize()
    assert bd.device_status() == 0


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bf16_rows(rng, shape, spread=1.0):
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return torch.from_numpy(x).to(torch.bfloat16)


class Batch:
    """A ragged batch whose pages lie in a random order in a pool that holds
    NaN wherever no row was stored."""

    def __init__(self, seed, lens, heads, dh, page, fp8, spare=3, spread=0.3, k_size=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.heads, self.dh, self.page, self.fp8 = list(lens), heads, dh, page, fp8
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)[:sum(need)]
        self.width = max(need + [1]) + 1
        table = np.full((len(lens), self.width), -1, np.int64)      # entries beyond a request's pages: never used
        for i, at in enumerate(np.cumsum([0] + need)[:-1]):
            table[i, :need[i]] = order[at:at + need[i]]
        self.table = i32(table)
        self.pages = bd.KVPages.empty(pages, page, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
        if fp8:
            for t in (self.pages.k, self.pages.v):
                t.view(torch.uint8).fill_(0x7F)
            self.pages.k_scale.fill_(255), self.pages.v_scale.fill_(255)
        else:
            self.pages.k.fill_(float("nan")), self.pages.v.fill_(float("nan"))
        off = np.cumsum([0] + self.lens)
        k = bf16_rows(rng, (off[-1], heads, dh), spread) * k_size
        v = bf16_rows(rng, (off[-1], heads, dh), spread)
        self.k_in, self.v_in = k.to(DEV), v.to(DEV)
        self.off = i32(off)
        bd.kv_write(self.pages, self.k_in, self.v_in, self.off, i32([0] * len(lens)), self.table)
        if fp8:
            k, v = (paged.restore(*paged.quantise(f64(t))) for t in (k, v))
        else:
            k, v = f64(k), f64(v)
        self.k = [k[off[i]:off[i + 1]] for i in range(len(lens))]
        self.v = [v[off[i]:off[i + 1]] for i in range(len(lens))]

    def queries(self, w, group, q_size=1.0, behind=0):
        self.w, self.group = list(w), group
        self.q_off = np.cumsum([0] + self.w)
        self.q = (bf16_rows(self.rng, (int(self.q_off[-1]) + behind, self.heads * group, self.dh), 0.2) * q_size).to(DEV)
        return self.q

    def run(self, pos=None, max_kv=None, **kw):
        return bd.paged_attn(self.q, self.pages, i32(self.q_off), i32(self.lens), self.table, max(self.w + [1]),
                             max_kv or max(self.lens + [1]), q_pos=i32(pos) if pos is not None else None, return_lse=True, **kw)

    def check(self, out, lse, pos=None, left=-1, right=-1, sinks=0, scale=None):
        scale = self.dh ** -0.5 if scale is None else scale
        fp32 = out.dtype == torch.float32
        out, lse = f64(out), f64(lse)
        for i, (w, n) in enumerate(zip(self.w, self.lens)):
            a, b = int(self.q_off[i]), int(self.q_off[i + 1])
            p = np.arange(w) + (n - w if pos is None else pos[i])
            want, z, absv, mag = paged.attention(f64(self.q[a:b]), self.k[i], self.v[i], p, scale, left, right, sinks)
            d = (self.dh + 8) * 2.0 ** -23 * mag
            tol = absv * (2.0 ** -8 + 2 * d[..., None] + 2.0 ** -20 + (n + 8) * 2.0 ** -23)
            tol = tol + (0 if fp32 else 2.0 ** -8 * (np.abs(want) + tol)) + 1e-38
            err = np.abs(out[a:b] - want)
            assert np.isfinite(out[a:b]).all(), f"request {i}: not finite"
            assert (err <= tol).all(), f"request {i} ({w} rows, {n} keys): {np.max(err / tol):.2f} of the tolerance"
            none = np.isinf(z)
            assert np.array_equal(none, np.isneginf(lse[a:b])), i
            zt = 2 * d + (n + 8) * 2.0 ** -23 + 2.0 ** -20 + 4 * 2.0 ** -23 * np.abs(np.where(none, 0, z))
            assert (np.abs(np.where(none, 0, lse[a:b] - np.where(none, 0, z))) <= zt).all(), f"lse of request {i}"


LENS = [0, 1, 17, 128, 129, 300, 15, 1000]

# ---------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads", [(64, 16, 3), (128, 32, 1), (128, 64, 8), (64, 128, 5)])
def test_write_stores_the_oracles_rows_and_nothing_else(dh, page, heads, fp8):
    rng = np.random.default_rng(dh + page)
    lens, w = [40, 1, 0, 129, 260], [7, 1, 0, 129, 101]
    b = Batch(3, lens, heads, dh, page, fp8)
    before = [t.clone() for t in (b.pages.k.view(torch.uint8), b.pages.v.view(torch.uint8))]
    off = np.cumsum([0] + w)
    both = bf16_rows(rng, (off[-1] + 2, 2, heads, dh), 2.0).to(DEV)          # K and V columns of one matrix, two rows behind
    pos0 = [n - m for n, m in zip(lens, w)]
    bd.kv_write(b.pages, both[:, 0], both[:, 1], i32(off), i32(pos0), b.table)
    table = b.table.cpu().numpy()
    for name, col in (("k", 0), ("v", 1)):
        pool = getattr(b.pages, name).view(torch.uint8).cpu().numpy()
        want = before[col].cpu().numpy()
        codes = both[:, col].cpu()
        scale = None
        if fp8:
            codes, scale = paged.quantise(f64(codes))
            sc = getattr(b.pages, name + "_scale").cpu().numpy()
        else:
            codes = codes.contiguous().view(torch.uint8).numpy()
        for i, m in enumerate(w):
            for t in range(m):
                u = pos0[i] + t
                pg, slot = table[i, u // page], u % page
                want[pg, :, slot] = codes[off[i] + t]
                if fp8:
                    assert np.array_equal(sc[pg, :, slot], scale[off[i] + t])
        assert np.array_equal(pool, want)


@pytest.mark.parametrize("dh", [64, 128])
def test_write_of_uncommon_values(dh):
    top = float(torch.finfo(torch.bfloat16).max)
    x = torch.zeros((9, 2, dh))
    x[1, 0, 3] = 2.0 ** -133                       # a bf16 subnormal
    x[2, 0, :4] = torch.tensor([top, -top, 1.0, -0.0])
    x[3, 0, 5], x[3, 0, 6], x[3, 0, 7] = float("inf"), -1.5, float("nan")
    x[4, :, :] = torch.linspace(-3, 3, dh)
    x[5, 0, :3] = torch.tensor([1.75, 17 / 256, 19 / 256])
    x[6, 1, dh - 1] = 1.7578125
    x[7, 0, 0] = 2.0 ** -117 * 448
    x[8, 1, :] = float("nan")
    x = x.to(torch.bfloat16)
    pages = bd.KVPages.empty(1, 16, 2, dh, torch.float8_e4m3fn, DEV)
    bd.kv_write(pages, x.to(DEV), x.flip(0).to(DEV), i32([0, 9]), i32([2]), i32([[0]]))
    for pool, scale, rows in ((pages.k, pages.k_scale, x), (pages.v, pages.v_scale, x.flip(0))):
        codes, b = paged.quantise(f64(rows))
        got = pool.view(torch.uint8).cpu().numpy()[0, :, 2:11].swapaxes(0, 1)
        assert np.array_equal(scale.cpu().numpy()[0, :, 2:11].T, b)
        assert np.array_equal(got[b < 255], codes[b < 255]) and (b == 255).sum() == 2
    k, _ = bd.kv_read(pages, i32([0, 9]), i32([2]), i32([[0]]), 9)
    codes, b = paged.quantise(f64(x))
    assert np.array_equal(f64(k), paged.restore(codes, b), equal_nan=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads", [(64, 32, 2), (128, 16, 3)])
def test_read_returns_what_the_rows_stand_for(dh, page, heads, fp8):
    b = Batch(4, LENS, heads, dh, page, fp8, spread=2.0)
    pos0 = [min(3, n) for n in LENS]
    off = np.cumsum([0] + [n - p for n, p in zip(LENS, pos0)])
    rows = int(off[-1]) + 2
    mark = torch.full((rows, heads, dh), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = bd.kv_read(b.pages, i32(off), i32(pos0), b.table, rows, k=mark.clone(), v=mark.clone())
    for got, want in ((k, b.k), (v, b.v)):
        got = f64(got)
        for i, p in enumerate(pos0):
            assert np.array_equal(got[off[i]:off[i + 1]], want[i][p:])
        assert (got[off[-1]:] == 7).all()


def test_bad_pages_and_positions_are_reported():
    b = Batch(5, [40, 40], 2, 64, 16, True)
    table = b.table.clone()
    table[0, 1] = 1 << 30
    table[1, 0] = -1
    x = b.k_in[:8]
    before = b.pages.k.view(torch.uint8).clone()
    bd.kv_write(b.pages, x, x, i32([0, 4, 8]), i32([16, 3]), table)             # both name a bad page
    bd.kv_write(b.pages, x, x, i32([0, 4, 8]), i32([-4, (1 << 31) - 2]), table)   # positions outside the table
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    assert torch.equal(before, b.pages.k.view(torch.uint8))
    k, v = bd.kv_read(b.pages, i32([0, 40, 80]), i32([0, 0]), table, 80)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    k = f64(k)
    assert np.array_equal(k[:16], b.k[0][:16]) and not k[16:32].any() and np.array_equal(k[32:40], b.k[0][32:])
    assert not k[40:56].any() and np.array_equal(k[56:], b.k[1][16:])
    # attention reads a bad page as zero rows
    b.queries([3, 2], 2)
    b.k[0][16:32] = b.v[0][16:32] = 0
    b.k[1][:16] = b.v[1][:16] = 0
    good, b.table = b.table, table
    out, lse = b.run(right=0)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    b.check(out, lse, right=0)
    b.table = good
    # rows beyond the buffers
    bd.kv_write(b.pages, x, x, i32([0, 4, 9]), i32([0, 0]), good)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

LARGE = 1 << 20     # a bound of the keys that makes the call a large one: row tiles of 256
MASKS = [(-1, -1, 0), (-1, 0, 0), (40, 0, 3), (200, 16, 0), (0, 0, 130), (5, -1, 1)]


@pytest.mark.parametrize("left,right,sinks", MASKS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group", [(64, 16, 2, 1), (128, 64, 2, 4), (128, 16, 1, 3)])
def test_single_tokens(dh, page, heads, group, fp8, left, right, sinks):
    b = Batch(10, LENS, heads, dh, page, fp8)
    b.queries([1 if n else 0 for n in LENS], group)
    b.check(*b.run(left=left, right=right, sinks=sinks), left=left, right=right, sinks=sinks)


@pytest.mark.parametrize("left,right,sinks", MASKS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group", [(64, 32, 2, 2), (128, 128, 1, 1), (128, 32, 2, 5)])
def test_blocks(dh, page, heads, group, fp8, left, right, sinks):
    # fewer, as many and more rows than keys: with more, the first rows lie before the cache
    b = Batch(11, LENS, heads, dh, page, fp8)
    b.queries([3, 5, 17, 32, 1, 33, 40, 24], group)
    b.check(*b.run(left=left, right=right, sinks=sinks), left=left, right=right, sinks=sinks)


@pytest.mark.parametrize("left,right,sinks", MASKS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group", [(64, 64, 1, 2), (128, 16, 1, 1), (128, 64, 1, 3)])
def test_chunks(dh, page, heads, group, fp8, left, right, sinks):
    b = Batch(12, [257, 90, 700, 0, 1500], heads, dh, page, fp8)
    b.queries([130, 200, 257, 150, 129], group)
    b.check(*b.run(left=left, right=right, sinks=sinks), left=left, right=right, sinks=sinks)


@pytest.mark.parametrize("group", [1, 2, 6, 8, 16, 64])
@pytest.mark.parametrize("w", [1, 2, 9, 31])
def test_row_counts(group, w):
    b = Batch(13, [200, 65], 1, 64, 16, False)
    b.queries([w, max(1, w - 1)], group)
    b.check(*b.run(right=0), right=0)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_keys_are_split_and_joined(fp8):
    b = Batch(14, [9001, 1, 5000], 2, 128, 64, fp8)
    b.queries([1, 1, 4], 4)
    b.check(*b.run(right=0), right=0)
    b.check(*b.run(left=3000, right=0, sinks=5), left=3000, right=0, sinks=5)
    b.check(*b.run(left=7, right=0, sinks=4900), left=7, right=0, sinks=4900)


@pytest.mark.parametrize("fp8", [False, True])
def test_given_positions_and_rows_that_see_nothing(fp8):
    b = Batch(15, [300, 64, 10, 500], 2, 64, 32, fp8)
    b.queries([20, 64, 5, 140], 2)
    pos = [100, -30, 400, 250]                       # inside, partly before, beyond the cache, inside
    for left, right, sinks in MASKS + [(3, 0, 0)]:
        b.check(*b.run(pos=pos, left=left, right=right, sinks=sinks), pos=pos, left=left, right=right, sinks=sinks)
    far = [1 << 30, -(1 << 31), (1 << 31) - 1, -5]
    lim = [1 << 30, -(1 << 30), 1 << 30, -5]
    b.check(*b.run(pos=far, left=100, right=0), pos=lim, left=100, right=0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [1, 40, 140])
def test_growing_scores_move_the_maximum(w, fp8):
    # later keys score far higher: the running maximum moves again and again
    b = Batch(16, [1000, 600], 1, 128, 64, fp8)
    b.queries([w, w], 2, q_size=0.0)
    b.q[:] = 2.0
    ramp = torch.linspace(-4, 4, 1000).repeat_interleave(1)
    rows = torch.cat([ramp, ramp[:600].flip(0)])[:, None, None].expand(-1, 1, 128).to(torch.bfloat16).contiguous()
    bd.kv_write(b.pages, rows.to(DEV), b.v_in, b.off, i32([0, 0]), b.table)
    k = paged.restore(*paged.quantise(f64(rows))) if fp8 else f64(rows)
    b.k = [k[:1000], k[1000:]]
    b.check(*b.run(right=0), right=0)
    b.check(*b.run(scale=-0.05), scale=-0.05)
    b.check(*b.run(scale=0.0), scale=0.0)


def test_scales_of_very_different_sizes():
    b = Batch(17, [700, 260], 2, 128, 16, True, spread=0.0)
    rng = np.random.default_rng(5)
    sizes = torch.from_numpy(2.0 ** rng.integers(-40, 20, size=(960, 2, 1))).float()
    v = (b.v_in.cpu().float() * sizes).to(torch.bfloat16)
    k = (b.k_in.cpu().float() * torch.from_numpy(2.0 ** rng.integers(-12, 2, size=(960, 2, 1))).float()).to(torch.bfloat16)
    bd.kv_write(b.pages, k.to(DEV), v.to(DEV), b.off, i32([0, 0]), b.table)
    k, v = (paged.restore(*paged.quantise(f64(t))) for t in (k, v))
    b.k, b.v = [k[:700], k[700:]], [v[:700], v[700:]]
    for w in ([1, 1], [30, 7], [140, 200]):
        b.queries(w, 2)
        b.check(*b.run(right=0), right=0)
        b.check(*b.run(left=0, right=0), left=0, right=0)      # every row sees one key alone


@pytest.mark.parametrize("w", [1, 16, 150])
@pytest.mark.parametrize("fp8", [False, True])
def test_one_far_key_takes_most_of_the_weight(w, fp8):
    # the rest, far below it, still adds up to a part that has to be right
    b = Batch(18, [4000], 1, 64, 64, fp8, spread=0.0, k_size=0.0)
    b.queries([w], 1, q_size=0.0)
    b.q[:] = 1.0
    k = torch.zeros((4000, 1, 64))
    k[0] = 1.25                                            # score 10 at scale 1/8: 2e4 times the others' weight
    v = torch.full((4000, 1, 64), 1.0)
    v[0] = 0.0
    bd.kv_write(b.pages, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), b.off, i32([0]), b.table)
    b.k, b.v = [k.double().numpy()], [v.double().numpy()]
    b.check(*b.run(out_fp32=True))


def test_output_types_strides_and_rows_behind():
    b = Batch(19, [100, 260], 2, 128, 32, False)
    b.queries([5, 40], 2, behind=3)
    fused = torch.empty((48, 3, 4, 128), dtype=torch.bfloat16, device=DEV)
    fused[:, 1] = b.q
    b.q = fused[:, 1]
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((48, 4, 128), 5.0, dtype=dtype, device=DEV)
        lse = torch.full((48, 4), 5.0, device=DEV)
        got, z = b.run(right=0, out=out, lse=lse)
        assert got is out and z is lse
        b.check(out, lse, right=0)
        assert (out[45:] == 5).all() and (lse[45:] == 5).all()


def test_out_of_bounds_metadata_is_clipped_and_reported():
    b = Batch(20, [100, 60], 1, 64, 16, False)
    b.queries([4, 6], 1)
    args = (b.pages, i32([0, 4, 11]), i32([100, 60]), b.table)
    out, lse = bd.paged_attn(b.q, *args, 7, 100, return_lse=True)           # one row more than q holds
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    b.check(out, lse)
    bd.paged_attn(b.q, b.pages, i32([0, 4, 10]), i32([200, 60]), b.table, 6, 128)   # more keys than max_kv, and than pages
    bd.paged_attn(b.q, b.pages, i32([0, 4, 10]), i32([-3, 60]), b.table, 6, 100)
    bd.paged_attn(b.q, b.pages, i32([8, 4, 2]), i32([100, 60]), b.table, 6, 100)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS | DEV_PAGE


@pytest.mark.parametrize("w", [1, 20])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_hold_nan_reach_what_sees_them(w, fp8):
    b = Batch(29, [700], 2, 64, 16, fp8)
    b.queries([w], 2)
    k, v = b.k_in.clone(), b.v_in.clone()
    k[600, 0, 3] = float("nan")
    v[300, 1, 5] = float("inf")
    bd.kv_write(b.pages, k, v, b.off, i32([0]), b.table)
    b.k[0][600] = b.v[0][300] = 0
    p = np.arange(700 - w, 700)
    for left in (-1, 250):
        out, lse = b.run(left=left, right=0)
        out = f64(out)
        see = paged.visible(p, 700, left, 0, 0)
        assert np.array_equal(np.isnan(out[:, :2]).any(-1).all(-1), see[:, 600])      # heads of cached head 0
        assert np.array_equal(np.isnan(f64(lse)[:, 0]), see[:, 600])
        assert np.array_equal(~np.isfinite(out[:, 2:]).all(-1).all(-1), see[:, 300])
        if not fp8:
            assert np.array_equal(np.isposinf(out[:, 2, 5]), see[:, 300])


@pytest.mark.parametrize("w", [1, 32, 300])
@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_every_time(w, fp8):
    b = Batch(21, [3000, 700, 40], 2, 128, 64, fp8)
    b.queries([w, w, min(w, 40)], 4)
    first = b.run(right=0)
    for _ in range(3):
        again = b.run(right=0)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("w", [1, 200])
def test_captured_calls_follow_the_device_metadata(w):
    b = Batch(22, [900, 300], 2, 64, 32, True)
    b.queries([w, w], 2)
    q_off, kv_len = i32(b.q_off), i32(b.lens)
    ws = bd._binding.workspace(bd.paged_attn_workspace(b.pages, 2, 4, w, 1000))
    out = torch.empty((2 * w, 4, 64), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((2 * w, 4), device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call = lambda: bd.paged_attn(b.q, b.pages, q_off, kv_len, b.table, w, 1000, right=0, out=out, lse=lse, ws=ws)  # noqa: E731
        call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    lens, k, v = b.lens, b.k, b.v
    for cut in ([900, 300], [411, 300], [w, 0], [1, 129]):
        kv_len.copy_(i32(cut))
        ws.random_(0, 255)                       # nothing of the workspace is kept between calls
        g.replay()
        torch.cuda.synchronize()
        b.lens, b.k, b.v = cut, [x[:n] for x, n in zip(k, cut)], [x[:n] for x, n in zip(v, cut)]
        b.check(out, lse, right=0)
    b.lens, b.k, b.v = lens, k, v


def test_calls_on_two_streams_at_once():
    b = [Batch(23 + i, [4000, 900], 2, 128, 64, i == 1) for i in range(2)]
    for x, w in zip(b, (1, 130)):
        x.queries([w, w], 4)
    want = [x.run(right=0) for x in b]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    got = []
    meta = [(i32(x.q_off), i32(x.lens)) for x in b]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s, (off, n) in zip(b, streams, meta):
            got.append(bd.paged_attn(x.q, x.pages, off, n, x.table, max(x.w), 4000, right=0, return_lse=True, stream=s))
    torch.cuda.synchronize()
    for n, (out, lse) in enumerate(got):
        assert torch.equal(out, want[n % 2][0]) and torch.equal(lse, want[n % 2][1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [1, 140])
def test_rows_far_into_a_large_pool(w, fp8):
    # byte offsets beyond 2^32: the last pages of a pool of over 8 GB
    page, heads, dh = 128, 4, 128
    n = (9 << 30) // (heads * page * dh * (1 if fp8 else 2))
    pages = bd.KVPages.empty(n, page, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
    b = Batch(25, [300], heads, dh, page, fp8)
    b.pages, b.table = pages, i32([[n - 1, n // 2 + 1, n - 2]])
    bd.kv_write(pages, b.k_in, b.v_in, b.off, i32([0]), b.table)
    k, v = bd.kv_read(pages, b.off, i32([0]), b.table, 300)
    assert np.array_equal(f64(k), b.k[0]) and np.array_equal(f64(v), b.v[0])
    b.queries([w], 2)
    b.check(*b.run(right=0), right=0)


def test_empty_calls_touch_nothing():
    b = Batch(26, [20], 1, 64, 16, False)
    none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    bd.kv_write(b.pages, none, none, i32([0, 0]), i32([0]), b.table)
    k, v = bd.kv_read(b.pages, i32([0, 0]), i32([0]), b.table, 0)
    out, lse = bd.paged_attn(none, b.pages, i32([0, 0]), i32([20]), b.table, 1, 20, return_lse=True)
    assert k.shape == v.shape == out.shape == (0, 1, 64) and lse.shape == (0, 1)


def test_binding_refusals():
    b = Batch(27, [20], 2, 64, 16, False)
    b.queries([3], 1)
    off, pos, n = i32([0, 3]), i32([0]), i32([20])
    with pytest.raises(TypeError):
        bd.kv_write(b.pages, b.q.float(), b.q, off, pos, b.table)
    with pytest.raises(ValueError):
        bd.kv_write(b.pages, b.q[..., ::2], b.q[..., ::2], off, pos, b.table)
    with pytest.raises(ValueError):
        bd.kv_write(b.pages, b.q.transpose(0, 1).contiguous().transpose(0, 1), b.q, off, pos, b.table)
    with pytest.raises(ValueError):
        bd.kv_write(b.pages, b.q, b.q[:2], off, pos, b.table)
    with pytest.raises(TypeError):
        bd.kv_write(b.pages, b.q, b.q, off.long(), pos, b.table)
    with pytest.raises(ValueError):
        bd.kv_write(b.pages, b.q, b.q, off, i32([0, 0]), b.table)
    with pytest.raises(ValueError):
        bd.paged_attn(b.q, b.pages, off, n, b.table[0], 3, 20)
    with pytest.raises(bd.DllmError):
        bd.paged_attn(b.q[:, :1], b.pages, off, n, b.table, 3, 20)          # fewer query heads than cached heads
    with pytest.raises(ValueError):
        bd.paged_attn(b.q, b.pages, off, n, b.table, 3, 20, out=torch.empty((3, 2, 64), device=DEV, dtype=torch.float16))
    with pytest.raises(TypeError):
        bd.paged_attn(b.q.cpu(), b.pages, off, n, b.table, 3, 20)



@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
def test_page_sizes_with_every_row_tile(dh, fp8, page):
    b = Batch(30, [650, 31, 129], 2, dh, page, fp8)
    for w, group in (([1, 1, 1], 3), ([9, 2, 8], 3), ([11, 40, 33], 3), ([140, 50, 129], 2)):
        b.queries(w, group)
        b.check(*b.run(left=150, right=0, sinks=20), left=150, right=0, sinks=20)
        b.check(*b.run())


@pytest.mark.parametrize("w", [1, 12, 40, 300])
@pytest.mark.parametrize("fp8", [False, True])
def test_leaps_of_the_scores(w, fp8):
    """Single keys whose scores lie 2^40 and more above all before them, in
    either half of a tile, first and last ones among them; some rows have them
    the other way round and see weights that vanish."""
    at = [0, 1, 31, 32, 63, 64, 100, 127, 128, 190, 200, 255, 256, 300, 383, 400, 511, 512, 600, 690]
    b = Batch(31, [700, 460], 1, 64, 64, fp8)
    b.queries([w, w], 2)
    b.q[:] = torch.where(torch.arange(2 * w, device=DEV) % 3 == 1, -0.5, 1.0)[:, None, None].to(torch.bfloat16)
    k = torch.zeros((1160, 1, 64))
    for n, u in enumerate(at):
        k[u] = 4.0 * n                                   # scores 32 n apart at scale 1/8: 2^46
        if u < 460:
            k[700 + 459 - u] = 4.0 * n
    k = k.to(torch.bfloat16)
    bd.kv_write(b.pages, k.to(DEV), b.v_in, b.off, i32([0, 0]), b.table)
    k = paged.restore(*paged.quantise(f64(k))) if fp8 else f64(k)
    b.k = [k[:700], k[700:]]
    for max_kv in (None, LARGE) if w == 300 else (None,):
        for left in (-1, 130):
            b.check(*b.run(left=left, right=0, max_kv=max_kv), left=left, right=0)
        b.check(*b.run(max_kv=max_kv))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [1, 12, 40, 200])
def test_large_values_do_not_overflow(w, fp8):
    # weights of up to 2^32 relative to a lagging reference, values of 2^60
    b = Batch(32, [500], 1, 128, 32, fp8)
    b.queries([w], 1, q_size=0.0)
    b.q[:] = 2.0
    k = torch.linspace(-1, 1, 500)[:, None, None].expand(-1, 1, 128).to(torch.bfloat16).contiguous()
    v = (b.v_in.float() * 2.0 ** 60).to(torch.bfloat16)
    bd.kv_write(b.pages, k.to(DEV), v, b.off, i32([0]), b.table)
    k, v = f64(k), f64(v)
    b.k, b.v = ([paged.restore(*paged.quantise(x))] if fp8 else [x] for x in (k, v))
    b.check(*b.run(right=0), right=0)
    b.check(*b.run(right=0, max_kv=LARGE), right=0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,most", [(4096, 1), (700, 7), (300, 60)])
def test_many_requests(B, most, fp8):
    # more than threads of a block, requests without rows or keys among them
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 180, B) * (rng.random(B) < 0.8)
    b = Batch(33, [int(n) for n in lens], 1, 64, 16, fp8)
    b.queries([int(x) for x in rng.integers(0, most + 1, B)], 2)
    b.check(*b.run(right=0), right=0)
    lens[B // 2] = 0
    b.check(*b.run(left=50, right=0, sinks=2), left=50, right=0, sinks=2)


@pytest.mark.parametrize("left,right,sinks", MASKS)
@pytest.mark.parametrize("fp8", [False, True])
def test_single_tokens_beside_pieces_of_prompts(fp8, left, right, sinks):
    b = Batch(34, [900, 333, 1, 50, 2100, 128, 600], 2, 128, 64, fp8)
    b.queries([290, 1, 1, 0, 1, 64, 1], 2)
    b.check(*b.run(left=left, right=right, sinks=sinks), left=left, right=right, sinks=sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [1, 40])
def test_bounds_far_above_the_batch(w, fp8):
    # max_q and max_kv as a server that serves every batch with one graph gives them
    b = Batch(35, [300, 5, 40], 2, 64, 16, fp8)
    b.queries([w, 1, 3], 2)
    table = torch.full((3, 1 << 12), -1, dtype=torch.int32, device=DEV)
    table[:, :b.width] = b.table
    got = bd.paged_attn(b.q, b.pages, i32(b.q_off), i32(b.lens), table, 5000, 1 << 16, right=0, return_lse=True)
    b.check(*got, right=0)


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_with_a_workspace_each(fp8):
    bs = [Batch(36 + i, [3500, 700], 2, 64, 32, fp8) for i in range(2)]
    runs = []
    for b, w in zip(bs, (1, 70)):
        b.queries([w, w], 2)
        args = (b.q, b.pages, i32(b.q_off), i32(b.lens), b.table, w, 4000)
        want = bd.paged_attn(*args, right=0, return_lse=True)
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            got = bd.paged_attn(*args, right=0, return_lse=True)      # its workspace lives in the graph's pool
        runs.append((s, g, want, got, args))
    for _ in range(20):
        for s, g, _, _, _ in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, want, got, _ in runs:
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("w", [1, 12, 40, 200])
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_in_one_head_of_one_request_stays_there(w, fp8):
    b = Batch(38, [400, 300, 350], 2, 64, 16, fp8)
    b.queries([w, w, w], 2)
    k, v = b.k_in.clone(), b.v_in.clone()
    k[410, 0, 7], v[420, 0, 9] = float("nan"), float("-inf")              # request 1, head 0
    bd.kv_write(b.pages, k, v, b.off, i32([0, 0, 0]), b.table)
    out, lse = b.run()
    assert not torch.isfinite(out[w:2 * w, :2]).all(-1).any()
    out[w:2 * w, :2], lse[w:2 * w, :2] = 0, 0
    b2 = Batch(38, [400, 300, 350], 2, 64, 16, fp8)
    b2.queries([w, w, w], 2)
    want, z = b2.run()
    want[w:2 * w, :2], z[w:2 * w, :2] = 0, 0
    assert torch.equal(out, want) and torch.equal(lse, z)                 # the rest has the same bits


@pytest.mark.parametrize("left,right,sinks", MASKS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group", [(64, 64, 1, 2), (128, 16, 1, 1), (128, 128, 2, 3)])
def test_chunks_of_large_calls(dh, page, heads, group, fp8, left, right, sinks):
    b = Batch(40, [257, 90, 700, 0, 1500, 60], heads, dh, page, fp8)
    b.queries([130, 200, 257, 150, 129, 20], group)
    b.check(*b.run(left=left, right=right, sinks=sinks, max_kv=LARGE), left=left, right=right, sinks=sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
def test_large_calls_with_many_pieces_each(dh, fp8):
    # CTAs go from item to item, between those with up to 128 rows and those with more
    rng = np.random.default_rng(41)
    lens, w = [int(n) for n in rng.integers(0, 800, 90)], [int(n) for n in rng.choice([1, 40, 64, 65, 100, 128, 129, 300], 90)]
    b = Batch(41, lens, 2, dh, 32, fp8)
    b.queries(w, 2)
    for max_kv in (LARGE, None):
        b.check(*b.run(right=0, max_kv=max_kv), right=0)
        b.check(*b.run(left=100, right=30, sinks=140, max_kv=max_kv), left=100, right=30, sinks=140)


@pytest.mark.parametrize("w", [3, 12, 40, 200])
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_and_infinite_queries_stay_in_their_rows(w, fp8):
    b = Batch(42, [600, 250], 2, 64, 32, fp8)
    b.queries([w, w], 2)
    want, z = b.run(right=0)
    q = b.q.clone()
    b.q[1, 2, 5], b.q[w + 2, 0, 9] = float("nan"), float("inf")
    out, lse = b.run(right=0)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2]) and torch.isnan(out[w + 2, 0]).all()
    b.q = q
    for t, good in ((out, want), (lse, z)):
        t[1, 2], t[w + 2, 0] = good[1, 2], good[w + 2, 0]
    b.check(out, lse, right=0)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_most_heads(fp8):
    b = Batch(43, [3, 140], 256, 64, 16, fp8)
    k, v = bd.kv_read(b.pages, b.off, i32([0, 0]), b.table, 143)
    assert np.array_equal(f64(k), np.concatenate(b.k)) and np.array_equal(f64(v), np.concatenate(b.v))
    for w in ([1, 2], [0, 20], [3, 129]):
        b.queries(w, 1)
        b.check(*b.run(right=0), right=0)


@pytest.mark.parametrize("w", [1, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_requests_that_share_pages(w, fp8):
    # the first 256 keys of both are the first request's, one of whose pages is named twice
    b = Batch(44, [700, 500], 2, 64, 64, fp8)
    b.table[1, :4] = b.table[0, :4]
    b.table[0, 5] = b.table[0, 2]
    b.k[1][:256], b.v[1][:256] = b.k[0][:256], b.v[0][:256]
    b.k[0][320:384], b.v[0][320:384] = b.k[0][128:192], b.v[0][128:192]
    b.queries([w, w], 2)
    b.check(*b.run(right=0), right=0)


@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(100 + seed)
    pick = lambda *x: x[rng.integers(len(x))]  # noqa: E731
    B, top = int(pick(1, 2, 5, 40, 150)), int(pick(3, 130, 700, 2500))
    lens = [int(n) for n in rng.integers(0, max(2, top // max(1, B // 20)), B)]
    b = Batch(200 + seed, lens, int(pick(1, 2, 3)), int(pick(64, 128)), int(pick(16, 32, 64, 128)), bool(pick(0, 1)))
    for _ in range(2):
        b.queries([int(x) for x in rng.integers(0, pick(2, 2, 10, 40, 140, 330) if B < 40 else pick(2, 10, 70), B)], int(pick(1, 2, 4, 5, 7)))
        mask = dict(left=int(pick(-1, 0, 9, 127, 128, 600)), right=int(pick(-1, 0, 0, 5, 200)), sinks=int(pick(0, 1, 4, 129, 1000)))
        pos = [int(x) for x in rng.integers(-50, top + 50, B)] if pick(0, 0, 1) else None
        b.check(*b.run(pos=pos, max_kv=pick(None, LARGE), out_fp32=bool(pick(0, 1)), **mask), pos=pos, **mask)


@pytest.mark.parametrize("name", ["max_q", "max_kv", "left", "right", "sinks"])
def test_numbers_beyond_32_bits_are_refused(name):
    b = Batch(39, [20], 1, 64, 16, False)
    b.queries([3], 1)
    kw = {"max_q": 3, "max_kv": 20, "left": -1, "right": -1, "sinks": 0, name: (1 << 32) + 3}
    with pytest.raises(ValueError):
        bd.paged_attn(b.q, b.pages, i32([0, 3]), i32([20]), b.table, **kw)
    if name in ("max_q", "max_kv"):
        with pytest.raises(ValueError):
            bd.paged_attn_workspace(b.pages, 1, 1, kw["max_q"], kw["max_kv"])

@pytest.mark.parametrize("fp8", [False, True])
def test_a_run_of_them_together(fp8):
    """Prompt pieces and single tokens as a server runs them: each piece's K/V
    enter the cache and its rows attend over it; at the end the whole cache is
    read back and contiguous block attention over it agrees."""
    rng = np.random.default_rng(28)
    H, G, dh, page, total = 2, 2, 64, 32, [333, 150]
    b = Batch(28, total, H, dh, page, fp8)
    pages = b.pages
    for t in (pages.k, pages.v):
        t.view(torch.uint8).fill_(0x7F)
    done = [0, 0]
    last = None
    for piece in ([200, 31], [100, 100], [1, 1], [1, 0], [31, 18]):
        off = np.cumsum([0] + piece)
        rows = [slice(o, o + n) for o, n in zip(np.cumsum([0] + total)[:-1] + done, piece)]
        k = torch.cat([b.k_in[r] for r in rows])
        v = torch.cat([b.v_in[r] for r in rows])
        q = bf16_rows(rng, (int(off[-1]), H * G, dh)).to(DEV)
        bd.kv_write(pages, k, v, i32(off), i32(done), b.table)
        done = [d + n for d, n in zip(done, piece)]
        out, lse = bd.paged_attn(q, pages, i32(off), i32(done), b.table, max(piece), max(done), right=0, return_lse=True)
        c = Batch.__new__(Batch)
        c.lens, c.w, c.q_off, c.q, c.dh, c.heads = done, piece, off, q, dh, H
        c.k, c.v = [x[:n] for x, n in zip(b.k, done)], [x[:n] for x, n in zip(b.v, done)]
        c.check(out, lse, right=0)
        last = q, off
    assert done == total
    k, v = bd.kv_read(pages, b.off, i32([0, 0]), b.table, sum(total))
    q, off = last
    both = bd.paged_attn(q, pages, i32(off), i32(total), b.table, 31, 333)
    rep = lambda t: t.repeat_interleave(G, dim=1).contiguous()  # noqa: E731
    block = bd.block_attn(q, rep(k), rep(v), i32(off), b.off, 31, 333)
    # two bf16 results, each within its own roundings of the same sum
    d = (both.float() - block.float()).abs()
    top = torch.stack([x.abs().float().amax() for x in (k, v)]).max()
    assert (d <= 4 * 2.0 ** -8 * top).all()
