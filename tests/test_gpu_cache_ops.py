"""GPU parity of the operators around the paged cache against the float64
oracle. Moves, evictions and tree masks are exact; attention over trees is held
to the bound that test_gpu_paged.py derives.

Rotation: an angle is off by at most pi 2^-24 (its rounding, in half turns), and
sine and cosine by 2 units of the last bit beside: 2^-21 in all. A result is two
products and a sum: 2^-21 (|x| + |y|) from the factors and 3 * 2^-24 (|x| + |y|)
from the arithmetic, within 2^-20 (|x| + |y|); then one rounding, 2^-8 of it for
bf16, or half an e4m3 step: 2^-4 of it, 2^-10 of the scale at least.
Mass: a weight is off by what the oracle gives with it, a sum of n weights by
(n + 8) 2^-23 of itself, and the old value's product by 2^-24 of it.
"""

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd
from oracle import cache_ops, paged
from test_gpu_paged import DEV, DEV_OFFSETS, DEV_PAGE, Batch, bf16_rows, f64, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV_TREE = 0x80
LENS = [0, 1, 17, 128, 129, 300, 15, 1000]


@pytest.fixture(autouse=True)
def _status_clear():
    bd.device_status()
    yield
    torch.cuda.synchronize()
    assert bd.device_status() == 0


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rope_case(rng, rows, heads, group, dh, spread=1.0):
    both = bf16_rows(rng, (rows, (group + 2) * heads, dh), spread).to(DEV)
    g = group * heads
    return both[:, :g], both[:, g:g + heads], both[:, g + heads:]


def pool_rows(b, name, table, page, i, pos):
    """The cached rows of request i at `pos` as (values [n][heads][dh], scale bytes or None)."""
    at = [(int(table[i, u // page]), u % page) for u in pos]
    pool = getattr(b, name)
    x = np.stack([f64(pool[p, :, s].float() if pool.dtype != torch.bfloat16 else pool[p, :, s]) for p, s in at])
    if b.k_scale is None:
        return x, None
    sc = np.stack([getattr(b, name + "_scale")[p, :, s].cpu().numpy() for p, s in at])
    return x * 2.0 ** (sc.astype(np.float64) - 127)[..., None], sc


def check_turned(got, want, size, scale=None):
    """got against want, size = |x| + |y| of each pair's elements; scale: bytes of 8-bit rows."""
    tol = 2.0 ** -20 * size
    if scale is None:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134
    else:
        step = 2.0 ** (scale.astype(np.float64) - 127)[..., None]
        tol = tol + np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * step)
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / tol))


def pair_sizes(x, half):
    s = np.abs(x)
    out = np.zeros_like(s)
    out[..., :half] = out[..., half:2 * half] = s[..., :half] + s[..., half:2 * half]
    out[..., 2 * half:] = s[..., 2 * half:]
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group,rot,axes,interleaved", [
    (64, 16, 3, 2, 64, 1, False), (128, 32, 1, 5, 128, 3, False), (128, 64, 8, 1, 64, 3, True), (64, 128, 5, 4, 16, 4, True),
    (128, 16, 2, 3, 48, 2, False), (64, 32, 4, 1, 0, 1, False)])
def test_rotated_rows_and_what_is_stored(dh, page, heads, group, rot, axes, interleaved, fp8):
    rng = np.random.default_rng(dh + rot + axes)
    w, lens = [7, 1, 0, 129, 40], [40, 1, 3, 129, 260]
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + 2)
    table = np.full((5, max(need)), -1)
    for i, a in enumerate(np.cumsum([0] + need)[:-1]):
        table[i, :need[i]] = order[a:a + need[i]]
    p = bd.KVPages.empty(sum(need) + 2, page, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
    p.k.view(torch.uint8).fill_(0x55), p.v.view(torch.uint8).fill_(0x55)
    if fp8:
        p.k_scale.fill_(99), p.v_scale.fill_(99)
    before = [p.k.view(torch.uint8).clone(), p.v.view(torch.uint8).clone()]
    off = np.cumsum([0] + w)
    rows = int(off[-1]) + 2                                   # two rows behind
    q, k, v = rope_case(rng, rows, heads, group, dh)
    half = rot // 2
    axis = [j % axes if interleaved else min(j * axes // max(half, 1), axes - 1) for j in range(half)] if half else []
    n_axes = max(axis, default=0) + 1
    pos = rng.integers(-1000, 40000, (n_axes, rows))
    pos[:, 3], pos[0, 9], pos[0, 10] = 0, 2 ** 31 - 1, -2 ** 31
    pos[0, 20:40] = rng.integers(10 ** 6, 10 ** 7, 20)
    freq = [10000.0 ** (-2.0 * j / max(rot, 1)) for j in range(half)]
    q_out = torch.full((rows, heads * group, dh), 7.0, dtype=torch.bfloat16, device=DEV)
    got = bd.rope_kv_write(p, bd.Rope(dh, axis, freq), i32(pos), q, k, v, i32(off), i32([n - m for n, m in zip(lens, w)]), i32(table),
                           q_out=q_out)
    assert got is q_out
    n = int(off[-1])
    check_turned(f64(got[:n]), cache_ops.rotate(f64(q), pos, axis, freq)[:n], pair_sizes(f64(q), half)[:n])
    assert (f64(got[n:]) == 7).all()
    want = cache_ops.rotate(f64(k), pos, axis, freq)
    size = pair_sizes(f64(k), half)
    seen = np.zeros((sum(need) + 2, page), bool)
    for i, m in enumerate(w):
        at = range(lens[i] - m, lens[i])
        if not m:
            continue
        kr, sc = pool_rows(p, "k", table, page, i, at)
        a, b = off[i], off[i + 1]
        check_turned(kr, want[a:b], size[a:b], sc)
        if fp8:
            # the least power of two, but where the row's largest element is next to a border
            top = np.abs(want[a:b]).max(-1) / 448
            e = sc.astype(np.float64) - 127
            slack = 1 + 2.0 ** -18 * (1 + size[a:b].max(-1) / np.maximum(np.abs(want[a:b]).max(-1), 1e-30))
            assert (top <= 2.0 ** e * slack).all() and ((top >= 2.0 ** (e - 1) / slack) | (sc == 10)).all()
        vr, sc = pool_rows(p, "v", table, page, i, at)
        rows_v = f64(v)[a:b]
        if fp8:
            codes, sb = paged.quantise(rows_v)
            assert np.array_equal(sb, sc) and np.array_equal(vr, paged.restore(codes, sb))
        else:
            assert np.array_equal(vr, rows_v)
        for u in at:
            seen[table[i, u // page], u % page] = True
    for name, was in (("k", before[0]), ("v", before[1])):      # nothing else is written
        now = getattr(p, name).view(torch.uint8).cpu().numpy()
        assert np.array_equal(now.swapaxes(1, 2)[~seen], was.cpu().numpy().swapaxes(1, 2)[~seen])


def test_rotation_in_place_without_q_and_of_uncommon_rows():
    rng = np.random.default_rng(5)
    q, k, v = rope_case(rng, 9, 2, 2, 64)
    rope = bd.Rope.standard(64, sections=[8, 12, 12])
    pos = i32(rng.integers(0, 3000, (3, 9)))
    args = (i32([0, 9]), i32([2]), i32([[0]]))
    k = k.clone()
    k[1, 0, 3], k[2, 1, 5], k[3] = float("inf"), float("nan"), 0
    k[4, 0, :] = 2.0 ** -120
    for fp8 in (False, True):
        p, p2 = (bd.KVPages.empty(1, 16, 2, 64, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV) for _ in range(2))
        for x in (p, p2):
            x.k.view(torch.uint8).zero_(), x.v.view(torch.uint8).zero_()
            if fp8:
                x.k_scale.zero_(), x.v_scale.zero_()
        want = bd.rope_kv_write(p, rope, pos, q, k, v, *args)
        both = q.clone()
        assert bd.rope_kv_write(p2, rope, pos, both, k, v, *args, q_out=both) is both and torch.equal(both, want)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in ((p.k, p2.k), (p.v, p2.v)))
        assert bd.rope_kv_write(p2, rope, pos, None, k, v, *args) is None
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in ((p.k, p2.k), (p.v, p2.v)))
        if fp8:
            sc = p.k_scale.cpu().numpy()[0]
            assert sc[0, 3] == 255 and sc[1, 4] == 255 and (sc == 255).sum() == 2 and sc[0, 5] == 10
        else:
            bad = ~torch.isfinite(p.k[0, :, 2:11].float()).all(-1)
            assert bad[0, 1] and bad[1, 2] and bad.sum() == 2


def test_far_positions_turn_by_the_exact_angle():
    # a pair (1, 0) turns to (cos, sin); fp32 products would be off by up to 2^31 * 2^-24 radians
    pos = np.array([[0, 1, 10 ** 6 + 1, 10 ** 7 + 3, 2 ** 31 - 1, -2 ** 31, -5, 123456789]])
    freq = [1.0, 0.75, 1e-3, 1e-6, 1000.0, -0.3, 1 / 3, 2.0 ** -30]
    x = torch.zeros((8, 1, 64), dtype=torch.bfloat16, device=DEV)
    x[..., :8] = 1
    p = bd.KVPages.empty(1, 16, 1, 64, torch.bfloat16, DEV)
    out = bd.rope_kv_write(p, bd.Rope(64, [0] * 8, freq), i32(pos), x, x, x, i32([0, 8]), i32([0]), i32([[0]]))
    # the angle in exact integers: freq is a dyadic fraction
    from fractions import Fraction
    from math import cos, pi, sin
    two_pi = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)
    for r in range(8):
        for j, f in enumerate(freq):
            a = float((Fraction(f) * int(pos[0, r])) % two_pi)
            a = a - 2 * pi if a > pi else a
            got = f64(out)[r, 0, [j, 8 + j]]
            tol = 2.0 ** -8 * np.abs([cos(a), sin(a)]) + 2.0 ** -20
            assert (np.abs(got - [cos(a), sin(a)]) <= tol).all(), (pos[0, r], f)


def test_rope_reports_rows_without_a_place():
    rng = np.random.default_rng(6)
    q, k, v = rope_case(rng, 6, 1, 1, 64)
    p = bd.KVPages.empty(2, 16, 1, 64, torch.bfloat16, DEV)
    p.k.zero_()
    rope = bd.Rope.standard(64)
    out = bd.rope_kv_write(p, rope, i32(range(6)), q, k, v, i32([0, 3, 6]), i32([15, -2]), i32([[0, 9], [1, 0]]))
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    want = cache_ops.rotate(f64(q), [range(6)], [0] * 32, [10000.0 ** (-j / 32) for j in range(32)])
    check_turned(f64(out), want, pair_sizes(f64(q), 32))       # q turns all the same
    used = p.k.float().abs().sum((1, 3)).cpu().numpy() > 0
    assert used[0, 15] and used[1, 0] and used.sum() == 2
    bd.rope_kv_write(p, rope, i32(range(6)), q, k, v, i32([0, 7]), i32([0]), i32([[0]]))
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------

def tree(rng, n, kind):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    return [int(rng.integers(-1, t)) if rng.random() < 0.9 else -1 for t in range(n)]


def unpack(mask, n):
    """[rows][n] truth values of a mask's bits."""
    m = mask.cpu().numpy().view(np.uint32)
    return np.stack([(m[:, c // 32] >> np.uint32(c % 32)) & 1 for c in range(n)], 1).astype(bool) if n else np.zeros((len(m), 0), bool)


@pytest.mark.parametrize("kind", ["chain", "star", "any"])
def test_masks_and_depths(kind):
    rng = np.random.default_rng(8)
    w = [1, 0, 5, 32, 33, 200, 64, 1024, 31]
    par = [tree(rng, n, kind) for n in w]
    off = np.cumsum([0] + w)
    mask = torch.full((int(off[-1]) + 1, 34), -1, dtype=torch.int32, device=DEV)
    parent = i32(sum(par, []) + [0])
    got, depth = bd.tree_mask(parent, i32(off), 1024, mask=mask)
    assert got is mask and (mask[-1] == -1).all() and (mask[:, 32:] == -1).all()
    bits, depth = unpack(mask, 1024), depth.cpu().numpy()
    for i, n in enumerate(w):
        see = cache_ops.ancestors(par[i])
        assert np.array_equal(bits[off[i]:off[i + 1], :n], see) and not bits[off[i]:off[i + 1], n:].any()
        assert np.array_equal(depth[off[i]:off[i + 1]], see.sum(1) - 1)


def test_bad_trees_are_reported():
    mask, depth = bd.tree_mask(i32([0, 0, 7, -2, 1]), i32([0, 5]), 5)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_TREE
    assert np.array_equal(unpack(mask, 5), cache_ops.ancestors([-1, 0, -1, -1, 1])) and depth.tolist() == [0, 1, 0, 0, 2]
    mask, _ = bd.tree_mask(i32([-1, 0, 1, 2, 3, 4]), i32([0, 6]), 4, mask=torch.zeros((6, 1), dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS                   # more tokens than max_q: the first four
    assert mask.view(-1).tolist() == [1, 3, 7, 15, 0, 0]


class Drafts(Batch):
    def drafts(self, w, group, seed, kind="any", q_size=1.0, behind=0):
        rng = np.random.default_rng(seed)
        self.queries(w, group, q_size, behind)
        self.parents = [tree(rng, n, kind) for n in w]
        self.mask, self.depth = bd.tree_mask(i32(sum(self.parents, []) + [-1] * behind), i32(self.q_off), max(w + [1]))

    def run_tree(self, mask=None, **kw):
        return bd.tree_attn(self.q, self.pages, i32(self.q_off), i32(self.lens), self.table, self.mask if mask is None else mask,
                            max(self.w + [1]), max(self.lens + [1]), return_lse=True, **kw)

    def check_tree(self, out, lse, see=None):
        self.see = [cache_ops.tree_visible(cache_ops.ancestors(p) if see is None else see[i], n)
                    for i, (p, n) in enumerate(zip(self.parents, self.lens))]
        real = paged.attention
        try:
            todo = iter([s for s in self.see])
            paged.attention = lambda q, k, v, p, scale, *a: real(q, k, v, p, scale, see=next(todo))
            self.check(out, lse)
        finally:
            paged.attention = real


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group,w", [
    (64, 16, 2, 1, [0, 1, 16, 5, 12, 13, 15, 16]), (128, 32, 1, 4, [0, 1, 4, 3, 4, 2, 1, 4]),
    (128, 64, 2, 2, [0, 1, 16, 9, 16, 13, 15, 7]), (64, 128, 1, 7, [0, 1, 4, 3, 4, 2, 1, 4]),
    (64, 32, 2, 32, [0, 1, 1, 1, 1, 1, 1, 1])])
def test_few_drafted_tokens(dh, page, heads, group, w, fp8):
    b = Drafts(20 + dh, LENS, heads, dh, page, fp8)
    b.drafts(w, group, 3)
    b.check_tree(*b.run_tree())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group,w", [
    (64, 16, 2, 1, [0, 1, 17, 64, 100, 33, 15, 40]), (128, 32, 1, 4, [0, 1, 9, 128, 129, 64, 15, 63]),
    (128, 64, 2, 3, [0, 1, 17, 90, 128, 200, 15, 300]), (64, 128, 1, 8, [0, 0, 17, 31, 33, 64, 15, 1000]),
    (128, 128, 1, 64, [0, 1, 2, 3, 4, 2, 1, 4])])
def test_many_drafted_tokens(dh, page, heads, group, w, fp8):
    b = Drafts(30 + dh, LENS, heads, dh, page, fp8)
    b.drafts(w, group, 4, behind=2)
    out = torch.full((b.q.shape[0], heads * group, dh), 7.0, dtype=torch.float32, device=DEV)
    lse = torch.full((b.q.shape[0], heads * group), 7.0, device=DEV)
    b.run_tree(out=out, lse=lse)
    n = int(b.q_off[-1])
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    b.check_tree(out[:n], lse[:n])


@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("w", [[6, 3, 8], [70, 33, 129]])
def test_a_chain_is_causal_and_a_star_is_alone(kind, w):
    lens = [400, 33, 129]
    b = Drafts(40, lens, 2, 64, 16, False)
    b.drafts(w, 2, 5, kind)
    out, lse = b.run_tree()
    b.check_tree(out, lse)
    if kind == "chain":
        o2, l2 = b.run(right=0)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("w", [[8, 3, 5], [70, 33, 90]])
def test_any_mask_and_more_tokens_than_cached_rows(w):
    # blocks that see each other in both directions; a mask wider than it needs to be; requests shorter than their drafts
    b = Drafts(41, [300, 2, 60], 2, 64, 16, False)
    b.drafts(w, 2, 6)
    rng = np.random.default_rng(7)
    see = [rng.random((n, n)) < 0.4 for n in w]
    words = (max(w) + 31) // 32 + 1
    m = np.zeros((int(b.q_off[-1]), words), np.uint32)
    for i, s in enumerate(see):
        for t, c in zip(*np.nonzero(s)):
            m[b.q_off[i] + t, c // 32] |= np.uint32(1) << np.uint32(c % 32)
        np.fill_diagonal(s, True)                             # a token sees itself, whatever its bit
    m[:, -1] = 0xffffffff
    out, lse = b.run_tree(mask=torch.from_numpy(m.view(np.int32)).to(DEV))
    b.check_tree(out, lse, see)


def test_long_requests_with_small_trees_are_divided():
    b = Drafts(42, [5000, 9000, 700], 1, 128, 64, True)
    b.drafts([5, 8, 3], 4, 8)
    first = b.run_tree()
    b.check_tree(*first)
    again = b.run_tree(ws=torch.empty(bd.paged_attn_workspace(b.pages, 3, 4, 8, 9000), dtype=torch.uint8, device=DEV))
    assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_drafts_beyond_their_bounds_are_clipped_and_reported():
    for w in ([6, 4], [60, 40]):
        b = Drafts(43, [200, 100], 1, 64, 16, False)
        b.drafts(w, 1, 9, "chain")
        q_max = w[0] - 2
        out = torch.zeros((sum(w), 1, 64), dtype=torch.bfloat16, device=DEV)
        bd.tree_attn(b.q, b.pages, i32(b.q_off), i32(b.lens), b.table, b.mask, q_max, 200, out=out)
        torch.cuda.synchronize()
        assert bd.device_status() == DEV_OFFSETS
        want, _ = b.run_tree()
        assert torch.equal(out[:q_max], want[:q_max]) and (out[q_max:w[0]] == 0).all() and torch.equal(out[w[0]:], want[w[0]:])


# ---------------------------------------------------------------------------
# mass
# ---------------------------------------------------------------------------

def slots(table, page, i, n):
    u = np.arange(n)
    return table[i, u // page], u % page


def check_mass(b, mass, old, lse, pos=None, right=-1, fresh=None, decay=1.0, scale=None, asked=None):
    scale = b.dh ** -0.5 if scale is None else scale
    table, got, old = b.table.cpu().numpy(), f64(mass), f64(old)
    q, lse = f64(b.q), f64(lse)
    touched = np.zeros(got.shape, bool)
    for i, (w, n) in enumerate(zip(b.w, b.lens)):
        a = int(b.q_off[i])
        if not w or not n:
            continue
        p = np.arange(w) + (n - w if pos is None else pos[i])
        total, off = cache_ops.mass(q[a:a + w], lse[a:a + w], b.k[i], p, scale, right)
        pg, sl = slots(table, b.page, i, n)
        before = np.where((np.arange(n) >= (n if fresh is None else fresh[i]))[:, None], 0.0, decay * old[pg, :, sl])
        tol = off + (w * b.group + 8) * 2.0 ** -23 * total + 2.0 ** -23 * (np.abs(before) + total) + 1e-37
        err = np.abs(got[pg, :, sl] - (before + total))
        assert (err <= tol).all(), f"request {i}: {float(np.max(err / tol)):.2f} of the tolerance"
        touched[pg, :, sl] = True
    assert np.array_equal(got[~touched], old[~touched], equal_nan=True)


def mass_of(b, seed=1):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(np.exp(rng.standard_normal(tuple(b.pages.k.shape[:3]))).astype(np.float32)).to(DEV)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page,heads,group,w,right", [
    (64, 16, 3, 1, [0, 1, 1, 1, 1, 1, 1, 1], 0), (128, 32, 1, 4, [0, 1, 3, 1, 2, 4, 1, 1], 0),
    (128, 64, 2, 2, [1, 1, 17, 64, 129, 300, 15, 100], 0), (64, 128, 5, 3, [0, 0, 17, 60, 70, 33, 15, 99], -1),
    (128, 16, 1, 8, [2, 1, 9, 128, 65, 64, 0, 257], 5), (64, 32, 1, 64, [0, 1, 2, 3, 4, 5, 6, 7], -1)])
def test_mass_of_every_cached_row(dh, page, heads, group, w, right, fp8):
    b = Batch(50 + dh, LENS, heads, dh, page, fp8)
    b.queries(w, group, 1.5)
    _, lse = b.run(right=right)
    mass = mass_of(b)
    old = mass.clone()
    got = bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, max(w), 1000, right=right)
    assert got is mass
    check_mass(b, mass, old, lse, right=right)


def test_mass_decays_and_starts_afresh():
    b = Batch(51, LENS, 2, 64, 16, True)
    w = [0, 1, 17, 40, 100, 33, 15, 64]
    b.queries(w, 2)
    _, lse = b.run(right=0)
    fresh = [0, 1, 5, 0, 129, 200, 15, 936]
    mass = mass_of(b)
    pg, sl = slots(b.table.cpu().numpy(), 16, 7, 1000)
    mass[pg[940:], :, sl[940:]] = float("nan")                # a fresh slot holds anything
    old = mass.clone()
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 100, 1000, fresh=i32(fresh), right=0, decay=0.25)
    old[pg[940:], :, sl[940:]] = 0
    check_mass(b, mass, old, lse, right=0, fresh=fresh, decay=0.25)


def test_mass_of_rows_at_given_positions_that_see_nothing_or_hold_nan():
    b = Batch(52, [50, 300, 20], 2, 64, 16, False)
    b.queries([20, 40, 3], 1)
    pos = [-10, 500, 2 ** 31 - 10]
    _, lse = b.run(pos=pos, right=0)
    lse[25] = float("inf")                                    # weights of 0
    mass = mass_of(b)
    old = mass.clone()
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 40, 300, q_pos=i32(pos), right=0)
    assert np.isneginf(f64(lse)[:10]).all()
    check_mass(b, mass, old, lse, pos=pos, right=0)
    b.q[3] = float("nan")                                     # request 0's row at position -7 sees nothing
    again = old.clone()
    bd.attn_mass(b.q, lse, b.pages, again, i32(b.q_off), i32(b.lens), b.table, 40, 300, q_pos=i32(pos), right=0)
    assert torch.equal(again, mass)


def test_mass_of_scores_that_are_large():
    b = Batch(53, [130, 700], 1, 128, 64, False, k_size=30.0)
    b.queries([4, 90], 2, 20.0)
    _, lse = b.run()
    mass = torch.zeros(tuple(b.pages.k.shape[:3]), device=DEV)
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 90, 700)
    check_mass(b, mass, torch.zeros_like(mass), lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -45, -0.125, 3.0])
@pytest.mark.parametrize("w", [3, 80])
def test_mass_at_any_scale(w, scale, fp8):
    b = Batch(56, [130, 700, 20], 2, 64, 16, fp8, spread=0.1)
    b.queries([w, w, 7], 1, 0.3)
    _, lse = b.run(right=0, scale=scale)
    mass = mass_of(b)
    old = mass.clone()
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, max(w, 7), 700, right=0, scale=scale)
    check_mass(b, mass, old, lse, right=0, scale=scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,page", [(64, 16), (128, 128)])
def test_mass_of_long_requests_and_many_rows(dh, page, fp8):
    # more items than CTAs, chunks that come by several times, rows of several requests behind each other
    b = Batch(57, [6000, 5000, 1, 4100], 8, dh, page, fp8, spread=0.1)
    b.queries([130, 300, 1, 65], 2, behind=3)
    pos = [6000 - 130, 100, 0, 4000]
    _, lse = b.run(pos=pos, right=0)
    mass = torch.zeros(tuple(b.pages.k.shape[:3]), device=DEV)
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 300, 6000, q_pos=i32(pos), right=0)
    check_mass(b, mass, torch.zeros_like(mass), lse, pos=pos, right=0)
    # single tokens of many requests
    lens = [int(n) for n in np.random.default_rng(58).integers(1, 2500, 40)]
    b = Batch(59, lens, 4, dh, page, fp8, spread=0.1)
    b.queries([1] * 40, 3)
    _, lse = b.run(right=0)
    mass = mass_of(b)
    old = mass.clone()
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 1, 2500, right=0, decay=0.5)
    check_mass(b, mass, old, lse, right=0, decay=0.5)


def test_mass_reports_what_it_does_not_reach():
    b = Batch(54, [200, 100], 1, 64, 16, False)
    b.queries([6, 4], 1)
    _, lse = b.run(right=0)
    mass = mass_of(b)
    old = mass.clone()
    table = b.table.clone()
    table[1, 2] = 10 ** 6
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), table, 6, 200, right=0)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    full = old.clone()
    bd.attn_mass(b.q, lse, b.pages, full, i32(b.q_off), i32(b.lens), b.table, 6, 200, right=0)
    skipped = int(b.table[1, 2])
    assert torch.equal(mass[skipped], old[skipped])
    keep = [p for p in range(mass.shape[0]) if p != skipped]
    assert torch.equal(mass[keep], full[keep])
    mass = old.clone()
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 6, 150, right=0)     # 150 of 200 keys
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    pg, sl = slots(b.table.cpu().numpy(), 16, 0, 200)
    assert torch.equal(mass[pg[:150], :, sl[:150]], full[pg[:150], :, sl[:150]])
    assert torch.equal(mass[pg[150:], :, sl[150:]], old[pg[150:], :, sl[150:]])


def test_mass_twice_gives_the_same_bits():
    b = Batch(55, [3000, 700, 1], 2, 128, 32, True)
    b.queries([64, 700, 1], 4)
    _, lse = b.run(right=0)
    runs = []
    for _ in range(2):
        mass = torch.ones(tuple(b.pages.k.shape[:3]), device=DEV)
        bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 700, 3000, right=0)
        runs.append(mass)
    assert torch.equal(*runs)


# ---------------------------------------------------------------------------
# moves and eviction
# ---------------------------------------------------------------------------

class Pool:
    """Pages of random bytes, tables, and the moves in NumPy."""

    def __init__(self, seed, lens, heads, dh, page, fp8, new=None):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.heads, self.page = list(lens), heads, page
        need, more = [-(-n // page) for n in lens], [-(-n // page) for n in new or []]
        pages = sum(need) + sum(more) + 2
        order = rng.permutation(pages)
        self.table, self.dst = (np.full((len(lens), max(c + [1])), -1) for c in (need, more))
        at = 0
        for t, counts in ((self.table, need), (self.dst, more)):
            for i, n in enumerate(counts):
                t[i, :n] = order[at:at + n]
                at += n
        self.pages = bd.KVPages.empty(pages, page, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
        for t in self.tensors():
            t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
        x = np.exp(2 * rng.standard_normal((pages, heads, page))).astype(np.float32)
        x[rng.random(x.shape) < 0.2] = 0.0                     # ties
        self.mass = torch.from_numpy(x).to(DEV)

    def tensors(self):
        p = self.pages
        return [t.view(torch.uint8) for t in (p.k, p.v, p.k_scale, p.v_scale) if t is not None]

    def state(self):
        return [t.cpu().numpy().copy() for t in self.tensors()] + [self.mass.cpu().numpy().copy()]

    def moved(self, lists, first, in_place, with_mass):
        """State after rows lists[i][h] moved to first[i] + 0, 1, .."""
        before = self.state()
        after = [t.copy() for t in before]
        dst = self.table if in_place else self.dst
        for i, per in enumerate(lists):
            for h in range(self.heads):
                src = np.asarray(per[h if len(per) > 1 else 0], np.int64)
                to = first[i] + np.arange(len(src))
                for k, (a, b) in enumerate(zip(after, before)):
                    if k < len(before) - 1 or with_mass:
                        a[dst[i, to // self.page], h, to % self.page] = b[self.table[i, src // self.page], h, src % self.page]
        return after

    def check(self, want):
        for got, w in zip(self.state(), want):
            assert np.array_equal(got, w)


def padded(lists, width):
    return i32([[list(x) + [-7] * (width - len(x)) for x in per] for per in lists])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dh,page,heads,per_head", [(64, 16, 3, True), (128, 32, 1, False), (128, 128, 4, True), (64, 64, 2, False)])
def test_moves(dh, page, heads, per_head, in_place, fp8):
    lens = [0, 1, 17, 300, 2500, 129, 5000]
    first = [0, 0, 3, 0, 70, 0, 1] if in_place else [0, 2, 0, 5, 0, 1, 0]
    p = Pool(60 + dh, lens, heads, dh, page, fp8, None if in_place else [n + 8 for n in lens])
    lists = []
    for n, a in zip(lens, first):
        low = a if in_place else 0
        m = max(n - low, 0)
        lists.append([np.sort(p.rng.permutation(m)[:p.rng.integers(0, m + 1)]) + low for _ in range(heads if per_head else 1)])
    lists = [[x[:min(len(y) for y in per)] for x in per] for per in lists]
    lists[5] = [np.arange(129 - first[5]) + first[5]] * len(lists[5])     # nothing changes place, in place
    if not in_place:
        lists[6] = [np.arange(5000)[::-1]] * len(lists[6])                 # elsewhere any order will do
    count = [len(per[0]) for per in lists]
    width = max(count) + 3
    want = p.moved(lists, first, in_place, True)
    bd.kv_move(p.pages, padded(lists, width), i32(count), i32(first), i32(p.table), dst_table=None if in_place else i32(p.dst), mass=p.mass)
    p.check(want)


def test_moves_without_mass_and_first():
    p = Pool(70, [100, 40], 2, 64, 16, True)
    lists = [[[3, 50, 51, 99]], [[0, 39]]]
    want = p.moved(lists, [0, 0], True, False)
    table = i32(p.table)
    bd.kv_move(p.pages, padded(lists, 4), i32([4, 2]), None, table, dst_table=table)      # the same table: in place
    p.check(want)


def test_moves_that_cannot_be_are_left_out_and_reported():
    p = Pool(71, [100, 40], 1, 64, 16, False)
    good = p.moved([[[5, 6]], [[]]], [0, 0], True, False)
    # what does not ascend, moves back, lies outside the table
    bd.kv_move(p.pages, i32([[[5, 6, 6, 2, 10 ** 6, -1]], [[0, 0, 0, 0, 0, 0]]]), i32([6, 0]), None, i32(p.table))
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    p.check(good)
    bd.kv_move(p.pages, i32([[[0, 1]], [[0, 1]]]), i32([3, -1]), None, i32(p.table))
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    p.check(good)
    table = p.table.copy()
    table[0, 0] = 999
    bd.kv_move(p.pages, i32([[[20, 21]], [[3, 4]]]), i32([2, 0]), None, i32(table))
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE
    p.check(good)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("in_place,move_mass", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dh,page,heads,budget,sinks,recent", [
    (64, 16, 3, 200, 4, 32), (128, 64, 1, 1000, 0, 0), (128, 32, 2, 64, 32, 32), (64, 128, 2, 1, 0, 1), (128, 16, 1, 129, 1, 0)])
def test_eviction(dh, page, heads, budget, sinks, recent, in_place, move_mass, fp8):
    lens = [0, 1, 17, 129, 200, 201, 3000, 9000]
    p = Pool(80 + budget, lens, heads, dh, page, fp8, None if in_place else [min(n, budget) for n in lens])
    table = p.table
    lists = []
    x = p.mass
    x[table[7, 10 // page], 0, 10 % page] = float("nan")
    x[table[7, 5000 // page], heads - 1, 5000 % page] = float("inf")
    x[table[6, 2000 // page], 0, 2000 % page] = -1.0
    x[table[6, 40 // page], 0, 40 % page] = -0.0
    m = f64(x)
    for i, n in enumerate(lens):
        pg, sl = slots(table, page, i, n)
        lists.append([cache_ops.keep(m[pg, h, sl], budget, sinks, recent) for h in range(heads)])
    want = p.moved(lists, [0] * len(lens), in_place, move_mass)
    new, keep = bd.kv_evict(p.pages, x, i32(lens), i32(table), budget, max(lens), sinks=sinks, recent=recent,
                            dst_table=None if in_place else i32(p.dst), move_mass=move_mass)
    assert new.tolist() == [min(n, budget) for n in lens]
    keep = keep.cpu().numpy()
    for i, per in enumerate(lists):
        for h, u in enumerate(per):
            assert np.array_equal(keep[i, h], list(u) + [-1] * (budget - len(u))), (i, h)
    for got, w in zip(p.state(), want):
        assert np.array_equal(got, w, equal_nan=got.dtype == np.float32)


@pytest.mark.parametrize("kind", ["equal", "few", "close", "falling"])
def test_eviction_of_weights_that_hardly_differ(kind):
    n, budget = 20000, 7001
    p = Pool(90, [n], 1, 64, 128, False)
    u = np.arange(n)
    w = {"equal": np.full(n, 0.5), "few": (u * 7919 % 3) * 1e-20, "close": 1 + (u * 104729 % 997) * 2.0 ** -23,
         "falling": 2.0 ** -(u / 150.0)}[kind].astype(np.float32)
    pg, sl = slots(p.table, 128, 0, n)
    p.mass[pg, 0, sl] = torch.from_numpy(w).to(DEV)
    new, keep = bd.kv_evict(p.pages, p.mass, i32([n]), i32(p.table), budget, n, sinks=3, recent=17)
    assert np.array_equal(keep.cpu().numpy()[0, 0], cache_ops.keep(w.astype(np.float64), budget, 3, 17))


def test_eviction_reports_lengths_beyond_their_bounds():
    p = Pool(91, [100, 64], 2, 64, 16, False)
    table = p.table
    m = f64(p.mass)
    new, keep = bd.kv_evict(p.pages, p.mass, i32([100, -5]), i32(table), 8, 50)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS
    pg, sl = slots(table, 16, 0, 50)
    assert new.tolist() == [8, 0] and (keep[1] == -1).all()
    for h in range(2):
        assert np.array_equal(keep.cpu().numpy()[0, h], cache_ops.keep(m[pg, h, sl], 8, 0, 0))


@pytest.mark.parametrize("dh,page,fp8", [(64, 16, True), (64, 128, False), (128, 32, True), (128, 16, False)])
@pytest.mark.parametrize("heads", [1, 6, 13, 28, 40])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (77, 3, 20), (300, 300, 0)])
def test_short_requests_cut_down_in_place(dh, page, fp8, heads, budget, sinks, recent):
    # 5 to 200 lists: eight CTAs a list, four, two, one, and two launches
    lens = [0, 1, 78, 700, 301]
    p = Pool(95 + heads + budget, lens, heads, dh, page, fp8)
    m = f64(p.mass)
    lists = [[cache_ops.keep(m[pg, h, sl], budget, sinks, recent) for h in range(heads)]
             for pg, sl in (slots(p.table, page, i, n) for i, n in enumerate(lens))]
    want = p.moved(lists, [0] * len(lens), True, True)
    new, keep = bd.kv_evict(p.pages, p.mass, i32(lens), i32(p.table), budget, max(lens), sinks=sinks, recent=recent)
    assert new.tolist() == [min(n, budget) for n in lens]
    keep = keep.cpu().numpy()
    for i, per in enumerate(lists):
        for h, u in enumerate(per):
            assert np.array_equal(keep[i, h], list(u) + [-1] * (budget - len(u))), (i, h)
    p.check(want)


def test_short_requests_with_bad_pages_in_place():
    lens = [100, 90]
    p = Pool(96, lens, 2, 64, 16, True)
    m = f64(p.mass)
    table = p.table.copy()
    table[0, 1], table[1, 0] = -1, 999                         # rows from there and to there stay where they are
    lists = []
    for i, n in enumerate(lens):
        pg, sl = slots(p.table, 16, i, n)
        gone = table[i, np.arange(n) // 16] != p.table[i, np.arange(n) // 16]
        lists.append([cache_ops.keep(np.where(gone, -np.inf, m[pg, h, sl]), 40, 0, 0) for h in range(2)])
    before = p.state()
    new, keep = bd.kv_evict(p.pages, p.mass, i32(lens), i32(table), 40, 100)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_PAGE and new.tolist() == [40, 40]
    keep, after = keep.cpu().numpy(), p.state()
    for i in range(2):
        for h in range(2):
            assert np.array_equal(keep[i, h], lists[i][h])
            for j, u in enumerate(keep[i, h]):
                to = (p.table[i, j // 16], h, j % 16)
                there = table[i, j // 16] == p.table[i, j // 16] and table[i, u // 16] == p.table[i, u // 16]
                for a, b in zip(after, before):
                    assert np.array_equal(a[to], b[p.table[i, u // 16], h, u % 16] if there else b[to])


@pytest.mark.parametrize("in_place", [True, False])
def test_lengths_that_are_cut_down_where_they_stand(in_place):
    # so many heads, and room for such long requests, that not all CTAs run at a time
    lens, heads, page = [70, 40, 8, 0, -3], 256, 16
    p = Pool(94, [70, 40, 8, 0, 0], heads, 64, page, True, None if in_place else [24, 24, 8, 0, 0])
    m = f64(p.mass)
    lists = [[cache_ops.keep(m[pg, h, sl], 24, 2, 3) for h in range(heads)]
             for pg, sl in (slots(p.table, page, i, max(n, 0)) for i, n in enumerate(lens))]
    want = p.moved(lists, [0] * len(lens), in_place, True)
    table = np.full((len(lens), 3000), -1)
    table[:, :p.table.shape[1]] = p.table
    kv_len = i32(lens)
    new, keep = bd.kv_evict(p.pages, p.mass, kv_len, i32(table), 24, 48000, sinks=2, recent=3, dst_table=None if in_place else i32(p.dst),
                            new_len=kv_len)
    torch.cuda.synchronize()
    assert bd.device_status() == DEV_OFFSETS               # the length below 0
    assert new is kv_len and kv_len.tolist() == [24, 24, 8, 0, 0]
    keep = keep.cpu().numpy()
    for i, per in enumerate(lists):
        for h, u in enumerate(per):
            assert np.array_equal(keep[i, h], list(u) + [-1] * (24 - len(u))), (i, h)
    p.check(want)


@pytest.mark.parametrize("n", [49152, 49153, 70001])
def test_eviction_from_long_requests(n):
    # more weights than shared memory holds, and just as many
    p = Pool(92, [n, 300], 1, 64, 128, True)
    m = f64(p.mass)
    pg, sl = slots(p.table, 128, 0, n)
    lists = [[cache_ops.keep(m[pg, 0, sl], 5000, 4, 100)], [list(range(300))]]
    want = p.moved(lists, [0, 0], True, True)
    new, keep = bd.kv_evict(p.pages, p.mass, i32([n, 300]), i32(p.table), 5000, n, sinks=4, recent=100)
    assert new.tolist() == [5000, 300] and keep[0, 0].tolist() == lists[0][0]
    p.check(want)


# ---------------------------------------------------------------------------
# many requests
# ---------------------------------------------------------------------------

def test_thousands_of_requests():
    rng = np.random.default_rng(120)
    B, heads, dh, page = 3000, 1, 64, 16
    w = rng.integers(0, 3, B)
    lens = w + rng.integers(0, 40, B)
    b = Batch(121, lens.tolist(), heads, dh, page, False, spread=0.1)
    off = np.cumsum(np.concatenate([[0], w]))
    rows = int(off[-1])
    q, k, v = rope_case(rng, rows, heads, 2, dh, 0.1)
    pos = rng.integers(0, 5000, rows)
    freq = [10000.0 ** (-j / 32) for j in range(32)]
    args = (i32(off), i32(lens - w), b.table)
    q2 = bd.rope_kv_write(b.pages, bd.Rope(dh, [0] * 32, freq), i32(pos), q, k, v, *args)
    check_turned(f64(q2), cache_ops.rotate(f64(q), [pos], [0] * 32, freq), pair_sizes(f64(q), 32))
    kk, vv = bd.kv_read(b.pages, *args, rows)
    check_turned(f64(kk), cache_ops.rotate(f64(k), [pos], [0] * 32, freq), pair_sizes(f64(k), 32))
    assert torch.equal(vv, v.contiguous())
    # the cache as it is now
    kr, vr = f64(kk), f64(vv)
    for i in range(B):
        if w[i]:
            b.k[i], b.v[i] = b.k[i].copy(), b.v[i].copy()
            b.k[i][lens[i] - w[i]:], b.v[i][lens[i] - w[i]:] = kr[off[i]:off[i + 1]], vr[off[i]:off[i + 1]]
    b.w, b.group, b.q_off, b.q = w.tolist(), 2, off, q2
    parent = i32(np.concatenate([np.arange(-1, n - 1) for n in w]).astype(np.int64))
    mask, depth = bd.tree_mask(parent, i32(off), 2)
    assert depth.tolist() == [t for n in w for t in range(n)]
    out, lse = bd.tree_attn(q2, b.pages, i32(off), i32(lens), b.table, mask, 2, 64, return_lse=True)
    b.check(out, lse, right=0)
    mass = mass_of(b)
    old = mass.clone()
    bd.attn_mass(q2, lse, b.pages, mass, i32(off), i32(lens), b.table, 2, 64, right=0)
    check_mass(b, mass, old, lse, right=0)
    new, keep = bd.kv_evict(b.pages, mass, i32(lens), b.table, 7, 64, recent=2)
    m, table = f64(mass), b.table.cpu().numpy()
    assert new.tolist() == np.minimum(lens, 7).tolist()
    # (the rows have moved in place: mass too)
    kept = keep.cpu().numpy()[:, 0]
    assert all((np.diff(kept[i, :n]) > 0).all() and (kept[i, n:] == -1).all() for i, n in enumerate(np.minimum(lens, 7)))
    for i in (5, 1500, 2999):
        n = int(min(lens[i], 7))
        pg, sl = slots(table, page, i, n)
        pages = b.pages.k.float()[pg, 0, sl].cpu().numpy()
        assert np.array_equal(pages, b.k[i][kept[i, :n], 0].astype(np.float32))


@pytest.mark.parametrize("w", [6, 70])
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_far_into_a_large_pool(fp8, w):
    # K and V pass 2^32 bytes: the same bits as in a small pool
    page, heads, group, dh, lens = 128, 4, 2, 128, [700, 130, 2000]
    need = [-(-n // page) for n in lens]
    small = np.full((3, max(need)), -1)
    for i, (a, n) in enumerate(zip(np.cumsum([0] + need), need)):
        small[i, :n] = np.arange(a, a + n)
    total = 2 * sum(need)                                      # the rows' pages, and those that they are moved to
    row = dh * (1 if fp8 else 2)
    pools = [total, (1 << 32) // (heads * page * row) + 2 * total]
    results = []
    rng = np.random.default_rng(140)
    old_k, old_v = (torch.from_numpy(rng.standard_normal((sum(lens), heads, dh), dtype=np.float32)).to(DEV, torch.bfloat16) for _ in range(2))
    q, k, v = rope_case(rng, 3 * w, heads, group, dh)
    par = i32([tree(rng, w, "any") for _ in lens]).flatten()
    start = torch.from_numpy(rng.random((total, heads, page), dtype=np.float32)).to(DEV)
    off, zero, pos0, kv_len = i32([0, w, 2 * w, 3 * w]), i32([0, 0, 0]), i32([n - w for n in lens]), i32(lens)
    for n in pools:
        first = n - total
        p = bd.KVPages.empty(n, page, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
        mass = torch.empty((n, heads, page), device=DEV)
        mass[first:] = start
        tensors = [t for t in (p.k, p.v, p.k_scale, p.v_scale) if t is not None]
        for t in tensors:
            t[first:].view(torch.uint8).zero_()
        table = np.where(small >= 0, small + first, -1)
        away = i32(np.where(small >= 0, small + first + sum(need), -1))
        table = i32(table)
        bd.kv_write(p, old_k, old_v, i32(np.cumsum([0] + lens)), zero, table)
        bd.kv_write(p, old_k, old_v, i32(np.cumsum([0] + lens)), zero, away)
        mask, depth = bd.tree_mask(par, off, w)
        q2 = bd.rope_kv_write(p, bd.Rope.standard(dh), depth + 1000, q, k, v, off, pos0, table)
        out, lse = bd.tree_attn(q2, p, off, kv_len, table, mask, w, max(lens), return_lse=True)
        bd.attn_mass(q2, lse, p, mass, off, kv_len, table, w, max(lens), right=0)
        new, keep = bd.kv_evict(p, mass, kv_len, table, 500, max(lens), sinks=2, recent=w, dst_table=away)
        new2, keep2 = bd.kv_evict(p, mass, kv_len, table, 400, max(lens), sinks=2, recent=w)
        bd.kv_move(p, keep2[:, :, 10:20].contiguous(), i32([10, 10, 10]), i32([3, 0, 7]), table, away, mass=mass)
        results.append([q2, out, lse, new, keep, new2, keep2, mass[first:].clone(), *(t[first:].view(torch.uint8).clone() for t in tensors)])
        torch.cuda.synchronize()
        assert bd.device_status() == 0
        del p, mass, tensors, t
    torch.cuda.empty_cache()
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.uint8) if x.dtype == torch.bfloat16 else x, y.view(torch.uint8) if y.dtype == torch.bfloat16 else y)


def test_two_calls_at_once():
    # two streams, a cache each: the calls share no memory of the library's
    cases = []
    for seed in (130, 131):
        b = Drafts(seed, [900, 3000, 17], 4, 128, 32, seed == 131)
        b.drafts([40, 64, 5], 2, seed)
        cases.append((b, mass_of(b), torch.empty(max(1, bd.paged_attn_workspace(b.pages, 3, 8, 64, 3000)), dtype=torch.uint8, device=DEV)))

    def work(b, mass, ws):
        out, lse = bd.tree_attn(b.q, b.pages, i32_cached(b.q_off), i32_cached(b.lens), b.table, b.mask, 64, 3000, return_lse=True, ws=ws)
        bd.attn_mass(b.q, lse, b.pages, mass, i32_cached(b.q_off), i32_cached(b.lens), b.table, 64, 3000, right=0)
        new, keep = bd.kv_evict(b.pages, mass, i32_cached(b.lens), b.table, 500, 3000, sinks=1, recent=70)
        return [out, lse, mass, new, keep, b.pages.k.view(torch.uint8), b.pages.v.view(torch.uint8)]

    start = [[t.clone() for t in (b.pages.k.view(torch.uint8), b.pages.v.view(torch.uint8), m)] for b, m, _ in cases]
    want = [[t.clone() for t in work(*c)] for c in cases]
    for (b, m, _), s in zip(cases, start):
        for t, x in zip((b.pages.k.view(torch.uint8), b.pages.v.view(torch.uint8), m), s):
            t.copy_(x)
        if b.pages.k_scale is not None:                        # the scales moved as well: write the rows again
            bd.kv_write(b.pages, b.k_in, b.v_in, b.off, i32([0, 0, 0]), b.table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append(work(*c))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            x, y = (t.view(torch.uint8) if t.dtype == torch.bfloat16 else t for t in (x, y))
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_a_draft_is_written_verified_and_its_accepted_path_kept(fp8):
    rng = np.random.default_rng(100)
    heads, group, dh, page, w, done = 2, 4, 64, 16, 12, [37, 5, 200]
    lens = [n + w for n in done]
    need = [-(-n // page) for n in lens]
    table = i32([list(range(a, a + n)) + [-1] * (max(need) - n) for a, n in zip(np.cumsum([0] + need), need)])
    p = bd.KVPages.empty(sum(need), page, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
    rope = bd.Rope.standard(dh)
    par = [tree(rng, w, "any") for _ in done]
    off = i32([0, w, 2 * w, 3 * w])
    mask, depth = bd.tree_mask(i32(sum(par, [])), off, w)
    # the committed tokens, then the drafts: slots in order, rotary positions by depth
    old = np.cumsum([0] + done)
    q, k, v = rope_case(rng, int(old[-1]), heads, group, dh)
    bd.rope_kv_write(p, rope, i32(np.concatenate([np.arange(n) for n in done])), None, k, v, i32(old), i32([0, 0, 0]), table)
    q, k, v = rope_case(rng, 3 * w, heads, group, dh)
    pos = depth + i32(np.repeat(done, w))
    q2 = bd.rope_kv_write(p, rope, pos, q, k, v, off, i32(done), table)
    out = bd.tree_attn(q2, p, off, i32(lens), table, mask, w, max(lens), out_fp32=True)
    # the deepest token's path is accepted: as if its tokens had come one after the other
    paths = []
    for x in par:
        see = cache_ops.ancestors(x)
        t = int(np.argmax(see.sum(1)))
        paths.append([int(c) for c in np.nonzero(see[t])[0]])
    n = max(len(x) for x in paths)
    src = i32([[[done[i] + c for c in x] + [0] * (n - len(x))] for i, x in enumerate(paths)])
    count = [len(x) for x in paths]
    bd.kv_move(p, src, i32(count), i32(done), table)
    lens2 = [a + b for a, b in zip(done, count)]
    rows = torch.cat([q2[i * w + torch.tensor(x)] for i, x in enumerate(paths)])
    chain = bd.paged_attn(rows, p, i32(np.cumsum([0] + count)), i32(lens2), table, n, max(lens2), right=0, out_fp32=True)
    want = torch.cat([out[i * w + torch.tensor(x)] for i, x in enumerate(paths)])
    # one row's weights and sums, rounded alike, over keys in other tiles' places
    assert (chain - want).abs().max() <= 2.0 ** -6 * want.abs().max()
    p2 = [t.clone() for t in (p.k.view(torch.uint8), p.v.view(torch.uint8))]
    # ... and as if the accepted tokens had been written where they lie now
    rows_k = torch.cat([k[i * w + torch.tensor(x)] for i, x in enumerate(paths)])
    rows_v = torch.cat([v[i * w + torch.tensor(x)] for i, x in enumerate(paths)])
    bd.rope_kv_write(p, rope, i32(np.concatenate([a + np.arange(b) for a, b in zip(done, count)])), None, rows_k, rows_v,
                     i32(np.cumsum([0] + count)), i32(done), table)
    assert torch.equal(p.k.view(torch.uint8), p2[0]) and torch.equal(p.v.view(torch.uint8), p2[1])


def test_weigh_evict_and_attend_again():
    b = Batch(101, [900, 300, 60], 2, 128, 16, True)
    b.queries([8, 8, 8], 2, 2.0)
    _, lse = b.run(right=0)
    mass = torch.zeros(tuple(b.pages.k.shape[:3]), device=DEV)
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 8, 900, right=0)
    new, keep = bd.kv_evict(b.pages, mass, i32(b.lens), b.table, 128, 900, sinks=2, recent=8)
    keep = keep.cpu().numpy()
    k, v = b.k, b.v
    b.k, b.v, b.lens = [], [], new.tolist()
    for i, n in enumerate(b.lens):
        b.k.append(np.stack([k[i][keep[i, h, :n], h] for h in range(2)], 1))
        b.v.append(np.stack([v[i][keep[i, h, :n], h] for h in range(2)], 1))
    b.check(*b.run(right=0), right=0)
    # the weights moved with their rows
    m2 = f64(mass)
    for i, n in enumerate(b.lens):
        pg, sl = slots(b.table.cpu().numpy(), 16, i, n)
        assert (m2[pg, :, sl] >= 0).all()


def _all_calls(b, rope, q, k, v, pos, par, mass, dst, ws):
    """One step of everything; returns what it gave back."""
    off, pos0 = i32_cached(b.q_off), i32_cached([n - m for n, m in zip(b.lens, b.w)])
    lens = i32_cached(b.lens)
    mask, depth = bd.tree_mask(par, off, max(b.w))
    q2 = bd.rope_kv_write(b.pages, rope, pos, q, k, v, off, pos0, b.table)
    out, lse = bd.tree_attn(q2, b.pages, off, lens, b.table, mask, max(b.w), max(b.lens), return_lse=True, ws=ws)
    bd.attn_mass(q2, lse, b.pages, mass, off, lens, b.table, max(b.w), max(b.lens), fresh=pos0, right=0, decay=0.5)
    new, keep = bd.kv_evict(b.pages, mass, lens, b.table, 100, max(b.lens), sinks=2, recent=10, dst_table=dst)
    bd.kv_move(b.pages, keep[:, :1, 3:9].contiguous(), i32_cached([4] * len(b.lens)), i32_cached([1] * len(b.lens)), dst, mass=mass)
    return [mask, depth, q2, out, lse, mass, new, keep, b.pages.k, b.pages.v]


_CACHED = {}


def i32_cached(x):
    """An int32 tensor made once: nothing is copied from the host under capture."""
    key = tuple(int(a) for a in x)
    if key not in _CACHED:
        _CACHED[key] = i32(key)
    return _CACHED[key]


@pytest.mark.parametrize("where", ["graph", "stream"])
def test_the_same_in_a_graph_and_on_another_stream(where):
    def setup():
        b = Drafts(110, [400, 130, 64], 2, 64, 16, False, spare=30)
        b.drafts([20, 33, 5], 2, 11)
        rng = np.random.default_rng(111)
        q, k, v = rope_case(rng, 58, 2, 2, 64)
        used = set(b.table.cpu().numpy().ravel().tolist())
        free = [x for x in range(b.pages.num_pages) if x not in used]
        dst = i32(np.array(free[:21]).reshape(3, 7))
        return (b, bd.Rope.standard(64), q, k, v, i32(rng.integers(0, 5000, 58)), i32(sum(b.parents, [])),
                torch.ones(tuple(b.pages.k.shape[:3]), device=DEV), dst,
                torch.empty(max(bd.paged_attn_workspace(b.pages, 3, 4, 33, 400), 1), dtype=torch.uint8, device=DEV))

    want = [t.clone() for t in _all_calls(*setup())]
    torch.cuda.synchronize()
    args = setup()
    start = [t.clone() for t in (args[0].pages.k, args[0].pages.v, args[7])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    if where == "stream":
        with torch.cuda.stream(s):
            got = _all_calls(*args)
        s.synchronize()
    else:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = _all_calls(*args)
        for _ in range(3):
            for t, x in zip((args[0].pages.k, args[0].pages.v, args[7]), start):
                t.copy_(x)
            g.replay()
        torch.cuda.synchronize()
    for a, b in zip(got, want):
        if a.dtype == torch.bfloat16:
            a, b = a.view(torch.int16), b.view(torch.int16)
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens,budget", [([700, 90, 400], 64), ([9000, 400, 65], 1000)])
def test_in_place_in_a_graph_replayed(lens, budget):
    # one launch and two; the replays go on from what the one before left
    def setup():
        p = Pool(150, lens, 2, 128, 32, True)
        return p, i32(lens), i32(p.table), i32([[[30, 33, 40]]] * 3), i32([3, 2, 3]), i32([20, 30, 29])

    def step(p, kv_len, table, src, count, first):
        new, keep = bd.kv_evict(p.pages, p.mass, kv_len, table, budget, max(lens), sinks=2, recent=9)
        bd.kv_move(p.pages, src, count, first, table, mass=p.mass)
        return new, keep

    a, b = setup(), setup()
    got = []
    for _ in range(3):
        got.append([t.clone() for t in step(*a)])
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        out = step(*b)
    for want in got:
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    assert bd.device_status() == 0
    b[0].check(a[0].state())
