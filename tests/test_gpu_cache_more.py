"""GPU parity of the operators around the paged cache, beyond what
test_gpu_cache_ops.py holds and with its bounds."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd
from oracle import cache_ops
from test_gpu_cache_ops import Drafts, _status_clear, check_mass, mass_of, rope_case, slots  # noqa: F401
from test_gpu_paged import DEV, Batch, f64, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sign", [1, -1])
def test_the_smallest_angles_of_far_positions(sign):
    # Far positions whose angle is next to a whole turn: a bf16 sine of a small angle shows errors that one of a large angle
    # hides. The angle is off by 2^-64 turns per position, 2^-24 of itself, and the sine rounded once: 2^-8 of it.
    freq = [sign * f for f in (0.3, 0.75, 1e-3, 1e-5, 0.5, 1 / 3, 1000.0, 0.01)]
    two_pi = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)
    far = 2 ** 31 - 1 - np.arange(1 << 21, dtype=np.uint64)
    pos = []
    for f in freq:
        turns = np.uint64(round(Fraction(f) / two_pi * 2 ** 64) % 2 ** 64)
        pos += [int(far[np.argsort(np.abs((far * turns).view(np.int64)))[n]]) for n in (0, 3, 40)]
    n = len(pos)
    x = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device=DEV)
    x[..., :8] = 1
    p = bd.KVPages.empty(2, 16, 1, 64, torch.bfloat16, DEV)
    out = f64(bd.rope_kv_write(p, bd.Rope(64, [0] * 8, freq), i32([pos]), x, x, x, i32([0, n]), i32([0]), i32([[0, 1]])))
    for r, u in enumerate(pos):
        j = r // 3
        a = Fraction(freq[j]) * u % two_pi
        a = float(a - two_pi if a > two_pi / 2 else a)
        assert abs(a) < 1e-4
        assert abs(out[r, 0, 8 + j] - math.sin(a)) <= (2.0 ** -8 + 2.0 ** -20) * abs(math.sin(a)) + 2.0 ** -33 * 6.4, (u, freq[j])


@pytest.mark.parametrize("fp8", [False, True])
def test_q_turned_where_the_projection_left_it(fp8):
    # q, k and v are views of one projection's rows, and q_out is q's
    rng = np.random.default_rng(310)
    heads, group, dh, rows = 2, 3, 64, 37
    q, k, v = rope_case(rng, rows, heads, group, dh)
    rope, pos = bd.Rope.standard(dh, sections=[8, 0, 24, 0]), i32(rng.integers(-5, 9000, (4, rows)))
    args = (i32([0, 20, rows]), i32([0, 40]), i32([[0, 1, -1, -1], [2, 3, 4, 5]]))
    got = []
    for joint in (False, True):
        p = bd.KVPages.empty(6, 16, heads, dh, torch.float8_e4m3fn if fp8 else torch.bfloat16, DEV)
        tensors = [t.view(torch.uint8) for t in (p.k, p.v, p.k_scale, p.v_scale) if t is not None]
        for t in tensors:
            t.zero_()
        kv = torch.cat([k, v], 1)
        out = bd.rope_kv_write(p, rope, pos, q, k, v, *args, q_out=q if joint else None)
        assert torch.equal(kv, torch.cat([k, v], 1)) and (out is q) == joint
        got.append([out.clone(), *tensors])
    assert all(torch.equal(x, y) for x, y in zip(*got))


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w,lens", [([13], [300]), ([20, 64, 33, 40], [8000, 700, 70, 3000]), ([5, 8, 6, 7], [20000, 9000, 400, 15000])])
def test_trees_repeat_themselves_bit_for_bit(w, lens, fp8):
    b = Drafts(320, lens, 4, 128, 16, fp8)
    b.drafts(w, 4, 321)
    first = b.run_tree()
    b.check_tree(*first)
    args = (b.q, b.pages, i32(b.q_off), i32(b.lens), b.table, b.mask, max(w), max(lens))
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        out = bd.tree_attn(*args, return_lse=True)
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(b.run_tree(), first))
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, first))


# ---------------------------------------------------------------------------
# mass
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("w,group", [(20, 4), (33, 2), (3, 64)])
def test_mass_of_heads_that_end_within_an_item(dh, w, group):
    # many items a CTA, one chunk each or two, of 65 to 128 rows; a head's last item has 1 to 3 tiles
    # beside full ones, so that tiles come and go for the groups that share the stages
    rng = np.random.default_rng(dh + w)
    heads = 8 if group < 64 else 2
    lens = [int(n) for n in rng.choice([1, 100, 129, 300, 384, 513, 640, 700, 896, 1025, 1300], 60 if group < 64 else 200)]
    w = [min(w, n) for n in lens]
    b = Batch(300 + dh, lens, heads, dh, 64, True, spread=0.1)
    b.queries(w, group)
    _, lse = b.run(right=0)
    old = mass_of(b)
    off, n = i32(b.q_off), i32(b.lens)
    first = None
    for _ in range(6):
        mass = old.clone()
        bd.attn_mass(b.q, lse, b.pages, mass, off, n, b.table, max(w), max(lens), right=0, decay=0.5)
        if first is None:
            first = mass
            check_mass(b, mass, old, lse, right=0, decay=0.5)
        assert torch.equal(mass, first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dh,heads,group", [(128, 2, 4), (64, 1, 1)])
def test_mass_of_as_many_rows_as_keys(dh, heads, group, fp8):
    # causal prompts weigh themselves: the chunks of early rows see none of the late keys
    b = Batch(330 + dh, [1000, 1200, 129], heads, dh, 32, fp8, spread=0.1)
    b.queries([1000, 1100, 129], group)
    _, lse = b.run(right=0)
    mass = mass_of(b)
    old = mass.clone()
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 1100, 1200, fresh=i32([0, 100, 129]), right=0)
    check_mass(b, mass, old, lse, right=0, fresh=[0, 100, 129])


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------

def evict_and_check(b, mass, budget, max_kv, in_place, **kw):
    """Evict by mass; what stays is the oracle's choice, and the weights lie with their rows."""
    before, table = f64(mass), b.table.cpu().numpy()
    dst, goes = None, table
    if not in_place:
        free = np.setdiff1d(np.arange(b.pages.num_pages), table[table >= 0])
        per = -(-budget // b.page)
        goes = free[:per * len(b.lens)].reshape(len(b.lens), per)
        dst = i32(goes)
    new, keep = bd.kv_evict(b.pages, mass, i32(b.lens), b.table, budget, max_kv, dst_table=dst, **kw)
    after, keep = f64(mass), keep.cpu().numpy()
    assert new.tolist() == [min(n, budget) for n in b.lens]
    for i, n in enumerate(b.lens):
        pg, sl = slots(table, b.page, i, n)
        for h in range(b.heads):
            want = cache_ops.keep(before[pg, h, sl], budget, kw.get("sinks", 0), kw.get("recent", 0))
            assert keep[i, h].tolist() == want + [-1] * (budget - len(want)), (i, h)
            to, at = slots(goes, b.page, i, len(want))
            assert np.array_equal(after[to, h, at], before[pg, h, sl][want]), (i, h)
    return new.tolist(), keep


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,budget", [([900, 300, 60], 128), ([9000, 300, 60], 128)])
def test_weights_move_with_their_rows(lens, budget, in_place):
    b = Batch(340, lens, 2, 128, 16, True, spare=30)
    b.queries([8, 8, 8], 2, 2.0)
    _, lse = b.run(right=0)
    mass = mass_of(b)
    bd.attn_mass(b.q, lse, b.pages, mass, i32(b.q_off), i32(b.lens), b.table, 8, max(lens), right=0)
    evict_and_check(b, mass, budget, max(lens), in_place, sinks=2, recent=8)


def test_what_thousands_of_requests_keep():
    rng = np.random.default_rng(341)
    b = Batch(342, rng.integers(0, 45, 3000).tolist(), 1, 64, 16, False, spread=0.1)
    evict_and_check(b, mass_of(b, 343), 7, 64, True, recent=2)
