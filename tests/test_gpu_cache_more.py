"""GPU parity of the operators around the paged cache, beyond what
test_gpu_cache_ops.py holds and with its bounds."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd
from test_gpu_cache_ops import _status_clear, check_mass, mass_of  # noqa: F401
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
