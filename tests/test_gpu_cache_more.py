"""GPU parity of the operators around the paged cache, beyond what
test_gpu_cache_ops.py holds and with its bounds."""

import numpy as np
import pytest
import torch

import block_decoding_gb300 as bd
from test_gpu_cache_ops import _status_clear, check_mass, mass_of  # noqa: F401
from test_gpu_paged import Batch, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


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
