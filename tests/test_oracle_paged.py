"""Pins of the paged-cache oracle against hand-worked values and torch."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import paged


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, paged.E4M3, equal_nan=True)
    assert paged.E4M3[0x7E] == 448 and paged.E4M3[1] == 2.0 ** -9


def test_nearest_code_rounds_to_even_like_torch():
    x = np.concatenate([np.linspace(-448, 448, 20011), [0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 21.0, -17.0]])
    want = torch.tensor(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x = x.astype(np.float32).astype(np.float64)
    got = paged.E4M3[paged.nearest_code(x)]
    assert np.array_equal(got, paged.E4M3[want])
    assert paged.E4M3[paged.nearest_code(np.array([17.0, 19.0]))].tolist() == [16.0, 20.0]   # ties


def test_scale_is_the_least_that_fits():
    x = np.zeros((5, 4))
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 448.0, 450.0, 1.75, 1.7578125
    codes, b = paged.quantise(x)
    assert (b.astype(int) - 127).tolist() == [0, 1, -8, -7, -117]
    assert paged.restore(codes, b)[0, 0] == 448 and paged.restore(codes, b)[2, 0] == 1.75
    x = np.array([[np.inf, 1.0, np.nan, -2.0]])
    codes, b = paged.quantise(x)
    assert b[0] == 255 and np.isnan(paged.restore(codes, b)).all()
    top = float(torch.finfo(torch.bfloat16).max)
    codes, b = paged.quantise(np.array([[top, -top, 0.0, 1.0]]))
    assert paged.restore(codes, b)[0, :2].tolist() == [1.875 * 2.0 ** 127, -1.875 * 2.0 ** 127]


def test_quantised_rows_are_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp(rng.standard_normal((200, 1)) * 3)
    codes, b = paged.quantise(x)
    e = b.astype(np.float64)[:, None] - 127
    assert (np.abs(paged.restore(codes, b) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e - 10))).all()


def test_visible_by_hand():
    v = paged.visible([3, 6], 8, left=2, right=0, sinks=1)
    assert v[0].nonzero()[0].tolist() == [0, 1, 2, 3] and v[1].nonzero()[0].tolist() == [0, 4, 5, 6]
    assert paged.visible([-1], 4, -1, 0, 0).sum() == 0
    assert paged.visible([9], 4, 2, 0, 2)[0].nonzero()[0].tolist() == [0, 1]
    assert paged.visible([1], 6, 1, 2, 0)[0].nonzero()[0].tolist() == [0, 1, 2, 3]


def test_attention_without_mask_is_block_attention():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    out, lse, absv, _ = paged.attention(q, k, v, np.arange(4, 9), 0.3)
    want = oracle.block_attention(q, k.repeat(2, axis=1), v.repeat(2, axis=1), [0, 5], [0, 9], 0.3)
    assert np.abs(out - want).max() < 1e-13 and (absv >= np.abs(out) - 1e-15).all()


@pytest.mark.parametrize("left,right,sinks", [(-1, 0, 0), (2, 0, 1), (3, 1, 0)])
def test_attention_by_single_rows(left, right, sinks):
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 2, 4)), rng.standard_normal((7, 1, 4)), rng.standard_normal((7, 1, 4))
    pos = [-1, 2, 5, 12]
    out, lse, _, _ = paged.attention(q, k, v, pos, 0.5, left, right, sinks)
    for t, p in enumerate(pos):
        keys = [u for u in range(7) if (right < 0 or u <= p + right) and (left < 0 or u >= p - left or u < sinks)]
        for h in range(2):
            if not keys:
                assert not out[t, h].any() and lse[t, h] == -np.inf
                continue
            w = [math.exp(0.5 * float(q[t, h] @ k[u, 0])) for u in keys]
            want = sum(a * v[u, 0] for a, u in zip(w, keys)) / math.fsum(w)
            assert np.abs(out[t, h] - want).max() < 1e-14 and abs(lse[t, h] - math.log(math.fsum(w))) < 1e-13


def test_hidden_rows_are_not_read():
    q, k, v = np.ones((1, 1, 4)), np.ones((3, 1, 4)), np.ones((3, 1, 4))
    k[2], v[2] = np.nan, np.inf
    out, lse, _, _ = paged.attention(q, k, v, [1], 1.0, right=0)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
