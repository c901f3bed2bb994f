"""The accuracy that include/dllm.h states for attention over e4m3 pages, from
the roundings themselves (CPU only)."""

import os
import re

import numpy as np
import torch

from oracle.paged import E4M3, nearest_code

HERE = os.path.dirname(os.path.abspath(__file__))


def _statement():
    """(a, b): elements of q from 2^-a of their row's largest on are exact, the others off by up to 2^-b of it."""
    with open(os.path.join(HERE, "..", "include", "dllm.h")) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    m = re.search(r"elements of q below 2\^-([\d.]+) of the largest of their row are off by up to 2\^-([\d.]+) of that", text)
    return float(m.group(1)), float(m.group(2))


def _two_parts(x):
    """x [..] bf16 values scaled into |x| <= 448, as the sum of two e4m3 parts."""
    hi = E4M3[nearest_code(x)]
    return hi + E4M3[nearest_code(x - hi)]


def test_query_parts_are_as_exact_as_stated():
    exact_from, off_by = _statement()
    m = 1 + np.arange(128) / 128.0                                   # every bf16 mantissa
    x = (m[None] * 2.0 ** np.arange(-40, 9)[:, None]).ravel()        # of every size up to the largest
    x = x[x <= 448]
    err = np.abs(_two_parts(x) - x)
    tops = np.concatenate([m[m > 1.75] * 128, m[m <= 1.75] * 256])    # what a row's largest is scaled to
    worst = 0.0
    for top in tops:
        of = x <= top
        rel, e = x[of] / top, err[of] / top
        assert not e[rel >= 2.0 ** -exact_from].any()
        worst = max(worst, e.max())
    assert worst <= 2.0 ** -off_by
    assert worst > 2.0 ** -(off_by + 0.25)                            # and the statement is no looser than it has to be


def _weights_statement():
    """(a, b): weight times V scale is off by up to 2^-a of itself, or 2^-b of the largest V scale where that is more."""
    with open(os.path.join(HERE, "..", "include", "dllm.h")) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    m = re.search(r"weight times V scale is off by up to 2\^-([\d.]+) of itself, or 2\^-([\d.]+) of the largest V scale", text)
    return float(m.group(1)), float(m.group(2))


def _three_parts(w):
    """w (fp32, 0 <= w <= 4) as the sum of three e5m2 parts of w 2^13, or of w 2^25 below 2^-10."""
    w = w.astype(np.float32)
    small = w < np.float32(2.0 ** -10)
    h = (w * np.where(small, np.float32(2.0 ** 25), np.float32(2.0 ** 13))).astype(np.float16)
    total, rest = np.zeros(w.shape), h
    for _ in range(2):                                               # e5m2 is the upper byte of fp16
        part = (rest.view(np.uint16) & 0xFF00).view(np.float16)
        total, rest = total + part, rest - part
    total = total + torch.from_numpy(rest).to(torch.float8_e5m2).double().numpy()
    return total * np.where(small, 2.0 ** -25, 2.0 ** -13)


def test_weight_parts_are_as_exact_as_stated():
    of_itself, of_largest = _weights_statement()
    rng = np.random.default_rng(0)
    worst = []
    for e in range(-60, 2):
        w = np.float32(2.0 ** e) * np.concatenate([1 + rng.random(20000), 1 + np.arange(4096) / 4096, [2 - 2.0 ** -23]]).astype(np.float32)
        err = np.abs(_three_parts(w) - w)
        # relative: half a step of nine bits and of fp16's eleven, 2^-9 + 2^-12 < 2^-8.8; else half of e5m2's least
        # step 2^-16, and of fp16's step where w is near 2^-33: (2^-17 + 2^-19) / 2^25 = 1.25 * 2^-42 < 2^-41.6
        assert (err <= np.maximum(2.0 ** -of_itself * w, 2.0 ** -of_largest)).all(), e
        worst.append((np.log2((err / w).max()), np.log2(err.max())))
    rel, absolute = np.array(worst).T
    assert rel[-30:].max() > -of_itself - 0.25 and absolute[:28].max() > -of_largest - 0.25     # no looser than it has to be
