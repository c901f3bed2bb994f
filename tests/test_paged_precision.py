"""The accuracy that include/dllm.h states for attention over e4m3 pages, from
the roundings themselves (CPU only)."""

import os
import re

import numpy as np

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
