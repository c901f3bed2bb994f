"""Rotary frequencies as 64-bit fractions of a turn (csrc/turns.cuh), compiled for
the host and held to exact integer arithmetic: within one unit of 2^-64 turns
for every frequency that the entry point takes, negative and tiny ones too."""

import math
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_decoding_gb300", "csrc")
CXX = os.environ.get("CXX") or shutil.which("g++")


def _pi(bits=400):
    """pi by Machin's formula, to some bits less than asked."""
    one = 1 << bits

    def arctan_inverse(x):
        term = total = one // x
        n, sign = 1, 1
        while term:
            term //= x * x
            n, sign = n + 2, -sign
            total += sign * (term // n)
        return total

    return Fraction(4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


PI = _pi()


@pytest.fixture(scope="module")
def fractions_of(tmp_path_factory):
    if not CXX:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("turns")
    (d / "main.cpp").write_text('#include <stdio.h>\n#include "turns.cuh"\nint main() {\n  double f;\n'
                                '  while (scanf("%la", &f) == 1) printf("%llu\\n", dllm::fraction_of_turn(f));\n}\n')
    cmd = [CXX, "-O2", "-std=c++17", "-x", "c++", str(d / "main.cpp"), "-I", CSRC, "-o", str(d / "main")]
    # (conversions out of range are errors where the compiler can tell)
    if subprocess.run(cmd + ["-fsanitize=undefined,float-cast-overflow", "-fno-sanitize-recover=all"], capture_output=True).returncode:
        subprocess.run(cmd, check=True)

    def run(freqs):
        r = subprocess.run([str(d / "main")], input="".join(f.hex() + "\n" for f in freqs), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return [int(x) for x in r.stdout.split()]
    return run


def check(freqs, got):
    assert len(got) == len(freqs)
    for f, n in zip(freqs, got):
        want = Fraction(f) / (2 * PI) * 2 ** 64
        off = (n - want + 2 ** 63) % 2 ** 64 - 2 ** 63            # modulo a turn
        assert abs(off) <= 1, (f, float(off))


def common():
    f = [b ** (-2.0 * j / r) for b in (1e4, 5e5, 1e6) for r in (64, 128) for j in range(r // 2)]
    return f + [1024.0, math.nextafter(1024.0, 0), 6.283185307179586, 3.141592653589793, 1e-300, 5e-324, 0.0]


@pytest.mark.parametrize("sign", [1, -1])
def test_fractions_are_exact(fractions_of, sign):
    rng = random.Random(7)
    f = [sign * x for x in common() + [rng.uniform(0, 1024) for _ in range(4000)] + [10 ** rng.uniform(-25, 3) for _ in range(4000)]]
    check(f, fractions_of(f))


@pytest.mark.parametrize("f", [-0.3, -1e-3, -1e-5, -0.5, -1e-16, -1e-20, -2.0 ** -54 * 6.283185307179586, -1024.0])
def test_negative_and_tiny_frequencies(fractions_of, f):
    check([f], fractions_of([f]))
