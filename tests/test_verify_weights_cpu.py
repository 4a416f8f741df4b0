"""The polynomial of the verification's weights (host only): its constants, read from the
source, against 2^f in 60 digits."""
import os
import re
from decimal import Decimal, getcontext

from w4a16_bit_matmul_amd import _build


def source():
    with open(os.path.join(_build.CSRC, "wq_verify.hip")) as f:
        return f.read()


def coefficients(text):
    """From the highest degree down."""
    top = re.search(r"double p = fma\((0x[0-9a-fp.+-]+), f, c8\)", text).group(1)
    c8 = re.search(r"c8 = (0x[0-9a-fp.+-]+);", text).group(1)
    rest = re.findall(r"p = fma\(p, f, (0x[0-9a-fp.+-]+|1\.0)\);", text)
    return [Decimal(float.fromhex(c) if c.startswith("0x") else float(c)) for c in [top, c8, *rest]]


def test_the_polynomial_is_as_near_as_the_source_says():
    getcontext().prec = 60
    text = source()
    c = coefficients(text)
    assert len(c) == 10 and c[-1] == 1  # degree 9; equal logits have whole weights
    stated = Decimal(re.search(r"polynomial, ([0-9.e-]+) of it off at most", text).group(1))
    worst, N = Decimal(0), 4000
    ln2 = Decimal(2).ln()
    for i in range(N + 1):
        f = Decimal(i) / N - Decimal("0.5")
        p = Decimal(0)
        for x in c:
            p = p * f + x
        worst = max(worst, abs(p / (f * ln2).exp() - 1))
    assert worst <= stated <= 2 * worst, (worst, stated)
