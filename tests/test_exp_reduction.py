"""The argument reduction of the score router's fp64 exponential, in exact
arithmetic on the host: the two parts of ln 2 that the source states, and that
the first step x - n LN2 is exact for the arguments that occur."""
import os
import re
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "int4_weight_only_router_amd", "csrc", "k_route_select.hip")


def _parts():
    m = re.search(r"LN2 = (0x\S+?), LN2_LO = (0x\S+?);", open(SRC).read())
    return float.fromhex(m.group(1)), float.fromhex(m.group(2))


def test_two_parts_of_ln_2():
    getcontext().prec = 60
    hi, lo = _parts()
    ln2 = Decimal(2).ln()
    assert hi == float(ln2) and lo == float(ln2 - Decimal(hi))


def test_first_step_is_exact():
    """Differences of fp32 logits, as fp64 rounds them, and fp64 values next to
    the borders of n, down to -746."""
    hi, lo = _parts()
    r = np.random.default_rng(0)
    a, b = r.normal(0, 3, 20000).astype(np.float32), r.normal(0, 300, 20000).astype(np.float32)
    x = [-np.abs(a.astype(np.float64) - b), -np.abs(a.astype(np.float64)), -r.uniform(0, 746, 20000)]
    edge = np.outer(np.arange(0.5, 1076), [hi])[:, 0]
    x += [-np.nextafter(edge, d) for d in (0.0, 1e9)] + [-edge]
    x = np.maximum(np.concatenate(x), -746.0)
    n = np.rint(x * (1.0 / hi))
    assert n.min() == -1076 and np.abs(n).max() <= 1076
    for xi, ni in zip(x.tolist(), n.tolist()):
        exact = Fraction(xi) - Fraction(ni) * Fraction(hi)
        assert Fraction(float(exact)) == exact and abs(exact) < Fraction(7, 20)
