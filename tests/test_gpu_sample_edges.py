"""Sampled verification where the sums' last units decide."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_util as U
from invariant_verify_gb300 import abi as B
from test_gpu_sample import check, run

pytestmark = pytest.mark.gpu


def plain(rows, us):
    """K = 0 requests: one row of probabilities and one uniform number each."""
    N, V = rows.shape
    return dict(target=rows.view(N, 1, V).contiguous(), draft_probs=None, draft=torch.zeros(N, 0, dtype=torch.int32),
                u_accept=torch.zeros(N, 0), u_sample=torch.tensor(us), p0=torch.zeros(N, dtype=torch.int32))


def pieces(x, at_most):
    """fp32 numbers, none above at_most, whose exact sum is x (a multiple of 2^-60)."""
    out = []
    while x:
        f = np.float32(float(min(x, at_most)))
        if Fraction(float(f)) > min(x, at_most):
            f = np.nextafter(f, np.float32(0))
        out.append(float(f))
        x -= Fraction(float(f))
    return out


# (S_0, the rest of the sum, u): u S lies within a few units (2^-60) of S_0
BORDERS = [(Fraction(1, 2), Fraction(1, 2) + d * Fraction(1, 2 ** 60), 0.5) for d in (-65, -4, -1, 0, 1, 4, 65)]
BORDERS += [(Fraction(1, 4), Fraction(3, 4) + d * Fraction(1, 2 ** 60), 0.25) for d in (-130, -3, 0, 3, 130)]
BORDERS += [(Fraction(1, 2 ** 30), 1 - Fraction(1, 2 ** 30) + d * Fraction(1, 2 ** 60), 2.0 ** -30) for d in (-7, 0, 7)]
# an odd significand of u: the smallest first entry that passes the border, and one unit less
for _u in (0.7, 0.3333333, 1 - 2.0 ** -24, 0.9):
    _u = float(np.float32(_u))
    for _s in (2 ** 60 - 1, 2 ** 60 + 12345677, 5 * 2 ** 60 - 3):
        _b = int(Fraction(_u) * _s)
        BORDERS += [(Fraction(_b + _d, 2 ** 60), Fraction(_s - _b - _d, 2 ** 60), _u) for _d in (1, 0)]


@pytest.mark.parametrize("pad", [0, 5000])
def test_border_is_exact_to_the_last_unit(pad):
    """token = min {v : S_v > u S} with S of up to 63 bits and u of 24: the product has more
    bits than a double."""
    rows, us, wrong = [], [], 0
    for first, rest, u in BORDERS:
        head, tail = pieces(first, Fraction(1)), pieces(rest, Fraction(1))
        rows.append(head + [0.0] * pad + tail)
        us.append(u)
        total = int((first + rest) * 2 ** 60)
        wrong += int(float(u) * float(total)) != int(Fraction(u) * total)
    assert wrong > 10                              # in so many cases a double's product is another border
    V = max(map(len, rows))
    c = plain(torch.tensor([r + [0.0] * (V - len(r)) for r in rows]), us)
    check(c)
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("N", [1, 9, 300])
def test_a_sum_of_eight_is_the_first_that_is_refused(N):
    """Decided on the exact sum: whatever order the entries are added in, however many
    requests share the device."""
    V = 9000
    under = [1.0] * 7 + [1 - 2.0 ** -24]           # rounds to 8 when it is added up in fp32
    spread = [1.0] * 7 + [2.0 ** -13] * 8191       # 8 - 2^-13, in parts that rounded sums may lose
    even = [1.0] * 8
    over = [1.0] * 8 + [2.0 ** -40]
    for row, fine in ((under, True), (spread, True), (even, False), (over, False)):
        row = row + [0.0] * (V - len(row))
        for order in (list(range(V)), list(range(V - 1, -1, -1)), torch.randperm(V, generator=U.gen(3)).tolist()):
            c = plain(torch.tensor(row)[order].expand(N, V), [0.99] * N)
            tokens, _, _ = run(c)
            assert B.biv_device_error() == (0 if fine else B.DEVERR_VALUE)
            want = U.verify(**{k: None if v is None else v[:1] for k, v in c.items()})[0][0] if fine else [0]
            assert (tokens == want).all()
