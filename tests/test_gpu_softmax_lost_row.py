"""A copy that never comes, in the softmax whose clusters stay: the kernel gives its rows up
and returns, and the context stays usable.  Nothing faults: the wait's limit ends it."""
import pytest
import torch

from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row", [100, 199])        # with rows after it, and the last one
def test_a_lost_row_ends_its_cluster_and_nothing_else(row):
    R, V, fill = 200, 40000, 7.0
    x = torch.randn(R, V, device="cuda")
    good, p = torch.empty_like(x), torch.full_like(x, fill)
    B.biv_softmax(x, good, 1.0)
    assert B.biv_device_error() == 0
    B.biv_selftest_softmax_lost_row(x, p, row)
    assert B.biv_device_error() == B.DEVERR_TIMEOUT
    right = (p == good).all(1).tolist()
    untouched = (p == fill).all(1).tolist()
    assert all(a != b for a, b in zip(right, untouched))
    lost = [r for r in range(R) if untouched[r]]
    assert lost[0] == row                          # the rows of the cluster from there on: every n-th
    assert len(lost) == 1 or lost == list(range(row, R, lost[1] - row))
    B.biv_softmax(x, p, 1.0)
    assert same_bits(p, good) and B.biv_device_error() == 0


def test_refusals():
    x = torch.zeros(2, 40000, device="cuda")
    for rows, v, row in ((2, 40000, 0), (2, 40000, 2), (2, 40000, -1), (2, 2000, 0), (2, 40002, 0)):
        y = torch.zeros(rows, v, device="cuda")
        with pytest.raises(B.BivError):
            B.biv_selftest_softmax_lost_row(y, torch.zeros_like(y), row)
    assert B.biv_device_error() == 0 and not bool(x.any())
