"""The last sizes that 32-bit integers hold (host validation only; the pointers are never dereferenced)."""
import pytest

from invariant_verify_gb300 import abi as B

OK, NULL, SHAPE = 0, 1, 2
LAST = 0x7fffffff
FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_verify_gb300 import build
    build.build()
    return B.lib()


def test_gemm(lib):
    """Tiles and blocks are counted in 32 bits: sizes whose rounding up would pass them are refused."""
    def f(M, N, K):
        return lib.biv_gemm_e4m3(None, None, None, None, None, None, None, 0, 0, M, N, K, None)
    top = LAST - 255
    assert f(top, 64, 64) == f(4, top // 16 * 16, 64) == f(4, 64, top // 16 * 16) == NULL
    for M in (top + 1, LAST - 31, LAST):
        assert f(M, 64, 64) == SHAPE
    for N in (LAST - 7, LAST - 127):
        assert f(4, N, 64) == SHAPE
    for K in (LAST - 15, LAST - 127):
        assert f(4, 64, K) == SHAPE


@pytest.mark.parametrize("block", [1, 128])
def test_quant(lib, block):
    """The number of groups of the longest rows; and how many blocks a grid holds."""
    K = LAST - 15

    def f(rows, K):
        return lib.biv_quant_e4m3(None, K, rows, K, block, None, None, None)
    assert f(1, K) == f(3, K - 112) == NULL
    assert f(LAST, K) == SHAPE
    assert f(LAST, 16) == NULL
