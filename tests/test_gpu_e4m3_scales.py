"""Products of e4m3 matrices whose scales lie far from one: the product of two scales may pass fp32's range at either end
where the sum that it multiplies brings the result back."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -126                                         # the smallest normal number
SHAPES = [(7, 136, 272), (70, 12000, 272), (200, 1040, 400), (300, 12904, 144), (256, 28672, 144)]


def run(A, sa, Bm, sb, M, out):
    C = torch.full((M, Bm.shape[0]), float("nan"), dtype=out, device="cuda")
    B.biv_gemm_e4m3(A, sa, Bm, sb, C)
    return C.cpu().double()


def each(s, K):                                             # [rows, groups] -> [rows, K]
    return s.double().repeat_interleave(128, 1)[:, :K]


def spread(n, groups, exponents, g):
    """Scales [n, groups] whose exponents go by the row."""
    e = torch.tensor(exponents)[torch.arange(n) % len(exponents)].double()
    return ((1 + torch.rand(n, groups, generator=g).double()) * 2.0 ** e[:, None]).float(), e


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_scales_of_every_size(gpu, M, N, K, out):
    """Products of scales from 2^-200 to 2^137.  Large scales meet values of 2^-9, so that every result is finite: below
    4 x 2^135 x 2^-18 x 400.  Tolerance: the sum's, half a step of the result, and fp32's and the output's smallest
    half steps."""
    B.biv_device_error()
    g = U.gen(M + N)
    groups, blocks = -(-K // 128), -(-N // 128)
    sa, rows = spread(M, groups, [-100, -60, 0, 45, 70], g)
    sb, cols = spread(blocks, groups, [-30, 65, -100, -41, 0, 58], g)
    sb, cols = sb.repeat_interleave(128, 0)[:N], cols.repeat_interleave(128)[:N]
    a, b = torch.randn(M, K, generator=g) * 40, torch.randn(N, K, generator=g) * 40
    A = torch.where(rows[:, None] > 40, a.sign() * 2.0 ** -9, a).to(E.E4M3)
    Bm = torch.where(cols[:, None] > 40, b.sign() * 2.0 ** -9, b).to(E.E4M3)
    want, size = E.gemm(A, each(sa, K), Bm, each(sb, K))
    assert want.abs().max() < 3e38
    C = run(A.cuda(), sa.t().contiguous().cuda(), Bm.cuda(), sb[::128].contiguous().cuda(), M, out)
    tol = E.gemm_tolerance(size, K) + want.abs() * U.HALF_STEP[out] + LEAST * U.HALF_STEP[out] + (groups + 4) * 2.0 ** -149
    bad = ~((C - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), C[bad][:4], want[bad][:4])
    # the case is what it says: there are normal results of products below the normal numbers
    below = (rows[:, None] + cols[None] < -128).expand(M, N)
    assert (want.abs()[below] > 8 * LEAST).any()
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_zeros_under_scales_whose_product_overflows(gpu, M, N, K):
    """Rows of zeros stay zeros; sums of positive products, some 2^150, are infinite."""
    g = U.gen(3)
    groups, blocks = -(-K // 128), -(-N // 128)
    a, b = (torch.randn(n, K, generator=g).abs() for n in (M, N))
    a[::3] = 0
    A, Bm = a.to(E.E4M3), b.to(E.E4M3)
    sa, sb = torch.full((groups, M), 2.0 ** 90), torch.full((blocks, groups), 2.0 ** 60)
    C = run(A.cuda(), sa.cuda(), Bm.cuda(), sb.cuda(), M, torch.float32)
    assert (C[::3] == 0).all()
    assert (C[1::3] == float("inf")).all()
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_rows_beside_rows_of_far_scales(gpu, M, N, K):
    """A row's bits do not depend on its neighbours' scales, nor on how many there are."""
    g = U.gen(4)
    groups, blocks = -(-K // 128), -(-N // 128)
    A, Bm = (torch.randn(n, K, generator=g).to(E.E4M3) for n in (M, N))
    sa, sb = torch.rand(groups, M, generator=g) + 0.5, torch.rand(blocks, groups, generator=g) + 0.5
    sb[::2] *= 2.0 ** -60
    sa[:, 1::2] *= 2.0 ** -80
    C = run(A.cuda(), sa.cuda(), Bm.cuda(), sb.cuda(), M, torch.float32)
    plain = sa.clone()
    plain[:, 1::2] = 1.0
    D = run(A.cuda(), plain.cuda(), Bm.cuda(), sb.cuda(), M, torch.float32)
    assert same_bits(C[::2], D[::2])
    r = slice(M - 2, M)
    E2 = run(A[r].cuda(), sa[:, r].contiguous().cuda(), Bm.cuda(), sb.cuda(), 2, torch.float32)
    assert same_bits(E2, C[r])


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_blocks_of_zeros_under_the_least_scale(gpu, M, N, K):
    """Empty rows and blocks of weights have the least scale; what meets there makes nothing, not the sign of a zero either,
    whatever other rows and blocks ask for."""
    g = U.gen(6)
    groups, blocks = -(-K // 128), -(-N // 128)
    A, Bm = (torch.randn(n, K, generator=g).to(E.E4M3) for n in (M, N))
    sa, sb = torch.full((groups, M), 2.0 ** -100), torch.full((blocks, groups), 2.0 ** -100)
    sa[:, 1::2] = 0.7
    sb[1::2] = 0.9
    C = run(A.cuda(), sa.cuda(), Bm.cuda(), sb.cuda(), M, torch.float32)
    assert (C[::2, :128] == 0).all() and (C[1::2, 128:256] != 0).any()
    sa[:, 1::2] = 2.0 ** -60                                # products of 2^-160
    D = run(A.cuda(), sa.cuda(), Bm.cuda(), sb.cuda(), M, torch.float32)
    assert same_bits(C[::2], D[::2])
    want = (A.float().double() @ Bm.float().double().t())[1::2, :128] * 2.0 ** -160
    assert (D[1::2, :128] - want).abs().max() <= (groups + 4) * 2.0 ** -149 + want.abs().max() * 2.0 ** -18


def test_small_values_through_the_quantiser(gpu):
    """bf16 values of some 1e-30 and 1e-7, as biv_quant_e4m3 holds them: results of some 1e-36, to fp32's precision."""
    M, N, K = 40, 256, 512
    g = U.gen(5)
    x, w = (torch.randn(M, K, generator=g) * 1e-30).bfloat16().cuda(), (torch.randn(N, K, generator=g) * 1e-7).bfloat16().cuda()
    q8 = lambda r, k: torch.empty(r, k, dtype=torch.uint8, device="cuda").view(E.E4M3)  # noqa: E731
    A, sa, Bm, sb = q8(M, K), torch.empty(4, M, device="cuda"), q8(N, K), torch.empty(2, 4, device="cuda")
    B.biv_quant_e4m3(x, A, sa, 1)
    B.biv_quant_e4m3(w, Bm, sb, 128)
    C = run(A, sa, Bm, sb, M, torch.float32)
    ea, eb = each(sa.cpu().t(), K), each(sb.cpu().repeat_interleave(128, 0), K)
    want, size = E.gemm(A.cpu(), ea, Bm.cpu(), eb)
    assert want.abs().max() > 8 * LEAST
    assert ((C - want).abs() <= E.gemm_tolerance(size, K) + LEAST * 2.0 ** -24).all()
