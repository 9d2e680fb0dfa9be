"""The forms of the product of e4m3 matrices and of the attention that a call may take, each at sizes where it runs through
all of its parts: more k-blocks than scales are copied at once, several tiles a CTA, rows of more splits than a warp joins."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def operands(M, N, K):
    """e4m3 matrices and scales on the GPU, with their values in 64 bits."""
    g = torch.Generator("cuda").manual_seed(M + N + K)
    groups, blocks = -(-K // 128), -(-N // 128)
    a, b = (torch.randn(n, K, generator=g, device="cuda").mul_(60).to(E.E4M3) for n in (M, N))
    sa, sb = (torch.rand(*s, generator=g, device="cuda") + 0.5 for s in ((groups, M), (blocks, groups)))
    wide = lambda s: s.double().repeat_interleave(128, 1)[:, :K]  # noqa: E731
    return a, sa, b, sb, a.float().double() * wide(sa.t()), b.float().double() * wide(sb.repeat_interleave(128, 0)[:N])


# tile widths of one row tile: 16 ceil(N / (16 SMs)); wider: by the rule on waves
@pytest.mark.parametrize("width", [16, 32, 48, 64, 80, 128, 144, 192, 208, 224, 240, 256])
@pytest.mark.parametrize("M,K", [(3, 2192), (64, 2304), (97, 4224), (128, 2176)])
def test_gemm_of_one_row_tile(gpu, M, K, width):
    """A tile for every SM, all widths, and an odd and an even number of k-blocks above sixteen."""
    check(M, sms() * width - 8, K)


@pytest.mark.parametrize("M,tiles,K", [(128, 400, 2176), (128, 600, 2304), (256, 150, 4224), (256, 300, 2176), (300, 110, 2192), (320, 300, 2304), (512, 112, 4224),
                                       (513, 80, 2176), (1023, 76, 4096)])
def test_gemm_of_several_waves(gpu, M, tiles, K):
    """Several tiles a CTA, or a pair: ``tiles`` times 128 columns on a GPU of 152 SMs."""
    check(M, tiles * 128 * sms() // 152 // 8 * 8, K)


def check(M, N, K):
    B.biv_device_error()
    a, sa, b, sb, va, vb = operands(M, N, K)
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    C = torch.full((M, N), float("nan"), device="cuda")
    B.biv_gemm_e4m3(a, sa, b, sb, C)
    tol = E.gemm_tolerance(size, K) + want.abs() * E.F32_STEP
    bad = ~((C.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((C.double() - want).abs() / tol).max()))
    half = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    B.biv_gemm_e4m3(a, sa, b, sb, half)
    assert same_bits(half, C.bfloat16())
    for rows in (slice(0, 1), slice(max(0, M - 33), M)):    # other forms, the same bits
        few = torch.empty(rows.stop - rows.start, N, device="cuda")
        B.biv_gemm_e4m3(a[rows].contiguous(), sa[:, rows].contiguous(), b, sb, few)
        assert same_bits(few, C[rows])
    assert B.biv_device_error() == 0


def attend(pool, q, slot, pos, rpg):
    W, Hq, hd = q.shape
    o = torch.full((W, Hq, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.biv_decode_attn_paged_workspace_size(W, Hq, hd, pool.table.shape[1], pool.page), dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B.biv_decode_attn_paged_e4m3(q.cuda(), *pool.on(), i32(slot), i32(pos), o, rpg, ws)
    return o


@pytest.mark.parametrize("hd,page", [(64, 256), (128, 64)])
def test_attention_of_more_splits_than_a_warp_joins(gpu, hd, page):
    """64 splits of 512 keys are 32768: rows on both sides, a window over the border, and so many rows that the joins take the
    other size of CTA."""
    B.biv_device_error()
    pool = E.HeldPool([33301, 32768, 70], 1, hd, page, seed=2, tail=48)
    q = U.bf16(U.gen(2), 3, 4, hd, std=1.5)
    slot, pos = [0, 1, 2], [33300, 32767, 69]
    o = attend(pool, q, slot, pos, 1)
    want, tol = E.attention(q, pool, slot, pos)
    assert ((o.cpu().double() - want).abs() <= tol).all()
    # positions 32767 and 32768 end and begin a split
    pool.lengths[0], ring = 32776, pool.tails
    for x in range(2):
        for t in range(32776 - 48, 32776):
            ring[x][0, :, t % 48] = pool.rows[0][x][:, t]
    K = 16
    w = U.bf16(U.gen(3), K, 4, hd, std=1.5)
    at = [32760 + j for j in range(K)]
    y = attend(pool, w, [0] * K, at, K)
    want, tol = E.attention(w, pool, [0] * K, at)
    assert ((y.cpu().double() - want).abs() <= tol).all()
    assert same_bits(attend(pool, w, [0] * K, at, 1), y)
    n = 16 * sms() // 4 // K + 1                            # groups of 4 heads: more pairs than 16 an SM
    many = attend(pool, w.repeat(n, 1, 1), [0] * K * n, at * n, K)
    assert same_bits(many, y.repeat(n, 1, 1))
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("std", [3e3, 3e4, 1e20])
def test_attention_of_large_queries(gpu, hd, std):
    """One key takes all of the weight: the row is that key's value, to half a bf16 step; a row of zeros is the mean.  A score
    may be off by (hd + 4) 2^-23 of the sum of its products' sizes; where the best leads by twice that and 30, the others
    weigh e^-30 each, 2^-24 of the largest |v| for the 400 of them;
    a weight of the row's own block keeps 16 bits."""
    B.biv_device_error()
    lengths, Hq, Hkv = [200, 333, 64, 17, 400], 8, 2
    pool = E.HeldPool(lengths, Hkv, hd, 32, seed=6)
    N = len(lengths)
    q = U.bf16(U.gen(5), N, Hq, hd, std=std)
    q[:, 0] = 0
    pos = [n - 1 for n in lengths]
    o = attend(pool, q, list(range(N)), pos, 1).cpu().double()
    sure = 0
    for r in range(N):
        k, v = E.seen(pool, r, pos[r])
        for h in range(Hq):
            kh, vh, qh = k[h // (Hq // Hkv)], v[h // (Hq // Hkv)], q[r, h].double()
            if h == 0:
                want = vh.mean(0)
                tol = want.abs() * U.HALF_STEP[torch.bfloat16] + (2.0 ** -11 + 2.0 ** -14) * vh.abs().mean(0)
            else:
                s = kh @ qh * hd ** -0.5
                ds = (kh.abs() @ qh.abs()).max() * hd ** -0.5 * (hd + 4) * 2.0 ** -23
                top = s.topk(2).values
                if top[0] - top[1] < 2 * ds + 30:
                    continue
                sure += 1
                want = vh[int(s.argmax())]
                tol = want.abs() * (U.HALF_STEP[torch.bfloat16] + 2.0 ** -16) + 2.0 ** -24 * vh.abs().max()
            assert ((o[r, h] - want).abs() <= tol).all(), (r, h)
    assert sure > N * (Hq - 1) * 3 // 4
    assert B.biv_device_error() == 0
