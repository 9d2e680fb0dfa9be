"""Which e4m3 number a value becomes: the quotient by its scale, rounded to fp32, and that to the nearest number of the
type, ties to even, bit for bit."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


def values(rows, K, kind):
    """Blocks of 128 values whose quotients are plain ones, exact ties, or near ties: small multiples of the largest's divisors."""
    g = U.gen(rows + K)
    if kind == "plain":
        return U.bf16(g, rows, K)
    # the largest is 448 2^n (a scale of 2^n: quotients are the values themselves) or some other number of 8 bits
    top = torch.full((rows, 1), 448.0) if kind == "ties" else torch.randint(128, 256, (rows, 1), generator=g).float()
    top = top * 2.0 ** torch.randint(-20, 20, (rows, 1), generator=g)
    steps = torch.randint(-448, 449, (rows, K), generator=g).float()       # odd numbers from 17 on: ties
    x = steps * top / 448.0 * 2.0 ** torch.randint(-12, 1, (rows, K), generator=g)
    x[:, ::128] = top
    return x.bfloat16()


@pytest.mark.parametrize("kind", ["plain", "ties", "near"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,K", [(3, 272), (256, 1024), (1500, 2048)])
def test_quant(gpu, rows, K, block, kind):
    x = values(rows, K, kind)
    if block == 128 and kind == "ties":
        x = torch.cat([x[:1] for _ in range(rows)])
    want, scales, each = E.quant(x, block)
    if kind == "ties":                                      # a part of the quotients lies half way between two numbers
        quot = (x.double() / each.double()).abs()
        step = 2.0 ** (quot.clamp(min=2.0 ** -6).log2().floor() - 3)
        assert ((quot / step).frac() == 0.5).float().mean() > 0.05
    q = torch.empty(rows, K, dtype=torch.uint8, device="cuda").view(E.E4M3)
    s = torch.empty_like(scales, device="cuda")
    B.biv_quant_e4m3(x.cuda(), q, s, block)
    assert torch.equal(s.cpu(), scales)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("kind", ["plain", "ties", "near"])
@pytest.mark.parametrize("hd", [64, 128])
def test_cache(gpu, hd, kind):
    """The blocks of a written cache, from the rows that the ring holds."""
    Hq, Hkv, K, page = 4, 2, 64, 32
    n = K // page + 1
    pools = [*[torch.zeros(n, Hkv, page, hd, dtype=torch.uint8, device="cuda").view(E.E4M3) for _ in "kv"],
             *[torch.zeros(n, Hkv, page // 16, dtype=torch.bfloat16, device="cuda") for _ in "kv"],
             *[torch.zeros(1, Hkv, 80, hd, dtype=torch.bfloat16, device="cuda") for _ in "kv"]]
    table = torch.arange(1, n, dtype=torch.int32, device="cuda").view(1, -1)
    qkv = values(K, (Hq + 2 * Hkv) * hd, kind).cuda()
    q = torch.empty(K, Hq, hd, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(K, dtype=torch.int32, device="cuda")
    B.biv_rope_kv_write_paged_e4m3(qkv, q, *pools, table, torch.zeros_like(pos), pos, 1e4, K)
    assert B.biv_device_error() == 0
    for x in range(2):
        rows = pools[4 + x][0, :, :K].cpu().view(Hkv, K // 16, 16, hd)
        s = E.scale_up(E.top(rows, (2, 3)))                                # [Hkv, blocks]
        want = (rows.double() / s.double()[..., None, None]).float().to(E.E4M3)
        got_s = pools[2 + x][1:].cpu().transpose(0, 1).reshape(Hkv, -1)
        got = pools[x][1:].cpu().view(torch.uint8).transpose(0, 1).reshape(Hkv, K // 16, 16, hd)
        assert torch.equal(got_s.view(torch.int16), s.view(torch.int16))
        assert torch.equal(got, want.view(torch.uint8))
