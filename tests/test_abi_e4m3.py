"""Refusals of the entry points on e4m3 numbers, host validation only (no GPU): the
pointers here are never dereferenced, the tensors have no memory."""
import math

import pytest
import torch

from invariant_verify_gb300 import abi as B

OK, NULL, SHAPE, ALIGN, VALUE, UNSUP = 0, 1, 2, 3, 4, 5
FAKE = 0x10000
MISALIGNED = 0x10008
BIG = (1 << 32) + 16                               # cut to 32 bits: 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_verify_gb300 import build
    build.build()
    return B.lib()


def caller(fn, **default):
    return lambda **kw: fn(*[kw.get(k, v) for k, v in default.items()])


def test_quant(lib):
    f = caller(lib.biv_quant_e4m3, x=FAKE, ld=256, rows=4, K=256, block=1, q=2 * FAKE, scales=3 * FAKE, s=None)
    assert f(rows=0) == OK
    for bad in (dict(rows=-1), dict(K=0), dict(K=24), dict(ld=255), dict(ld=260), dict(K=272)):
        assert f(**bad) == SHAPE
    for block in (0, 2, 64, 256, -1):
        assert f(block=block) == UNSUP
    for name in ("x", "q", "scales"):
        assert f(**{name: None}) == NULL
        assert f(**{name: MISALIGNED}) == ALIGN
    assert f(q=FAKE) == VALUE                      # in place


def test_gemm(lib):
    f = caller(lib.biv_gemm_e4m3, A=FAKE, sa=2 * FAKE, B=3 * FAKE, sb=4 * FAKE, bias=5 * FAKE, residual=6 * FAKE, C=7 * FAKE, dt=0,
               act=0, M=4, N=64, K=64, s=None)
    assert f(M=0) == OK
    for bad in (dict(M=-1), dict(N=0), dict(N=60), dict(K=0), dict(K=72)):
        assert f(**bad) == SHAPE
    for bad in (dict(dt=7), dict(act=-1), dict(act=5)):
        assert f(**bad) == VALUE
    for name in ("A", "sa", "B", "sb", "C"):
        assert f(**{name: None}) == NULL
    for name in ("A", "sa", "B", "sb", "bias", "residual", "C"):
        assert f(**{name: MISALIGNED}) == ALIGN
    for at in (1, 2, 3, 4, 5):
        assert f(C=at * FAKE) == VALUE             # C over an input
    assert f(C=6 * FAKE, dt=1) == VALUE            # an fp32 C over a bf16 residual


PAGES = dict(n_slots=4, max_pages=8, n_pages=16, page=64, tail=32)
POOLS = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, kt=FAKE, vt=FAKE)


def check_pools(f):
    for name in POOLS:
        assert f(**{name: None}) == NULL
    for name in ("k", "v"):                        # read 32 bytes at a time
        assert f(**{name: FAKE + 16}) == ALIGN
    for name in ("ks", "vs"):
        assert f(**{name: FAKE + 1}) == ALIGN
    for name in ("kt", "vt"):
        assert f(**{name: MISALIGNED}) == ALIGN
    for page in (1, 8, 24, 48, 512):
        assert f(page=page) == UNSUP
    for bad in (dict(n_slots=0), dict(n_pages=0), dict(max_pages=0), dict(max_pages=1 << 26), dict(page=0), dict(tail=0), dict(tail=-16),
                dict(tail=40), dict(Hq=7), dict(Hkv=0)):
        assert f(**bad) == SHAPE, bad
    for hd in (16, 96, 256):
        assert f(hd=hd) == UNSUP


def test_write(lib):
    f = caller(lib.biv_rope_kv_write_paged_e4m3, qkv=FAKE, q=FAKE, **POOLS, table=FAKE, slot=FAKE, pos=FAKE, keep=None, W=8, K=2, Hq=8,
               Hkv=2, hd=128, **PAGES, theta=10000.0, s=None)
    assert f(W=0) == OK
    assert f(W=7) == SHAPE
    assert f(K=0) == SHAPE
    assert f(W=0, K=17) == OK                      # 17 rows and 15 before them
    assert f(W=0, K=18) == SHAPE
    check_pools(f)
    for theta in (1.0, 0.0, -5.0, math.inf, math.nan):
        assert f(theta=theta) == VALUE
    for name in ("qkv", "q", "table", "slot", "pos"):
        assert f(**{name: None}) == NULL
    for name in ("qkv", "q"):
        assert f(**{name: MISALIGNED}) == ALIGN


def test_attention(lib):
    size = lib.biv_decode_attn_paged_workspace_size
    f = caller(lib.biv_decode_attn_paged_e4m3, q=FAKE, **POOLS, table=FAKE, slot=FAKE, pos=FAKE, o=2 * FAKE, W=8, rpg=1, Hq=8, Hkv=2,
               hd=128, **PAGES, ws=FAKE, ws_bytes=1 << 30, s=None)
    assert f(W=0) == OK
    assert f(W=-1) == SHAPE
    assert f(rpg=0) == SHAPE
    check_pools(f)
    assert f(ws_bytes=size(8, 8, 128, 8, 64) - 1) == SHAPE
    assert f(o=FAKE) == VALUE                      # o over q
    for name in ("q", "table", "slot", "pos", "o", "ws"):
        assert f(**{name: None}) == NULL
    for name in ("q", "o", "ws"):
        assert f(**{name: MISALIGNED}) == ALIGN


# --------------------------------------------------- sizes of more than 31 bits
def meta(*s, t=torch.bfloat16):
    return torch.empty(*s, dtype=t, device="meta")


def refused(fn, *args, **kw):
    with pytest.raises(B.BivError) as e:
        fn(*args, **kw)
    assert e.value.status == SHAPE and "31 bits" in str(e.value), str(e.value)


E4M3, F32, I32 = torch.float8_e4m3fn, torch.float32, torch.int32


def test_large_sizes():
    refused(B.biv_quant_e4m3, meta(BIG, 128), meta(BIG, 128, t=E4M3), meta(1, BIG, t=F32))
    refused(B.biv_quant_e4m3, meta(1, BIG), meta(1, BIG, t=E4M3), meta(BIG // 128 + 1, 1, t=F32))
    for M, N, K in ((BIG, 64, 128), (4, BIG, 128), (4, 64, BIG)):
        g = -(-K // 128)
        refused(B.biv_gemm_e4m3, meta(M, K, t=E4M3), meta(g, M, t=F32), meta(N, K, t=E4M3), meta(-(-N // 128), g, t=F32), meta(M, N))
    q, i = meta(8, 4, 64), lambda *s: meta(*s, t=I32)  # noqa: E731

    def cache(n_pages=9, slots=2, tail=32, wide=3):
        return [*[meta(n_pages, 2, 16, 64, t=E4M3)] * 2, *[meta(n_pages, 2, 1)] * 2, *[meta(slots, 2, tail, 64)] * 2, i(slots, wide)]

    for bad in (dict(n_pages=BIG), dict(slots=BIG), dict(tail=BIG), dict(wide=BIG)):
        c = cache(**bad)
        refused(B.biv_rope_kv_write_paged_e4m3, meta(8, 512), q, *c, i(8), i(8), 1e4, 8)
        refused(B.biv_decode_attn_paged_e4m3, q, *c, i(8), i(8), q, 8, meta(64, t=torch.uint8))
    refused(B.biv_rope_kv_write_paged_e4m3, meta(8, 512), q, *cache(), i(8), i(8), 1e4, BIG)
    refused(B.biv_decode_attn_paged_e4m3, q, *cache(), i(8), i(8), q, BIG, meta(64, t=torch.uint8))


def test_what_the_library_has_no_type_for():
    x, q = meta(4, 256, t=torch.float16), meta(4, 256, t=E4M3)
    with pytest.raises(B.BivError) as e:
        B.biv_quant_e4m3(x, q, meta(2, 4, t=F32))
    assert e.value.status == VALUE
    with pytest.raises(B.BivError) as e:
        B.biv_gemm_e4m3(q, meta(2, 4, t=F32), q, meta(1, 2, t=F32), meta(4, 4, t=torch.float16))
    assert e.value.status == VALUE
