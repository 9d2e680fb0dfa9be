"""Refusals of the paged and sampled entry points, host validation only (no GPU):
the pointers here are never dereferenced."""
import math

import pytest
import torch

OK, NULL, SHAPE, ALIGN, VALUE, UNSUP, DEVICE = 0, 1, 2, 3, 4, 5, 7
FAKE = 0x10000
MISALIGNED = 0x10008


@pytest.fixture(scope="module")
def lib():
    from invariant_verify_gb300 import abi, build
    build.build()
    return abi.lib()


def caller(fn, **default):
    return lambda **kw: fn(*[kw.get(k, v) for k, v in default.items()])


def test_gemm_bias_act(lib):
    f = caller(lib.biv_gemm_bias_act, A=FAKE, B=2 * FAKE, bias=3 * FAKE, residual=4 * FAKE, C=5 * FAKE, dt=0, act=0,
               M=4, N=64, K=64, s=None)
    assert f(M=0) == OK
    assert f(M=-1) == SHAPE
    assert f(N=60) == SHAPE
    assert f(K=60) == SHAPE
    assert f(dt=7) == VALUE
    assert f(act=-1) == VALUE
    assert f(act=5) == VALUE
    assert f(A=None) == NULL
    assert f(bias=MISALIGNED) == ALIGN
    assert f(residual=MISALIGNED) == ALIGN
    assert f(C=MISALIGNED) == ALIGN
    assert f(C=FAKE) == VALUE                      # C over A
    assert f(C=3 * FAKE) == VALUE                  # C over the bias
    assert f(C=4 * FAKE, dt=1) == VALUE            # an fp32 C over a bf16 residual


PAGES = dict(n_slots=4, max_pages=8, n_pages=16, page=64)


def test_rope_kv_write_paged(lib):
    f = caller(lib.biv_rope_kv_write_paged, qkv=FAKE, q=FAKE, k=FAKE, v=FAKE, table=FAKE, slot=FAKE, pos=FAKE,
               keep=None, W=8, K=2, Hq=8, Hkv=2, hd=128, **PAGES, theta=10000.0, s=None)
    assert f(W=0) == OK
    assert f(W=7) == SHAPE
    assert f(K=0) == SHAPE
    assert f(hd=24) == SHAPE
    assert f(hd=272) == SHAPE
    assert f(Hkv=0) == SHAPE
    assert f(n_pages=0) == SHAPE
    assert f(max_pages=1 << 26) == SHAPE           # positions past 31 bits
    for page in (1, 8, 24, 48, 512):
        assert f(page=page) == UNSUP
    assert f(page=0) == SHAPE
    for theta in (1.0, 0.0, -5.0, math.inf, math.nan):
        assert f(theta=theta) == VALUE
    for name in ("qkv", "q", "k", "v", "table", "slot", "pos"):
        assert f(**{name: None}) == NULL
    for name in ("qkv", "q", "k", "v"):
        assert f(**{name: MISALIGNED}) == ALIGN


def test_decode_attn_paged(lib):
    size = lib.biv_decode_attn_paged_workspace_size
    assert size(64, 8, 128, 36, 64) == 64 * 8 * 9 * 130 * 4 + 16
    assert size(1, 1, 64, 1, 16) == 66 * 4 + 16
    assert size(0, 8, 128, 36, 64) == 0
    f = caller(lib.biv_decode_attn_paged, q=FAKE, k=FAKE, v=FAKE, table=FAKE, slot=FAKE, pos=FAKE, o=2 * FAKE, W=8,
               rpg=1, Hq=8, Hkv=2, hd=128, **PAGES, ws=FAKE, ws_bytes=1 << 30, s=None)
    assert f(W=0) == OK
    assert f(W=-1) == SHAPE
    assert f(rpg=0) == SHAPE
    assert f(Hq=7) == SHAPE
    assert f(hd=96) == UNSUP
    assert f(hd=256) == UNSUP
    for name in ("k", "v"):                        # read 32 bytes at a time
        assert f(**{name: FAKE + 16}) == ALIGN
    assert f(page=8) == UNSUP
    assert f(n_slots=0) == SHAPE
    assert f(ws_bytes=size(8, 8, 128, 8, 64) - 1) == SHAPE
    assert f(ws=None) == NULL
    assert f(o=FAKE) == VALUE                      # o over q
    for name in ("q", "k", "v", "table", "slot", "pos", "o"):
        assert f(**{name: None}) == NULL
    for name in ("q", "k", "v", "o", "ws"):
        assert f(**{name: MISALIGNED}) == ALIGN


def test_softmax(lib):
    f = caller(lib.biv_softmax, x=FAKE, R=4, V=100, ld=100, T=1.0, p=2 * FAKE, ldp=104, s=None)
    assert f(R=0) == OK
    assert f(R=-1) == SHAPE
    assert f(V=0) == SHAPE
    assert f(ld=99) == SHAPE
    assert f(ldp=99) == SHAPE
    assert f(V=(1 << 22) + 1, ld=1 << 23, ldp=1 << 23) == UNSUP
    for T in (-1.0, math.nan, math.inf):
        assert f(T=T) == VALUE
    assert f(x=None) == NULL
    assert f(p=None) == NULL
    assert f(p=FAKE + 2) == ALIGN
    assert f(p=FAKE) == VALUE                      # in place with another leading dimension


def test_verify_sample(lib):
    f = caller(lib.biv_verify_sample, p=FAKE, q=FAKE, d=FAKE, ua=FAKE, us=FAKE, p0=FAKE, N=2, K=3, V=100, t=FAKE, a=FAKE,
               n=FAKE, s=None)
    assert f(N=0) == OK
    assert f(N=-1) == SHAPE
    assert f(K=-1) == SHAPE
    assert f(K=1025) == SHAPE
    assert f(V=0) == SHAPE
    assert f(V=(1 << 22) + 1) == UNSUP
    for name in ("p", "d", "ua", "us", "p0", "t", "a", "n"):
        assert f(**{name: None}) == NULL


# -------------------------------------------------- the Python binding's own checks
def refused(status, fn, *a, **kw):
    from invariant_verify_gb300.abi import BivError
    with pytest.raises(BivError) as e:
        fn(*a, **kw)
    assert e.value.status == status, str(e.value)


def test_binding_refuses_wrong_tensors(lib):
    from invariant_verify_gb300 import abi as B
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    refused(VALUE, B.biv_gemm_bias_act, z(4, 64).half(), z(64, 64), z(4, 64))
    refused(VALUE, B.biv_gemm_bias_act, z(4, 64), z(64, 64), z(4, 64).half())
    refused(VALUE, B.biv_gemm_bias_act, z(4, 64), z(64, 64), z(4, 64), act="swish")
    refused(SHAPE, B.biv_gemm_bias_act, z(4, 64), z(64, 64), z(4, 64), bias=z(63))
    refused(SHAPE, B.biv_gemm_bias_act, z(64, 4).t(), z(64, 64), z(4, 64))
    refused(DEVICE, B.biv_gemm_bias_act, z(4, 64), z(64, 64), z(4, 64))
    pool, q = z(9, 2, 16, 128), z(4, 8, 128)
    ws = torch.zeros(64, dtype=torch.uint8)
    refused(VALUE, B.biv_decode_attn_paged, q, pool, pool.half(), i(4, 3), i(4), i(4), z(4, 8, 128), 1, ws)
    refused(SHAPE, B.biv_decode_attn_paged, q, pool, z(9, 2, 32, 128), i(4, 3), i(4), i(4), z(4, 8, 128), 1, ws)
    refused(SHAPE, B.biv_decode_attn_paged, q, pool, pool, i(4, 3), i(4), i(4), z(4, 8, 64), 1, ws)
    refused(DEVICE, B.biv_decode_attn_paged, q, pool, pool, i(4, 3), i(4), i(4), z(4, 8, 128), 1, ws)
    refused(SHAPE, B.biv_rope_kv_write_paged, z(4, 11 * 128), q, pool, pool, i(4, 3), i(4), i(4), 1e4, 1)
    refused(DEVICE, B.biv_rope_kv_write_paged, z(4, 12 * 128), q, pool, pool, i(4, 3), i(4), i(4), 1e4, 1)
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    refused(VALUE, B.biv_softmax, f(4, 8).double(), f(4, 8), 1.0)
    refused(SHAPE, B.biv_softmax, f(4, 8), f(4, 7), 1.0)
    refused(SHAPE, B.biv_softmax, f(8, 4).t(), f(4, 8), 1.0)
    refused(SHAPE, B.biv_softmax, f(1, 8).expand(4, 8), f(4, 8), 1.0)      # one row for all: not a matrix of rows
    refused(DEVICE, B.biv_softmax, f(4, 8), f(4, 8), 1.0)
    refused(SHAPE, B.biv_verify_sample, f(5, 10), f(4, 10), i(2, 2), f(2, 2), f(2), i(2), i(2, 3), i(2), i(2))
    refused(VALUE, B.biv_verify_sample, f(6, 10), f(4, 10), i(2, 2), f(2, 2).double(), f(2), i(2), i(2, 3), i(2), i(2))
    refused(DEVICE, B.biv_verify_sample, f(6, 10), f(4, 10), i(2, 2), f(2, 2), f(2), i(2), i(2, 3), i(2), i(2))
