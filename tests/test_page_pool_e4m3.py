"""The page pool of a cache in e4m3, and what the verifier refuses (host only)."""
import pytest
import torch

from invariant_verify_gb300 import synth
from invariant_verify_gb300.paged import PagedVerifier, PagePool


def pool(page=32, tail=32):
    return PagePool(4, page, 2, 3, 64, 5, 6, device="cpu", tail=tail)


def test_layout():
    p = pool()
    for l in range(2):
        k, v, ks, vs, kt, vt = p.layer(l)
        assert k.shape == v.shape == (4, 3, 32, 64) and k.dtype == v.dtype == torch.float8_e4m3fn
        assert ks.shape == vs.shape == (4, 3, 2) and ks.dtype == vs.dtype == torch.bfloat16
        assert kt.shape == vt.shape == (5, 3, 32, 64) and kt.dtype == vt.dtype == torch.bfloat16
        assert all(int(t.view(torch.uint8).max()) == 0 and t.is_contiguous() for t in (k, v, ks, vs, kt, vt))
    k, v = pool(tail=None).layer(0)
    assert k.dtype == v.dtype == torch.bfloat16 and k.shape == (4, 3, 32, 64)


@pytest.mark.parametrize("page,tail", [(32, 0), (32, 17), (8, 32), (32, -16)])
def test_refused_pools(page, tail):
    with pytest.raises(ValueError, match="multiples of 16"):
        pool(page, tail)


def test_refused_verifiers():
    cfg = synth.DecoderConfig(name="refused", layers=2, d=64, Hq=3, Hkv=3, hd=64, ffn=64, vocab=64)
    with pytest.raises(ValueError, match="wk"):
        PagedVerifier(cfg, {}, pool(), 1, 0, device="cpu", held=("wk",))
    with pytest.raises(ValueError, match="tail of 33"):
        PagedVerifier(cfg, {}, pool(), 1, 17, device="cpu")
