"""The biases of a paged verifier's projections, each in its place."""
import pytest
import torch

import paged_util as U
from invariant_verify_gb300 import abi as B
from invariant_verify_gb300 import synth
from invariant_verify_gb300.paged import PagedVerifier, PagePool

pytestmark = pytest.mark.gpu

CFG = synth.DecoderConfig(name="paged bias decoder", layers=3, d=256, Hq=4, Hkv=2, hd=64, ffn=320, vocab=512, temperature=1.0)


def test_every_layer_adds_its_own_qkv_bias():
    """Output projections of zero leave the residual stream at the embedding, so that every
    layer's q, k and v are those of the embedding's norm, plus the layer's bias."""
    w = dict(synth.decoder_weights(CFG, seed=7))
    g = U.gen(3)
    for l in range(CFG.layers):
        w[f"l{l}.wo"] = torch.zeros_like(w[f"l{l}.wo"])
        w[f"l{l}.wdown"] = torch.zeros_like(w[f"l{l}.wdown"])
        w[f"l{l}.bqkv"] = U.bf16(g, CFG.qkv_n, std=2.0)
    n, page, slot = 37, 16, 1
    pool = PagePool(8, page, CFG.layers, CFG.Hkv, CFG.hd, 2, 4)
    ver = PagedVerifier(CFG, w, pool, 1, 4)
    prompt = torch.randint(0, CFG.vocab, (n,), generator=g)
    ver.prefill(slot, prompt)
    torch.cuda.synchronize()
    x = w["embed"].cpu()[prompt].cuda().contiguous()
    h = torch.empty_like(x)
    pages = pool.table[slot].cpu().tolist()
    pos = torch.arange(n)
    for l in range(CFG.layers):
        B.biv_rmsnorm(x, w[f"l{l}.attn_norm"].cuda(), h, CFG.eps)
        a, b, bias = h.double().cpu(), w[f"l{l}.wqkv"].double().cpu(), w[f"l{l}.bqkv"].double()
        y = a @ b.T + bias
        # half a step of bf16 for qkv; K partial sums in fp32
        tol = U.HALF_STEP[torch.bfloat16] * y.abs() + CFG.d * 2.0 ** -23 * (a.abs() @ b.abs().T + bias.abs())
        y, tol = (t.view(n, -1, CFG.hd) for t in (y, tol))
        Hq, Hkv, half = CFG.Hq, CFG.Hkv, CFG.hd // 2
        k, v = y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
        kt, vt = tol[:, Hq:Hq + Hkv], tol[:, Hq + Hkv:]
        k = U.rope(k, pos, CFG.rope_theta)
        # the rotation mixes two errors, and rounds to bf16 once more
        kt = kt + torch.cat([kt[..., half:], kt[..., :half]], -1)
        kt = kt + (U.HALF_STEP[torch.bfloat16] + 2.0 ** -20) * (k.abs() + kt)
        got = [torch.cat([p[i] for i in pages[:-(-n // page)]], 1)[:, :n].permute(1, 0, 2).double().cpu() for p in (pool.k[l], pool.v[l])]
        assert bool(((got[0] - k).abs() <= kt).all()), l
        assert bool(((got[1] - v).abs() <= vt).all()), l
        if l + 1 == CFG.layers:                    # q of the last window's rows
            m = (n - 1) % ver.W + 1
            q = U.rope(y[n - m:, :Hq], pos[n - m:], CFG.rope_theta)
            qt = tol[n - m:, :Hq]
            qt = qt + torch.cat([qt[..., half:], qt[..., :half]], -1)
            qt = qt + (U.HALF_STEP[torch.bfloat16] + 2.0 ** -20) * (q.abs() + qt)
            assert bool(((ver.q[:m].double().cpu() - q).abs() <= qt).all())
    assert B.biv_device_error() == 0
