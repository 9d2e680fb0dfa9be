"""The paged operators together, as a server runs them: a decoder's verify step
over pages, sampled verification, prefill, generation and its CUDA graph."""
import numpy as np
import pytest
import torch

import paged_util as U
from gpu_util import e2e_logit_envelope, same_bits
from oracle.model import OracleDecoder
from invariant_verify_gb300 import abi as B
from invariant_verify_gb300 import synth
from invariant_verify_gb300.paged import PagedVerifier, PagePool, paged_generate

pytestmark = pytest.mark.gpu

CFG = synth.DecoderConfig(name="paged test decoder", layers=2, d=256, Hq=8, Hkv=2, hd=128, ffn=320, vocab=2048,
                          temperature=0.9)


@pytest.fixture(scope="module")
def weights():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return synth.decoder_weights(CFG, seed=5)


def pool_for(slots, page=32, max_pages=16, n_pages=None):
    return PagePool(n_pages or slots * max_pages, page, CFG.layers, CFG.Hkv, CFG.hd, slots, max_pages)


def prompt(n, seed):
    return torch.randint(0, CFG.vocab, (n,), generator=U.gen(seed)).tolist()


def test_step_against_the_oracle(weights):
    """Logits of a window behind prefilled prompts: within the drift of bf16 storage
    that the oracle's composition gives (this path rounds at fewer places: the
    residual is added before a projection is rounded).  The emitted tokens are those
    that exact arithmetic gives for the kernel's own probabilities."""
    N, K = 3, 3
    prompts = [prompt(n, n) for n in (5, 40, 70)]
    ver = PagedVerifier(CFG, weights, pool_for(N), N, K)
    zero = torch.zeros(N, CFG.Hkv, 128, CFG.hd, dtype=torch.bfloat16)
    orc = OracleDecoder(CFG, weights, [(zero, zero) for _ in range(CFG.layers)], N, 128)
    for r, p in enumerate(prompts):
        ver.prefill(r, p[:-1])
        orc.forward(np.array(p[:-1]), np.full(len(p) - 1, r), np.arange(len(p) - 1))
        ver.pool.reserve(r, len(p) + K)
    g = U.gen(3)
    draft = torch.randint(0, CFG.vocab, (N, K), generator=g).int()
    ua, us = torch.rand(N, K, generator=g), torch.rand(N, generator=g)
    p0 = [len(p) - 1 for p in prompts]
    ver.set_window(range(N), [p[-1] for p in prompts], p0, draft, ua, us)
    ver.step()
    ref, tol = e2e_logit_envelope(orc, ver.tokens.cpu().numpy(), ver.row_slot.cpu().numpy(), ver.row_pos.cpu().numpy())
    drift = np.abs(ver.logits.cpu().numpy() - ref).max(axis=1)
    assert (drift <= tol).all(), (drift, tol)
    want = U.verify(ver.probs.cpu(), None, draft, ua, us, torch.tensor(p0).int())
    for got, w in zip((ver.emitted, ver.accept_len, ver.new_len), want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert B.biv_device_error() == 0


def test_biases_enter_the_projections(weights):
    """A bias equals the same column of the weight met by a constant input: here, zero
    weights and a bias alone reach the residual stream."""
    w = dict(weights)
    for l in range(CFG.layers):
        w[f"l{l}.wo"] = torch.zeros_like(w[f"l{l}.wo"])
        w[f"l{l}.wdown"] = torch.zeros_like(w[f"l{l}.wdown"])
        w[f"l{l}.bo"] = torch.full((CFG.d,), 0.5, dtype=torch.bfloat16)
        w[f"l{l}.bdown"] = torch.full((CFG.d,), 0.25, dtype=torch.bfloat16)
        w[f"l{l}.bqkv"] = torch.ones(CFG.qkv_n, dtype=torch.bfloat16)
    ver = PagedVerifier(CFG, w, pool_for(1), 1, 0)
    ver.pool.reserve(0, 1)
    ver.set_window([0], [7], [0], torch.zeros(1, 0), None, [0.5])
    ver.step()
    x = w["embed"][7].float()
    for _ in range(CFG.layers):
        x = (x + 0.5).bfloat16().float()
        x = (x + 0.25).bfloat16().float()
    assert torch.equal(ver.x[0].cpu().float(), x)


def test_requests_do_not_see_their_neighbours(weights):
    """A request alone, among others, in another seat and with other pages: the same bits."""
    K = 2
    prompts = [prompt(n, 10 + n) for n in (33, 64, 3, 100)]
    draft = torch.randint(0, CFG.vocab, (4, K), generator=U.gen(2)).int()
    us, ua = torch.rand(4, generator=U.gen(5)), torch.rand(4, K, generator=U.gen(6))

    def run(order, N, page):
        ver = PagedVerifier(CFG, weights, pool_for(N, page=page, max_pages=256 // page), N, K)
        for seat, r in enumerate(order):
            ver.prefill(seat, prompts[r][:-1])
            ver.pool.reserve(seat, len(prompts[r]) + K)
        ver.set_window(range(len(order)), [prompts[r][-1] for r in order], [len(prompts[r]) - 1 for r in order],
                       draft[order], ua[order], us[order])
        ver.step()
        assert B.biv_device_error() == 0
        probs = ver.probs.view(N, K + 1, -1)
        return {r: (probs[s].clone(), ver.emitted[s].clone()) for s, r in enumerate(order)}

    every = run([0, 1, 2, 3], 4, 32)
    for other in (run([2], 1, 16), run([3, 0], 7, 64), run([1], 3, 128), run([3, 2, 1, 0], 4, 16)):
        for r, (p, t) in other.items():
            assert same_bits(p, every[r][0]) and torch.equal(t, every[r][1]), r


def test_generation_with_and_without_drafts_at_temperature_zero(weights):
    """T = 0 leaves one possible text: the n-gram drafter only changes how many steps it takes."""
    prompts = [prompt(20, 1) * 2, prompt(7, 2), prompt(50, 3)]
    plain = PagedVerifier(CFG, weights, pool_for(3), 3, 0, temperature=0.0)
    drafted = PagedVerifier(CFG, weights, pool_for(4, page=64, max_pages=8), 4, 4, temperature=0.0)
    a, per_a = paged_generate(plain, prompts, 40)
    b, per_b = paged_generate(drafted, prompts, 40)
    assert a == b and per_a == 1.0 and per_b >= 1.0
    assert B.biv_device_error() == 0


def test_generation_goes_by_the_generator(weights):
    prompts = [prompt(9, 4), prompt(30, 5)]
    runs = []
    for seed in (1, 1, 2):
        ver = PagedVerifier(CFG, weights, pool_for(2), 2, 3)
        runs.append(paged_generate(ver, prompts, 24, U.gen(seed))[0])
    assert runs[0] == runs[1] != runs[2]
    assert all(len(t) == 24 and all(0 <= x < CFG.vocab for x in t) for t in runs[0])


def test_captured_step_equals_the_eager_one(weights):
    """One graph, replayed on windows with empty seats and without, beside an eager
    verifier on a pool of its own; draft probabilities given."""
    N, K = 3, 2
    prompts = [prompt(n, 20 + n) for n in (12, 90, 31)]
    eager, graphed = (PagedVerifier(CFG, weights, pool_for(N), N, K) for _ in range(2))
    q = torch.empty(N * K, CFG.vocab, device="cuda")
    q.fill_(1.0 / CFG.vocab)
    for v in (eager, graphed):
        for r, p in enumerate(prompts):
            v.prefill(r, p[:-1])
            v.pool.reserve(r, 128)
        v.set_window([], [], [], torch.zeros(0, K))
    graph = graphed.capture(q)
    g = U.gen(1)
    for i, order in enumerate(([0, 1, 2], [1], [2, 0])):
        n = len(order)
        q.copy_(torch.softmax(torch.randn(N * K, CFG.vocab, generator=g), 1))
        args = (order, [prompts[r][-1] for r in order], [len(prompts[r]) - 1 for r in order],
                torch.randint(0, CFG.vocab, (n, K), generator=g), torch.rand(n, K, generator=g), torch.rand(n, generator=g))
        for v in (eager, graphed):
            v.set_window(*args)
        eager.step(q)
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(eager.probs[:n * (K + 1)], graphed.probs[:n * (K + 1)])
        assert torch.equal(eager.emitted[:n], graphed.emitted[:n])
        assert all(same_bits(a, b) for a, b in zip(eager.pool.k + eager.pool.v, graphed.pool.k + graphed.pool.v))
    assert B.biv_device_error() == 0
