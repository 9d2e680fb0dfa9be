"""The operators on e4m3 numbers together, as a server runs them: a decoder's verify step with
its weights, its cache or both in 8 bits."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B
from invariant_verify_gb300 import synth
from invariant_verify_gb300.paged import PagedVerifier, PagePool, paged_generate

pytestmark = pytest.mark.gpu

CFG = synth.DecoderConfig(name="e4m3 test decoder", layers=2, d=256, Hq=8, Hkv=2, hd=128, ffn=320, vocab=2048,
                          temperature=0.9)
ALL = PagedVerifier.HELD


@pytest.fixture(scope="module")
def weights():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    w = synth.decoder_weights(CFG, seed=5)
    w["l0.bqkv"] = synth.bf16_normal((CFG.qkv_n,), 0.1, synth.generator(1))
    w["l1.bdown"] = synth.bf16_normal((CFG.d,), 0.1, synth.generator(2))
    return w


def verifier(weights, N, K, page=32, max_pages=8, tail=48, held=ALL, cls=PagedVerifier, **kw):
    return cls(CFG, weights, PagePool(N * max_pages, page, CFG.layers, CFG.Hkv, CFG.hd, N, max_pages, tail=tail), N, K, held=held, **kw)


def prompt(n, seed):
    return torch.randint(0, CFG.vocab, (n,), generator=U.gen(seed)).tolist()


class Checked(PagedVerifier):
    """Every product of the step against 64 bits on the inputs that it had."""

    seen = 0

    def project(self, x, name, out, bias=None, residual=None):
        before = x.cpu(), None if residual is None else residual.cpu()
        super().project(x, name, out, bias=bias, residual=residual)
        W = x.shape[0]
        a, _, each_a = E.quant(before[0], 1)
        b, _, each_b = E.quant(self.weights[name].cpu(), 128)
        want, size = E.gemm(a, each_a, b, each_b)
        tol = E.gemm_tolerance(size, x.shape[1])
        for extra in (bias, before[1]):
            if extra is not None:
                want = want + extra.cpu().double()
                tol = tol + want.abs() * E.F32_STEP
        half = 0.0 if out.dtype == torch.float32 else U.HALF_STEP[torch.bfloat16]
        err = (out.cpu().double() - want).abs()
        tol = tol + (want.abs() + tol) * half
        assert (err <= tol).all(), (name, W, float((err - tol).max()))
        self.seen += 1


def test_products_of_a_step(weights):
    ver = verifier(weights, 2, 3, cls=Checked)
    ver.weights = weights
    ver.prefill(0, prompt(30, 1))
    ver.pool.reserve(0, 34)
    ver.pool.reserve(1, 4)
    ver.set_window([0, 1], [3, 5], [30, 0], torch.tensor([[1, 2, 3], [4, 5, 6]]), torch.rand(2, 3), torch.rand(2))
    ver.step()
    assert ver.seen == 4 * 4 * CFG.layers + 4 * CFG.layers + 1          # four windows of prompt, the step and its head
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("tail,held", [(32, ()), (32, ALL), (64, ("wqkv", "wdown")), (None, ALL)])
def test_a_window_is_its_tokens_one_by_one(weights, tail, held):
    """A text in windows of five rows, some of whose drafts are wrong and are written over by the next window, and
    one token at a time: the same hidden states and the same cache."""
    text = prompt(60, 3)
    single, windows = verifier(weights, 1, 0, tail=tail, held=held), verifier(weights, 2, 4, tail=tail, held=held)
    single.pool.reserve(0, 70)
    windows.pool.reserve(1, 70)
    rows = []
    for p, t in enumerate(text):
        single.set_window([0], [t], [p], torch.zeros(1, 0))
        single.forward()
        rows.append(single.h[0].clone())
    p, g = 0, U.gen(4)
    while p + 5 <= len(text):
        right = int(torch.randint(0, 5, (1,), generator=g))              # drafts that are the text's
        draft = text[p + 1:p + 1 + right] + prompt(4 - right, 100 + p)
        windows.set_window([1], [text[p]], [p], torch.tensor([draft]))
        # the seat's slot is 1; the other seat is empty
        windows.forward()
        for j in range(right + 1):
            assert same_bits(windows.h[j], rows[p + j]), (p, j)
        p += right + 1
    full = p // 16 * 16
    for a, b in zip(single.pool.k + single.pool.v, windows.pool.k + windows.pool.v):
        x = [y[pool.table[s].long()].transpose(1, 2).flatten(0, 1)[:full] for y, pool, s in ((a, single.pool, 0), (b, windows.pool, 1))]
        assert torch.equal(*(y.contiguous().view(torch.uint8) for y in x))
    assert B.biv_device_error() == 0


def test_prefill_by_any_window(weights):
    """A prompt by the whole window, by what a short tail lets through, and by single tokens."""
    text = prompt(75, 6)
    states = []
    for N, K, tail in ((1, 0, 16), (3, 3, 32), (20, 4, 128), (20, 4, 32)):
        ver = verifier(weights, N, K, tail=tail)
        ver.prefill(0, text[:-1])
        ver.pool.reserve(0, 75 + K)
        ver.set_window([0], [text[-1]], [74], torch.zeros(1, K))
        ver.step()
        states.append(ver.probs[0].clone())
    assert all(same_bits(s, states[0]) for s in states[1:])
    assert B.biv_device_error() == 0


def test_requests_do_not_see_their_neighbours(weights):
    K = 2
    prompts = [prompt(n, 10 + n) for n in (33, 64, 3, 100)]
    draft = torch.randint(0, CFG.vocab, (4, K), generator=U.gen(2)).int()
    us, ua = torch.rand(4, generator=U.gen(5)), torch.rand(4, K, generator=U.gen(6))

    def run(order, N, page, tail):
        ver = verifier(weights, N, K, page, 256 // page, tail)
        for seat, r in enumerate(order):
            ver.prefill(seat, prompts[r][:-1])
            ver.pool.reserve(seat, len(prompts[r]) + K)
        ver.set_window(range(len(order)), [prompts[r][-1] for r in order], [len(prompts[r]) - 1 for r in order],
                       draft[order], ua[order], us[order])
        ver.step()
        assert B.biv_device_error() == 0
        probs = ver.probs.view(N, K + 1, -1)
        return {r: (probs[s].clone(), ver.emitted[s].clone()) for s, r in enumerate(order)}

    every = run([0, 1, 2, 3], 4, 32, 48)
    for other in (run([2], 1, 16, 32), run([3, 0], 7, 64, 48), run([1], 50, 128, 32), run([3, 2, 1, 0], 4, 16, 80)):
        for r, (p, t) in other.items():
            assert same_bits(p, every[r][0]) and torch.equal(t, every[r][1]), r


def test_generation_with_and_without_drafts_at_temperature_zero(weights):
    prompts = [prompt(20, 1) * 2, prompt(7, 2), prompt(50, 3)]
    plain = verifier(weights, 3, 0, tail=16, temperature=0.0)
    drafted = verifier(weights, 4, 4, page=64, max_pages=8, tail=32, temperature=0.0)
    a, per_a = paged_generate(plain, prompts, 40)
    b, per_b = paged_generate(drafted, prompts, 40)
    assert a == b and per_a == 1.0 and per_b >= 1.0
    assert B.biv_device_error() == 0


def test_captured_step_equals_the_eager_one(weights):
    N, K = 3, 2
    prompts = [prompt(n, 20 + n) for n in (12, 90, 31)]
    eager, graphed = (verifier(weights, N, K) for _ in range(2))
    for v in (eager, graphed):
        for r, p in enumerate(prompts):
            v.prefill(r, p[:-1])
            v.pool.reserve(r, 128)
        v.set_window([], [], [], torch.zeros(0, K))
    graph = graphed.capture()
    g = U.gen(1)
    for order in ([0, 1, 2], [1], [2, 0]):
        n = len(order)
        args = (order, [prompts[r][-1] for r in order], [len(prompts[r]) - 1 for r in order],
                torch.randint(0, CFG.vocab, (n, K), generator=g), torch.rand(n, K, generator=g), torch.rand(n, generator=g))
        for v in (eager, graphed):
            v.set_window(*args)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(eager.probs[:n * (K + 1)], graphed.probs[:n * (K + 1)])
        assert torch.equal(eager.emitted[:n], graphed.emitted[:n])
        for l in range(CFG.layers):
            for a, b in zip(eager.pool.layer(l), graphed.pool.layer(l)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert B.biv_device_error() == 0
