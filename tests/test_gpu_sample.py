"""Softmax with temperature and the sampled verification against 64-bit and
exact rational arithmetic."""
import numpy as np
import pytest
import torch

import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


def softmax(x, T, V=None, out=None):
    p = torch.full_like(x, float("nan")).cuda() if out is None else out
    B.biv_softmax(x.cuda(), p, T, V=V)
    torch.cuda.synchronize()
    return p


def check_softmax(p, x, T):
    ref, tol = U.softmax(x, T)
    err = (p.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


SIZES = [1, 2, 3, 31, 100, 2047, 2048, 2049, 8192, 8195, 16390, 32000, 40003, 128256, 152064, 262147]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("T", [1.0, 0.7, 0.0])
def test_softmax(V, T):
    x = torch.randn(3, V, generator=U.gen(V)) * 4
    check_softmax(softmax(x, T), x, T)
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("V", [5, 2048, 32000, 128256, 300000])
def test_softmax_special_rows(V):
    inf, nan = float("inf"), float("nan")
    x = torch.randn(8, V, generator=U.gen(V))
    x[0] = -inf                                    # nothing left by a mask
    x[1] = nan
    x[2, V // 2:] = -inf
    x[3, ::2] = nan
    x[4, V - 1], x[4, 0] = inf, inf
    x[5] = torch.finfo(torch.float32).min          # the type's lowest value everywhere
    x[6, 1:] = torch.finfo(torch.float32).min
    x[7] = 3e38
    x[7, 2] = -3e38
    for T in (1.0, 0.3, 0.0):
        p = softmax(x, T)
        check_softmax(p, x, T)
        assert same_bits(softmax(x.repeat(12, 1), T), p.repeat(12, 1))
    check_softmax(softmax(x[:1], 1e-45), x[:1], 1e-45)
    y = torch.tensor([[1.0, 3.0, 3.0, 2.0]])
    assert softmax(y, 1e-42).tolist() == [[0.0, 0.5, 0.5, 0.0]]
    assert softmax(y, 0.0).tolist() == [[0.0, 1.0, 0.0, 0.0]]


@pytest.mark.parametrize("V", [3, 1000, 33333, 40004, 128256, 152064])
def test_softmax_layouts_give_the_same_bits(V):
    """Strided rows, rows off 16-byte alignment, in place, one row alone; columns past V stay."""
    R = 4
    x = torch.randn(R, V, generator=U.gen(1)).cuda()
    base = softmax(x, 0.7)
    for r in range(R):
        assert same_bits(softmax(x[r:r + 1], 0.7), base[r:r + 1])
    for pad, off in ((4, 0), (1, 0), (3, 1), (8, 4)):
        wide = torch.full((R, V + pad + off), 50.0, device="cuda")
        wide[:, off:off + V] = x
        out = torch.full((R, V + pad + off), 7.0, device="cuda")
        B.biv_softmax(wide[:, off:], out[:, off:], 0.7, V=V)
        assert same_bits(out[:, off:off + V].contiguous(), base)
        assert bool((out[:, :off] == 7).all()) and bool((out[:, off + V:] == 7).all())
        B.biv_softmax(wide[:, off:], wide[:, off:], 0.7, V=V)
        assert same_bits(wide[:, off:off + V].contiguous(), base)
        assert bool((wide[:, off + V:] == 50).all())
    many = x.repeat(100, 1)                        # row after row by clusters that stay
    out = softmax(many, 0.7)
    assert same_bits(out, base.repeat(100, 1))
    B.biv_softmax(many, many, 0.7)                 # in place
    assert same_bits(many, out)


@pytest.mark.parametrize("V", [33001, 40003, 128254, 152061])
def test_softmax_many_rows_with_a_ragged_end(V):
    """Rows that start on 16 bytes and end off them, as many as persistent clusters would take."""
    R, ld = 60, V + (-V) % 4
    wide = torch.full((R, ld), 50.0, device="cuda")
    wide[:, :V] = torch.randn(3, V, generator=U.gen(V)).cuda().repeat(20, 1)
    out = torch.full((R, ld), 7.0, device="cuda")
    B.biv_softmax(wide, out, 0.7, V=V)
    check_softmax(out[:3, :V], wide[:3, :V].cpu(), 0.7)
    assert same_bits(out[:, :V].contiguous(), out[:3, :V].repeat(20, 1))
    assert bool((out[:, V:] == 7).all()) and B.biv_device_error() == 0


# ------------------------------------------------------------------ verify
def case(N, K, V, seed, point=False, near=0.7, T=1.0):
    g = U.gen(seed)
    z = torch.randn(N, K + 1, V, generator=g) * 3
    p = torch.softmax(z / T, -1)
    q = torch.softmax(z[:, :K] + near * torch.randn(N, K, V, generator=g), -1)
    d = torch.multinomial((p[:, :K] if point else q).reshape(N * K, V), 1, generator=g).view(N, K).int()
    return dict(target=p, draft_probs=None if point else q, draft=d, u_accept=torch.rand(N, K, generator=g),
                u_sample=torch.rand(N, generator=g), p0=torch.randint(0, 9999, (N,), generator=g).int())


def run(c):
    N, K = c["draft"].shape
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    tokens = torch.full((N, K + 1), -9, dtype=torch.int32, device="cuda")
    a, n = (torch.full((N,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    B.biv_verify_sample(d["target"], d["draft_probs"], d["draft"], d["u_accept"], d["u_sample"], d["p0"], tokens, a, n)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), a.cpu().numpy(), n.cpu().numpy()


def check(c):
    got, want = run(c), U.verify(**c)
    for g, w in zip(got, want):
        assert np.array_equal(g, w), (g, w)
    return got


@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (1, 1, 2), (2, 3, 7), (4, 5, 129), (3, 2, 2048), (2, 4, 2050), (2, 4, 8193),
                                    (2, 3, 32000), (3, 2, 40001), (1, 4, 128256), (1, 2, 152064), (1, 1, 270001),
                                    (40, 12, 500), (300, 2, 64)])
@pytest.mark.parametrize("point", [False, True])
def test_verify(N, K, V, point):
    check(case(N, K, V, seed=N + V, point=point))
    assert B.biv_device_error() == 0


def test_verify_lengths_cover_everything():
    """Every accepted length from none to all occurs, and the emitted tokens keep to the rule."""
    c = case(200, 4, 50, seed=1, near=0.5)
    tokens, a, n = check(c)
    assert set(a.tolist()) == {1, 2, 3, 4, 5}
    assert np.array_equal(n, c["p0"].numpy() + a)


def test_verify_without_drafts_is_plain_sampling():
    c = case(64, 1, 300, seed=2)
    c = dict(target=c["target"][:, :1].contiguous(), draft_probs=None, draft=torch.zeros(64, 0, dtype=torch.int32),
             u_accept=torch.zeros(64, 0), u_sample=c["u_sample"], p0=c["p0"])
    tokens, a, _ = check(c)
    assert (a == 1).all() and tokens.shape == (64, 1)


def test_verify_borders():
    """Uniform numbers on the borders of the distribution, at 0 and just below 1."""
    p = torch.tensor([0.25, 0.0, 0.25, 0.5, 0.0])
    us = [0.0, 0.25, 0.2499999, 0.5, 0.75, 1 - 2.0 ** -24, 1.0, -1.0, float("nan")]
    N = len(us)
    c = dict(target=p.expand(N, 1, 5).contiguous(), draft_probs=None, draft=torch.zeros(N, 0, dtype=torch.int32),
             u_accept=torch.zeros(N, 0), u_sample=torch.tensor(us), p0=torch.zeros(N, dtype=torch.int32))
    tokens, _, _ = check(c)
    assert tokens[:, 0].tolist() == [0, 2, 0, 3, 3, 3, 3, 0, 0]
    # accept borders: u q < p is strict, and exact where a division would round
    q = torch.tensor([0.5, 0.5])
    for u, want in ((0.5, 0), (0.49999997, 1), (0.0, 1)):
        c = dict(target=torch.tensor([[[0.25, 0.75]] * 2]), draft_probs=q.view(1, 1, 2),
                 draft=torch.zeros(1, 1, dtype=torch.int32), u_accept=torch.tensor([[u]]),
                 u_sample=torch.tensor([0.3]), p0=torch.zeros(1, dtype=torch.int32))
        _, a, _ = check(c)
        assert a[0] == want + 1


def test_verify_draws_from_every_part_of_a_long_row():
    """Many requests share the device, so that a warp goes over its part of a row in several goes."""
    N, V = 160, 36004
    g = U.gen(21)
    p = torch.rand(V, generator=g, dtype=torch.float64) ** 4
    p = (p / p.sum()).float()
    c = dict(target=p.expand(N, 1, V).contiguous(), draft_probs=None, draft=torch.zeros(N, 0, dtype=torch.int32),
             u_accept=torch.zeros(N, 0), u_sample=(torch.arange(N) + torch.rand(N, generator=g)) / N, p0=torch.zeros(N, dtype=torch.int32))
    tokens, _, _ = check(c)
    assert len(set(tokens[:, 0].tolist())) > N * 0.9


def test_verify_special_probabilities():
    nan, inf = float("nan"), float("inf")
    V = 3000
    c = case(7, 2, V, seed=4)
    p, q = c["target"], c["draft_probs"]
    p[0, :, ::2] = nan
    q[1, :, 1::3] = nan
    p[2, 0] = q[2, 0]                              # equal rows: u q < p accepts whenever u < 1
    c["u_accept"][2] = 1.0                         # ... and at u = 1 the residual is empty: sampled from p
    p[3, 0] = 0
    p[3, 0, 17] = 1                                # the greedy target (T = 0)
    c["draft"][3, 0] = 17
    p[4] = p[4].flip(-1)
    q[5, 0] = 0                                    # a drafter that cannot have drawn its token
    p[6, 1, 5] = inf                               # counts as 1, and the row sums to less than 8
    check(c)
    assert B.biv_device_error() == 0


def test_verify_faults_raise_bits():
    c = case(4, 2, 100, seed=5)
    c["draft"][1, 0] = 100
    c["draft"][2, 1] = -1
    check(c)
    assert B.biv_device_error() == 2
    c = case(4, 2, 100, seed=5)
    c["target"][1] = 0
    check(c)
    assert B.biv_device_error() == 8
    c = case(4, 2, 100, seed=5)
    good = run(c)
    c["target"][3] = 1.0                           # a hundred ones are no distribution
    c["draft_probs"][3] = 0.0
    c["u_accept"][3] = 1.0
    tokens, a, _ = run(c)
    assert B.biv_device_error() == 8
    assert np.array_equal(tokens[:3], good[0][:3]) and tokens[3, a[3] - 1] == 0


def test_verify_does_not_depend_on_the_batch():
    c = case(50, 3, 20000, seed=6)
    tokens, a, n = run(c)
    for r in (0, 7, 49):
        one = {k: None if v is None else v[r:r + 1].contiguous() for k, v in c.items()}
        t1, a1, n1 = run(one)
        assert np.array_equal(t1[0], tokens[r]) and a1[0] == a[r] and n1[0] == n[r]


def test_verify_follows_the_target_whatever_the_drafter():
    """Chi-square of the first emitted token over 200000 requests (7 degrees of freedom, alpha 1e-4: 29.9)."""
    N, V = 200000, 8
    g = U.gen(11)
    p = torch.softmax(torch.randn(V, generator=g), 0)
    for point in (False, True):
        q = torch.softmax(torch.randn(V, generator=g) * 1.5, 0)
        d = torch.multinomial(q, N, replacement=True, generator=g).int().view(N, 1)
        c = dict(target=p.expand(N, 2, V).contiguous(), draft_probs=None if point else q.expand(N, 1, V).contiguous(),
                 draft=d, u_accept=torch.rand(N, 1, generator=g), u_sample=torch.rand(N, generator=g),
                 p0=torch.zeros(N, dtype=torch.int32))
        tokens, _, _ = run(c)
        seen = np.bincount(tokens[:, 0], minlength=V)
        want = p.double().numpy() * N
        assert ((seen - want) ** 2 / want).sum() < 29.9


# ------------------------------------------------------- the run together
def test_softmax_then_verify_in_a_graph():
    """Logits of target and drafter to tokens, captured and replayed on new logits."""
    N, K, V = 6, 3, 32000
    z, y = torch.empty(N * (K + 1), V, device="cuda"), torch.empty(N * K, V, device="cuda")
    p, q = torch.empty_like(z), torch.empty_like(y)
    draft = torch.zeros(N, K, dtype=torch.int32, device="cuda")
    ua, us = torch.rand(N, K).cuda(), torch.rand(N).cuda()
    p0 = torch.arange(N, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(N, K + 1, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda"),
            torch.zeros(N, dtype=torch.int32, device="cuda")]

    def step():
        B.biv_softmax(z, p, 0.8)
        B.biv_softmax(y, q, 0.8)
        B.biv_verify_sample(p, q, draft, ua, us, p0, *outs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    B.biv_device_error()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        g = U.gen(i)
        zc = torch.randn(N, K + 1, V, generator=g) * 3
        z.copy_(zc.view(-1, V))
        y.copy_((zc[:, :K] + 0.5 * torch.randn(N, K, V, generator=g)).reshape(-1, V))
        draft.copy_(y.argmax(1).view(N, K).int())
        graph.replay()
        torch.cuda.synchronize()
        want = U.verify(p.cpu(), q.cpu(), draft.cpu(), ua.cpu(), us.cpu(), p0.cpu())
        for got, w in zip(outs, want):
            assert np.array_equal(got.cpu().numpy(), w)
    assert B.biv_device_error() == 0
