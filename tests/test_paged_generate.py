"""What paged_generate asks of its verifier and pool (host only: a verifier that emits a script)."""
import pytest
import torch

import invariant_verify_gb300.paged as P
from invariant_verify_gb300.paged import PagePool, paged_generate


class Scripted:
    """Accepts every draft of the requests named fast and none of the others'."""

    def __init__(self, N, K, pool, fast):
        self.N, self.K, self.pool, self.fast = N, K, pool, set(fast)
        self.tokens = torch.zeros(1)
        self.windows = []

    def prefill(self, slot, prompt):
        self.pool.reserve(slot, len(prompt))

    def set_window(self, slots, last, p0, draft, u_accept=None, u_sample=None):
        slots = list(slots)
        assert len(slots) == len(last) == len(p0) == draft.shape[0] == u_accept.shape[0] == u_sample.shape[0] <= self.N
        assert draft.shape == u_accept.shape == (len(slots), self.K)
        for s, p in zip(slots, p0):                # pages for every row of the window
            assert p + self.K + 1 <= len(self.pool.pages[s]) * self.pool.page_size
        self.windows.append((slots, u_accept.clone(), u_sample.clone()))

    def step(self):
        slots = self.windows[-1][0]
        self.emitted = torch.full((self.N, self.K + 1), -1, dtype=torch.int32)
        self.accept_len = torch.ones(self.N, dtype=torch.int32)
        for seat, s in enumerate(slots):
            c = self.K + 1 if s in self.fast else 1
            self.accept_len[seat] = c
            self.emitted[seat, :c] = 100 * s + torch.arange(c, dtype=torch.int32)


@pytest.fixture
def zero_drafts(monkeypatch):
    monkeypatch.setattr(P.B, "biv_ngram_draft", lambda hist, n, a, b, out, src: out.zero_())


@pytest.mark.parametrize("fast", [(0,), (1,), (0, 2), ()])
def test_a_request_that_has_its_tokens_leaves_the_windows(zero_drafts, fast):
    """A pool and a table that hold each prompt, its n tokens and one window's drafts are enough."""
    K, want, prompts = 3, 20, [[1] * 9, [2] * 5, [3] * 9]
    pages = [-(-(len(p) + want + K) // 8) for p in prompts]
    pool = PagePool(sum(pages), 8, 1, 1, 16, 3, max(pages), device="cpu")
    ver = Scripted(4, K, pool, fast)
    text, mean = paged_generate(ver, prompts, want, torch.Generator().manual_seed(3))
    for s, t in enumerate(text):
        step = range(K + 1) if s in fast else range(1)
        assert t == [100 * s + i for _ in range(want) for i in step][:want]
    steps = [-(-want // (K + 1)) if s in fast else want for s in range(3)]
    assert [sum(s in w[0] for w in ver.windows) for s in range(3)] == steps
    assert mean == pytest.approx(sum(n * (K + 1 if s in fast else 1) for s, n in enumerate(steps)) / sum(steps))


def test_a_request_keeps_its_random_numbers_when_another_ends(zero_drafts):
    """Each step draws K accept numbers and one sample number for every request, live or not."""
    K, n = 2, 3
    ver = Scripted(n, K, PagePool(30, 8, 1, 1, 16, n, 10, device="cpu"), (1,))
    paged_generate(ver, [[1] * 4] * n, 9, torch.Generator().manual_seed(5))
    g = torch.Generator().manual_seed(5)
    for slots, ua, us in ver.windows:
        a, b = torch.rand(n, K, generator=g), torch.rand(n, generator=g)
        assert torch.equal(ua, a[slots]) and torch.equal(us, b[slots])
    assert {len(w[0]) for w in ver.windows} == {2, 3}
