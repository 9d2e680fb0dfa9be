"""The verify step over a paged key-value cache, with sampled verification.

``PagePool`` owns the pages of every layer and deals them to requests;
``PagedVerifier`` runs the pre-norm Llama decoder of ``verifier.py`` on windows
of N requests x (K + 1) rows whose cache lies in pages, and verifies drafts by
rejection sampling from given uniform numbers (``biv_verify_sample``), for
drafters that do not share the target's Gumbel noise.  Row j of a request takes
its last committed token (j = 0) or draft d_j at position p0 + j; the target's
distribution of row j judges d_{j+1}, that of row K yields the token after a
fully accepted window.

A fixed batch shape serves any number of requests: a seat without a request has
position -1 in all of its rows.  Every kernel computes a row without regard to
the others, so a request's tokens depend neither on its neighbours nor on where
its pages lie.

Projections may carry a bias (``l{l}.bqkv``, ``l{l}.bo``, ``l{l}.bdown`` beside the
weights of ``synth.decoder_weights``); the residual is added in the epilogues of
the two projections that end on it.
"""
from __future__ import annotations

import torch

from . import abi as B


class PagePool:
    """Pages of every layer's K and V, and the tables of ``n_slots`` requests.

    The table lives on the device (``table``, int32 [n_slots, max_pages]); the
    host keeps the free list.  ``reserve`` gives a slot the pages for positions
    [0, length); ``release`` takes a slot's pages back.  Both copy the slot's row
    to the device on the current stream and raise before anything has changed if
    the pool or the table is too small.
    """

    def __init__(self, n_pages: int, page_size: int, layers: int, Hkv: int, hd: int, n_slots: int, max_pages: int,
                 device="cuda"):
        shape = (n_pages, Hkv, page_size, hd)
        self.page_size, self.max_pages = page_size, max_pages
        self.k = [torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(layers)]
        self.v = [torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(layers)]
        self.table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=device)
        self.free = list(range(n_pages - 1, -1, -1))
        self.pages: list[list[int]] = [[] for _ in range(n_slots)]

    def reserve(self, slot: int, length: int) -> None:
        need = -(-length // self.page_size)
        more = need - len(self.pages[slot])
        if need > self.max_pages:
            raise ValueError(f"slot {slot}: {length} positions need {need} pages, the table holds {self.max_pages}")
        if more > len(self.free):
            raise ValueError(f"slot {slot}: {more} pages needed, {len(self.free)} free")
        if more > 0:
            self.pages[slot] += [self.free.pop() for _ in range(more)]
            self._show(slot)

    def release(self, slot: int) -> None:
        self.free += reversed(self.pages[slot])
        self.pages[slot] = []
        self._show(slot)

    def _show(self, slot: int) -> None:
        row = self.pages[slot] + [-1] * (self.max_pages - len(self.pages[slot]))
        self.table[slot].copy_(torch.tensor(row, dtype=torch.int32))


class PagedVerifier:
    """Decoder verifier for windows of exactly N x (K + 1) rows over a page pool.

    The window's inputs are the object's own device buffers (``tokens``,
    ``row_slot``, ``row_pos``: int32 [W]; ``draft``: int32 [N, K]; ``p0``: int32 [N];
    ``u_accept``: fp32 [N, K]; ``u_sample``: fp32 [N]), filled by ``set_window`` or by
    the caller, so that ``capture`` can put the step into a CUDA graph.  Results:
    ``emitted`` int32 [N, K + 1] (-1 behind a request's last token),
    ``accept_len`` and ``new_len`` int32 [N], ``probs`` fp32 [W, vocab].
    """

    def __init__(self, cfg, weights: dict, pool: PagePool, N: int, K: int, temperature: float | None = None,
                 device="cuda"):
        self.cfg, self.pool, self.N, self.K = cfg, pool, N, K
        self.rows = K + 1
        self.W = W = N * (K + 1)
        self.temperature = cfg.temperature if temperature is None else temperature
        dev = torch.device(device)
        self.w = {k: v.to(dev).contiguous() for k, v in weights.items()}
        for l in range(cfg.layers):
            wgu = self.w[f"l{l}.wgu"]
            self.w[f"l{l}.wgu_packed"] = torch.empty_like(wgu)
            B.biv_swiglu_pack_weights(wgu, self.w[f"l{l}.wgu_packed"])
        bf = dict(device=dev, dtype=torch.bfloat16)
        i32 = dict(device=dev, dtype=torch.int32)
        f32 = dict(device=dev, dtype=torch.float32)
        self.x = torch.empty(W, cfg.d, **bf)
        self.h = torch.empty(W, cfg.d, **bf)
        self.qkv = torch.empty(W, cfg.qkv_n, **bf)
        self.q = torch.empty(W, cfg.Hq, cfg.hd, **bf)
        self.o = torch.empty(W, cfg.Hq, cfg.hd, **bf)
        self.act = torch.empty(W, cfg.ffn, **bf)
        self.logits = torch.empty(W, cfg.vocab, **f32)
        self.probs = torch.empty(W, cfg.vocab, **f32)
        self.tokens = torch.zeros(W, **i32)
        self.row_slot = torch.zeros(W, **i32)
        self.row_pos = torch.full((W,), -1, **i32)
        self.draft = torch.zeros(N, K, **i32)
        self.p0 = torch.zeros(N, **i32)
        self.u_accept = torch.zeros(N, K, **f32)
        self.u_sample = torch.zeros(N, **f32)
        self.emitted = torch.empty(N, K + 1, **i32)
        self.accept_len = torch.empty(N, **i32)
        self.new_len = torch.empty(N, **i32)
        ws = B.biv_decode_attn_paged_workspace_size(W, cfg.Hq, cfg.hd, pool.max_pages, pool.page_size)
        self.workspace = torch.empty(ws, device=dev, dtype=torch.uint8)

    # -------------------------------------------------------------- inputs
    def set_window(self, slots, last, p0, draft, u_accept=None, u_sample=None) -> None:
        """Requests r < n at slots[r]: last committed token, its position p0[r]
        and the drafts after it ([n, K]); seats n..N-1 stay empty.  Host lists or
        tensors; pages for p0 + K + 1 positions must have been reserved."""
        n, K, rows = len(slots), self.K, self.rows
        t = lambda v, d=torch.int32: torch.as_tensor(v, dtype=d, device="cpu")  # noqa: E731
        draft, p0 = t(draft).reshape(n, K), t(p0)
        tokens = torch.zeros(self.N, rows, dtype=torch.int32)
        pos = torch.full((self.N, rows), -1, dtype=torch.int32)
        slot = torch.zeros(self.N, rows, dtype=torch.int32)
        tokens[:n] = torch.cat([t(last)[:, None], draft], 1)
        pos[:n] = p0[:, None] + torch.arange(rows, dtype=torch.int32)
        slot[:n] = t(slots)[:, None]
        self.tokens.copy_(tokens.view(-1))
        self.row_slot.copy_(slot.view(-1))
        self.row_pos.copy_(pos.view(-1))
        self.draft[:n].copy_(draft)
        self.p0[:n].copy_(p0)
        if u_accept is not None:
            self.u_accept[:n].copy_(torch.as_tensor(u_accept).reshape(n, K))
        if u_sample is not None:
            self.u_sample[:n].copy_(torch.as_tensor(u_sample))

    # -------------------------------------------------------------- stages
    def forward(self) -> None:
        """Final normalised hidden state of every window row (``h``); the rows' K and V are in their pages."""
        c, w, p = self.cfg, self.w, self.pool
        W = self.W
        B.biv_embed_rmsnorm(w["embed"], self.tokens, w["l0.attn_norm"], self.x, self.h, c.eps)
        for l in range(c.layers):
            B.biv_gemm_bias_act(self.h, w[f"l{l}.wqkv"], self.qkv, bias=w.get(f"l{l}.bqkv"))
            B.biv_rope_kv_write_paged(self.qkv, self.q, p.k[l], p.v[l], p.table, self.row_slot, self.row_pos,
                                      c.rope_theta, self.rows)
            B.biv_decode_attn_paged(self.q, p.k[l], p.v[l], p.table, self.row_slot, self.row_pos, self.o, self.rows,
                                    self.workspace)
            B.biv_gemm_bias_act(self.o.view(W, -1), w[f"l{l}.wo"], self.x, bias=w.get(f"l{l}.bo"), residual=self.x)
            B.biv_rmsnorm(self.x, w[f"l{l}.ffn_norm"], self.h, c.eps)
            B.biv_gemm_swiglu(self.h, w[f"l{l}.wgu_packed"], self.act)
            B.biv_gemm_bias_act(self.act, w[f"l{l}.wdown"], self.x, bias=w.get(f"l{l}.bdown"), residual=self.x)
            gain = w["final_norm"] if l + 1 == c.layers else w[f"l{l + 1}.attn_norm"]
            B.biv_rmsnorm(self.x, gain, self.h, c.eps)

    def verify(self, draft_probs=None) -> None:
        """Probabilities of every row and the verified tokens.  ``draft_probs``: fp32
        [N * K, vocab], or None for a drafter that is certain of its tokens."""
        B.biv_gemm_nosplitk(self.h, self.w["lm_head"], self.logits)
        B.biv_softmax(self.logits, self.probs, self.temperature)
        B.biv_verify_sample(self.probs, draft_probs, self.draft, self.u_accept, self.u_sample, self.p0, self.emitted,
                            self.accept_len, self.new_len)

    def step(self, draft_probs=None) -> None:
        self.forward()
        self.verify(draft_probs)

    def capture(self, draft_probs=None):
        """The step as a CUDA graph on the object's buffers (and ``draft_probs``')."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.step(draft_probs)                # sets kernel attributes outside the capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step(draft_probs)
        return g

    def prefill(self, slot: int, prompt) -> None:
        """K and V of a prompt's tokens at positions 0.. of ``slot``: full windows of
        W rows, the last one padded with empty seats."""
        prompt = torch.as_tensor(prompt, dtype=torch.int32, device="cpu")
        self.pool.reserve(slot, prompt.numel())
        self.row_slot.fill_(slot)
        for a in range(0, prompt.numel(), self.W):
            part = prompt[a:a + self.W]
            pos = torch.full((self.W,), -1, dtype=torch.int32)
            tokens = torch.zeros(self.W, dtype=torch.int32)
            pos[:part.numel()] = torch.arange(a, a + part.numel(), dtype=torch.int32)
            tokens[:part.numel()] = part
            self.row_pos.copy_(pos)
            self.tokens.copy_(tokens)
            self.forward()


@torch.no_grad()
def paged_generate(ver: PagedVerifier, prompts: list, n_tokens: int, generator: torch.Generator | None = None,
                   ngram=(3, 1)) -> tuple[list, float]:
    """``n_tokens`` tokens after each prompt (slots 0..), with n-gram drafts
    (``biv_ngram_draft``; none if the verifier's K is 0) verified by sampling.  The
    pool and its table have to hold a prompt, ``n_tokens`` and K more positions of each.
    Returns the tokens and the mean number emitted per request and step that it took
    part in."""
    n, K = len(prompts), ver.K
    if n > ver.N:
        raise ValueError(f"{n} prompts, the verifier has {ver.N} seats")
    if not all(len(p) for p in prompts):
        raise ValueError("a prompt has at least one token")
    text = [[int(t) for t in p] for p in prompts]
    for r, p in enumerate(text):
        ver.prefill(r, p[:-1])                    # the last token is the first window's row 0
    done, emitted, steps = [0] * n, 0, 0
    dev = ver.tokens.device
    while min(done, default=n_tokens) < n_tokens:
        # a request that has its tokens leaves its seat: its text, pages and share of the mean stay as they are
        live = [r for r in range(n) if done[r] < n_tokens]
        m = len(live)
        draft = torch.zeros(m, K, dtype=torch.int32)
        if K > 0:
            longest = max(len(text[r]) for r in live)
            hist = torch.zeros(m, longest, dtype=torch.int32)
            for i, r in enumerate(live):
                hist[i, :len(text[r])] = torch.tensor(text[r], dtype=torch.int32)
            out, src = torch.empty(m, K, dtype=torch.int32, device=dev), torch.empty(m, dtype=torch.int32, device=dev)
            B.biv_ngram_draft(hist.to(dev), torch.tensor([len(text[r]) for r in live], dtype=torch.int32, device=dev),
                              ngram[0], ngram[1], out, src)
            draft = out.cpu()
        p0 = [len(text[r]) - 1 for r in live]
        for r, p in zip(live, p0):
            ver.pool.reserve(r, p + K + 1)
        # numbers for every request, so that one's do not depend on which others have ended
        u_accept, u_sample = torch.rand(n, K, generator=generator), torch.rand(n, generator=generator)
        ver.set_window(live, [text[r][-1] for r in live], p0, draft, u_accept[live], u_sample[live])
        ver.step()
        tokens, count = ver.emitted.cpu(), ver.accept_len.cpu()
        steps += m
        for i, r in enumerate(live):
            c = int(count[i])
            text[r] += tokens[i, :c].tolist()
            done[r] += c
            emitted += c
    return [p[len(prompts[r]):len(prompts[r]) + n_tokens] for r, p in enumerate(text)], emitted / max(1, steps)
