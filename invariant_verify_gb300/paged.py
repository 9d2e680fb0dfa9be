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

Either half of a step's bytes may be held in 8 bits: the cache (a pool with a ``tail``) and
any of the weights (the verifier's ``held``).  The rows' independence of their window,
neighbours, drafts and pages stays.
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

    With ``tail`` (a multiple of 16, or None) the pages are e4m3 with a bf16 scale for 16
    positions and a head (``k_scales``, ``v_scales``), and the last ``tail`` positions
    of a slot lie in bf16 rings (``k_tail``, ``v_tail``).
    """

    def __init__(self, n_pages: int, page_size: int, layers: int, Hkv: int, hd: int, n_slots: int, max_pages: int,
                 device="cuda", tail: int | None = None):
        shape = (n_pages, Hkv, page_size, hd)
        self.page_size, self.max_pages, self.tail = page_size, max_pages, tail
        if tail is not None and (tail < 16 or tail % 16 or page_size % 16):
            raise ValueError(f"a cache in e4m3 needs a tail and pages of multiples of 16 positions, not {tail} and {page_size}")

        def pools(shape, dtype=torch.bfloat16):
            size = torch.empty(0, dtype=dtype).element_size()
            return [torch.zeros((*shape[:-1], shape[-1] * size), dtype=torch.uint8, device=device).view(dtype) for _ in range(layers)]

        dtype = torch.bfloat16 if tail is None else torch.float8_e4m3fn
        self.k, self.v = pools(shape, dtype), pools(shape, dtype)
        if tail is not None:
            self.k_scales, self.v_scales = (pools((n_pages, Hkv, page_size // 16)) for _ in range(2))
            self.k_tail, self.v_tail = (pools((n_slots, Hkv, tail, hd)) for _ in range(2))
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

    def layer(self, l: int) -> tuple:
        """Layer l's cache in the order in which the writes and attention calls take it."""
        if self.tail is None:
            return self.k[l], self.v[l]
        return self.k[l], self.v[l], self.k_scales[l], self.v_scales[l], self.k_tail[l], self.v_tail[l]

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

    ``held`` names the weights that are kept in e4m3 with a scale for 128 x 128 values
    (of ``HELD``; "lm_head" among them): their products take the rows in e4m3 as well.  A
    pool with a tail needs tail >= K + 16, and is prefilled by up to tail - 15 tokens at a time:
    for whole windows of prompt it needs N (K + 1) + 16 (2047 tokens through two 8B-shaped layers by windows of
    320 rows: 4.0 ms; by the 17 rows that tail = 32 leaves: 56 ms).
    """

    HELD = ("wqkv", "wo", "wgu", "wdown", "lm_head")

    def __init__(self, cfg, weights: dict, pool: PagePool, N: int, K: int, temperature: float | None = None,
                 device="cuda", held: tuple = ()):
        if not set(held) <= set(self.HELD):
            raise ValueError(f"held: {sorted(set(held) - set(self.HELD))} not among {self.HELD}")
        if pool.tail is not None and pool.tail < K + 16:
            raise ValueError(f"a window of {K + 1} rows needs a tail of {K + 16} positions, the pool has {pool.tail}")
        self.cfg, self.pool, self.N, self.K = cfg, pool, N, K
        self.rows = K + 1
        self.W = W = N * (K + 1)
        self.temperature = cfg.temperature if temperature is None else temperature
        dev = torch.device(device)
        self.w, self.w8, self.rows8 = {}, {}, {}
        for k, v in weights.items():
            v = v.to(dev).contiguous()
            if k.split(".")[-1] in held:
                self.w8[k] = self._matrix8(*v.shape, 128, dev)
                B.biv_quant_e4m3(v, *self.w8[k], 128)
                if v.shape[1] not in self.rows8:
                    self.rows8[v.shape[1]] = self._matrix8(W, v.shape[1], 1, dev)
            else:
                self.w[k] = v
        for l in range(cfg.layers if "wgu" not in held else 0):
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
        self.gu = torch.empty(W, 2 * cfg.ffn, **bf) if "wgu" in held else None
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

    @staticmethod
    def _matrix8(rows, K, block, dev):
        """An e4m3 matrix and its scales."""
        groups, blocks = -(-K // 128), rows if block == 1 else -(-rows // 128)
        return (torch.empty(rows, K, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn),
                torch.empty((groups, rows) if block == 1 else (blocks, groups), device=dev))

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
    def project(self, x, name: str, out, bias=None, residual=None) -> None:
        """out = x w^T (+ bias) (+ residual) with the weight ``name``, in the type in which it is held."""
        if name in self.w8:
            x8 = self.rows8[x.shape[1]]
            B.biv_quant_e4m3(x, *x8, 1)
            B.biv_gemm_e4m3(*x8, *self.w8[name], out, bias=bias, residual=residual)
        else:
            B.biv_gemm_bias_act(x, self.w[name], out, bias=bias, residual=residual)

    def attend(self, l: int, group: int) -> None:
        """Layer l's K and V of the window into the cache, and its attention.  A cache in e4m3 takes
        a slot's rows in one group: ``group`` rows from each multiple of it on; rows behind the last whole group are not written."""
        c, p = self.cfg, self.pool
        at = (p.table, self.row_slot, self.row_pos)
        if p.tail is None:
            B.biv_rope_kv_write_paged(self.qkv, self.q, *p.layer(l), *at, c.rope_theta, self.rows)
            B.biv_decode_attn_paged(self.q, *p.layer(l), *at, self.o, self.rows, self.workspace)
        else:
            n = self.W // group * group
            B.biv_rope_kv_write_paged_e4m3(self.qkv[:n], self.q[:n], *p.layer(l), p.table, self.row_slot[:n], self.row_pos[:n],
                                           c.rope_theta, group)
            B.biv_decode_attn_paged_e4m3(self.q, *p.layer(l), *at, self.o, self.rows, self.workspace)

    def forward(self, group: int | None = None) -> None:
        """Final normalised hidden state of every window row (``h``); the rows' K and V are in their pages.
        ``group``: the rows of a window that are one request's, in their order (K + 1 unless given); whole groups make up the window."""
        if group is not None and (group < 1 or self.W % group):
            raise ValueError(f"a window of {self.W} rows is not made up of groups of {group}")
        self._forward(group or self.rows)

    def _forward(self, group: int) -> None:
        """``forward``, whose rows behind the last whole group have no position."""
        c, w = self.cfg, self.w
        W = self.W
        B.biv_embed_rmsnorm(w["embed"], self.tokens, w["l0.attn_norm"], self.x, self.h, c.eps)
        for l in range(c.layers):
            self.project(self.h, f"l{l}.wqkv", self.qkv, bias=w.get(f"l{l}.bqkv"))
            self.attend(l, group)
            self.project(self.o.view(W, -1), f"l{l}.wo", self.x, bias=w.get(f"l{l}.bo"), residual=self.x)
            B.biv_rmsnorm(self.x, w[f"l{l}.ffn_norm"], self.h, c.eps)
            if self.gu is None:
                B.biv_gemm_swiglu(self.h, w[f"l{l}.wgu_packed"], self.act)
            else:
                self.project(self.h, f"l{l}.wgu", self.gu)
                B.biv_silu_mul(self.gu, self.act)
            self.project(self.act, f"l{l}.wdown", self.x, bias=w.get(f"l{l}.bdown"), residual=self.x)
            gain = w["final_norm"] if l + 1 == c.layers else w[f"l{l + 1}.attn_norm"]
            B.biv_rmsnorm(self.x, gain, self.h, c.eps)

    def verify(self, draft_probs=None) -> None:
        """Probabilities of every row and the verified tokens.  ``draft_probs``: fp32
        [N * K, vocab], or None for a drafter that is certain of its tokens."""
        if "lm_head" in self.w8:
            self.project(self.h, "lm_head", self.logits)
        else:
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
        W rows (of tail - 15, if the pool's tail holds no more), the last one padded
        with empty seats."""
        prompt = torch.as_tensor(prompt, dtype=torch.int32, device="cpu")
        self.pool.reserve(slot, prompt.numel())
        self.row_slot.fill_(slot)
        window = self.W if self.pool.tail is None else min(self.W, self.pool.tail - 15)
        for a in range(0, prompt.numel(), window):
            part = prompt[a:a + window]
            pos = torch.full((self.W,), -1, dtype=torch.int32)
            tokens = torch.zeros(self.W, dtype=torch.int32)
            pos[:part.numel()] = torch.arange(a, a + part.numel(), dtype=torch.int32)
            tokens[:part.numel()] = part
            self.row_pos.copy_(pos)
            self.tokens.copy_(tokens)
            self._forward(window)


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
