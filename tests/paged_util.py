"""Plain 64-bit forms of the paged and sampled operators, for their tests
(torch on the CPU, Python integers for the sampling; no code of the package)."""
from fractions import Fraction

import numpy as np
import torch

# half a step of a type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


class Pool:
    """Requests of the given lengths (positions 0..n-1 hold keys) in shuffled pages of a pool."""

    def __init__(self, lengths, Hkv, hd, page, seed, spare=3, cap=None, fill=float("nan")):
        g = gen(seed)
        self.lengths, self.page = list(lengths), page
        need = [-(-n // page) for n in self.lengths]
        wide = max([1, *need]) if cap is None else -(-cap // page)
        total = sum(need) + spare
        order = torch.randperm(total, generator=g).tolist()
        self.table = torch.full((len(self.lengths), wide), -1, dtype=torch.int32)
        self.k = torch.full((total, Hkv, page, hd), fill, dtype=torch.bfloat16)
        self.v = self.k.clone()
        self.rows = []                                   # (k, v) [Hkv, n, hd] of each request
        at = 0
        for r, n in enumerate(self.lengths):
            ids = order[at:at + need[r]]
            at += need[r]
            self.table[r, :need[r]] = torch.tensor(ids, dtype=torch.int32)
            k, v = bf16(g, Hkv, n, hd), bf16(g, Hkv, n, hd)
            self.rows.append((k, v))
            for i, p in enumerate(ids):
                m = min(page, n - i * page)
                self.k[p, :, :m] = k[:, i * page:i * page + m]
                self.v[p, :, :m] = v[:, i * page:i * page + m]


def attention(q, rows, slot, pos):
    """(o, tolerance) in 64 bits.  The tolerance: half a bf16 step of o; fp32
    scores (a sum of hd products, each partial sum within 2^-23) move every
    weight by at most twice that relative error, and the 16 bits kept of each
    weight, the exponential and the sums stay below 2^-14 of sum p |v|."""
    W, Hq, hd = q.shape
    o = torch.zeros(W, Hq, hd, dtype=torch.float64)
    tol = torch.zeros_like(o)
    for w in range(W):
        n = int(pos[w]) + 1
        if n <= 0:
            continue
        k, v = (x[:, :n].double() for x in rows[int(slot[w])])
        G = Hq // k.shape[0]
        for h in range(Hq):
            qh, kh, vh = q[w, h].double(), k[h // G], v[h // G]
            p = torch.softmax(kh @ qh * hd ** -0.5, 0)
            o[w, h] = p @ vh
            ds = (kh.abs() @ qh.abs()).max() * hd ** -0.5 * hd * 2.0 ** -23
            tol[w, h] = HALF_STEP[torch.bfloat16] * o[w, h].abs() + (2 * ds + 2.0 ** -14) * (p @ vh.abs())
    return o, tol


def rope(x, pos, theta):
    """Rotate-half RoPE of x [W, H, hd] in 64 bits."""
    hd = x.shape[-1]
    a = pos.double()[:, None, None] * theta ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64) / hd)
    lo, hi = x[..., :hd // 2].double(), x[..., hd // 2:].double()
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def act(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x / 2 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)))
    if name == "silu":
        return x * torch.sigmoid(x)
    return x


def softmax(x, T):
    """(p, tolerance): a NaN counts as -inf; the fp32 exponent (x - max) log2(e) / T
    carries three roundings, the exponential two units, and the sum at most
    300 roundings of each term."""
    z = torch.where(x.isnan(), -torch.inf, x.double())
    p = torch.zeros_like(z)
    z2 = torch.zeros_like(z)
    for r in range(z.shape[0]):
        m = z[r].max()
        if m == -torch.inf:
            continue
        if T == 0:
            p[r, int((z[r] == m).nonzero()[0])] = 1
        elif m == torch.inf:
            p[r] = (z[r] == m).double() / (z[r] == m).sum()
        else:
            z2[r] = ((z[r] - m) / T * 1.4426950408889634).clamp(min=-1000)
            p[r] = torch.exp2(z2[r])
            p[r] /= p[r].sum()
    tol = p * (z2.abs() * 4 + 310) * 2.0 ** -24 + 2.0 ** -126
    return p, tol


def _units(w):
    w = np.asarray(w, np.float32)
    w = np.where(np.isnan(w), np.float32(0), np.clip(w, np.float32(0), np.float32(1)))
    return [int(Fraction(float(x)) * 2 ** 60) for x in w]


def verify(target, draft_probs, draft, u_accept, u_sample, p0):
    """(tokens, accept_len, new_len) by exact rational arithmetic."""
    N, K = draft.shape
    V = target.shape[-1]
    p = target.reshape(N, K + 1, V).numpy()
    q = None if draft_probs is None else draft_probs.reshape(N, K, V).numpy()
    clamp = lambda x: Fraction(0) if np.isnan(x) else Fraction(float(min(max(x, np.float32(0)), np.float32(1))))  # noqa: E731
    tokens = np.full((N, K + 1), -1, np.int32)
    length = np.zeros(N, np.int32)
    for r in range(N):
        n = 0
        while n < K:
            d = int(draft[r, n])
            if not 0 <= d < V:
                break
            qd = Fraction(1) if q is None else clamp(q[r, n, d])
            u = float(u_accept[r, n])
            if np.isnan(u) or not Fraction(u) * qd < clamp(p[r, n, d]):
                break
            tokens[r, n] = d
            n += 1
        if n == K:
            w = _units(p[r, K])
        elif q is None:
            w = _units(p[r, n])
            if 0 <= int(draft[r, n]) < V:
                w[int(draft[r, n])] = 0
        else:
            w = _units(p[r, n] - q[r, n])
        if sum(w) == 0:
            w = _units(p[r, n])
        u = Fraction(float(np.clip(np.nan_to_num(np.float32(u_sample[r]), nan=0.0), 0, np.float32(1 - 2.0 ** -24))))
        border, s, token = u * sum(w), 0, 0
        for v, x in enumerate(w):
            s += x
            if s > border:
                token = v
                break
        tokens[r, n] = token
        length[r] = n + 1
    return tokens, length, p0.numpy() + length
