"""What a paged, stochastically verified decoding step asks of libbiv, as measured cases.

Five operators that a server uses one after the other in a step: the rotation of
the new rows and their write into a paged key-value cache, the attention of the
rows over their pages, a projection with bias, activation and residual in its
epilogue, the softmax of the head's logits, and the verification of drafted tokens
against the target's probabilities from given uniform numbers.

With ``own`` false, run() computes each of them in plain torch; with ``own`` true
it calls the library.  exact() gives the same outputs in 64 bits.
"""
import math
import random
import statistics

import torch

own = False


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short conversation, the small decoder: nothing but latency
        {"name": "attn 1 request ctx 700", "op": "attn", "N": 1, "K": 1, "Hq": 8, "Hkv": 2, "hd": 128, "page": 16,
         "median": 700, "sigma": 0.0, "lo": 1, "hi": 2303, "cap": 2304, "pad": 0},
        # a batch in service: 64 requests of very different length, one new token each, two seats of the batch free
        {"name": "attn 64 requests", "op": "attn", "N": 64, "K": 1, "Hq": 32, "Hkv": 8, "hd": 128, "page": 64,
         "median": 1024, "sigma": 1.0, "lo": 256, "hi": 8192, "cap": 8448, "pad": 2},
        # one request with a very long context
        {"name": "attn 1 request ctx 131071", "op": "attn", "N": 1, "K": 1, "Hq": 32, "Hkv": 8, "hd": 128,
         "page": 256, "median": 131071, "sigma": 0.0, "lo": 1, "hi": 131071, "cap": 131072, "pad": 0},
        # a verify window: four drafts and the last token of each of 32 requests
        {"name": "attn 32 windows of 5", "op": "attn", "N": 32, "K": 5, "Hq": 32, "Hkv": 8, "hd": 128, "page": 32,
         "median": 1024, "sigma": 1.0, "lo": 256, "hi": 8192, "cap": 8448, "pad": 0},
        # the rows of one decoding step of the small decoder
        {"name": "rope write 8 rows", "op": "write", "N": 8, "K": 1, "Hq": 8, "Hkv": 2, "hd": 128, "page": 16,
         "median": 700, "sigma": 1.0, "lo": 1, "hi": 2048, "cap": 2304, "theta": 10000.0},
        # a prompt of 4095 tokens
        {"name": "rope write prompt of 4095", "op": "write", "N": 1, "K": 4095, "Hq": 32, "Hkv": 8, "hd": 128,
         "page": 64, "median": 1, "sigma": 0.0, "lo": 1, "hi": 1, "cap": 8192, "theta": 500000.0},
        # the down projection of a small batch: the weights stream once
        {"name": "gemm down 64 rows", "op": "gemm", "M": 64, "N": 4096, "K": 14336, "act": "none", "bias": False,
         "residual": True, "out": "bf16"},
        # an MLP's first projection over a prompt: bound by the matrix product
        {"name": "gemm up gelu 1023 rows", "op": "gemm", "M": 1023, "N": 14336, "K": 4096, "act": "gelu",
         "bias": True, "residual": False, "out": "bf16"},
        # the small decoder's vocabulary, one window
        {"name": "softmax 5 x 32000", "op": "softmax", "R": 5, "V": 32000, "T": 1.0},
        # 64 windows of five rows at the large vocabulary
        {"name": "softmax 320 x 128256", "op": "softmax", "R": 320, "V": 128256, "T": 0.7},
        # one request's window
        {"name": "verify 1 x 4 of 32000", "op": "verify", "N": 1, "K": 4, "V": 32000, "near": 0.7, "point": False},
        # the batch's windows at the large vocabulary
        {"name": "verify 64 x 4 of 128256", "op": "verify", "N": 64, "K": 4, "V": 128256, "near": 0.7,
         "point": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "write", "gemm", "softmax", "verify"))
    if op in ("attn", "write"):
        Hq, Hkv = rng.choice(((8, 2), (32, 8), (8, 1), (12, 4), (16, 16), (40, 8), (32, 2)))
        hd, page = rng.choice((128, 128, 64)), rng.choice((16, 32, 64, 128, 256))
    if op == "attn":
        N, K = _log(rng, 1, 96), rng.choice((1, 1, 1, _log(rng, 2, 16)))
        # the keys and values of all requests together stay below the long request's
        most = min(131071, (1 << 27) // (N * Hkv * hd))
        median = _log(rng, 16, max(17, most // 4))
        sigma = rng.choice((0.0, 0.5, 1.0))
        hi = min(most, 8 * median)
        return {"op": op, "N": N, "K": K, "Hq": Hq, "Hkv": Hkv, "hd": hd, "page": page, "median": median,
                "sigma": sigma, "lo": 1, "hi": hi, "cap": page * -(-(hi + K) // page), "pad": rng.choice((0, 0, 1, 3))}
    if op == "write":
        K = rng.choice((1, _log(rng, 2, 16), _log(rng, 64, 4096)))
        N = _log(rng, 1, max(1, min(256, 4096 // K)))
        cap = page * -(-(K + 4096) // page)
        return {"op": op, "N": N, "K": K, "Hq": Hq, "Hkv": Hkv, "hd": hd, "page": page, "median": _log(rng, 1, 2048),
                "sigma": 0.5, "lo": 1, "hi": 4096, "cap": cap, "theta": rng.choice((10000.0, 500000.0))}
    if op == "gemm":
        N, K = rng.choice(((1024, 1024), (1024, 2816), (5632, 1024), (4096, 4096), (4096, 14336), (14336, 4096),
                           (6144, 4096), (8 * _log(rng, 1, 1024), 8 * _log(rng, 1, 1024))))
        return {"op": op, "M": _log(rng, 1, 1023), "N": N, "K": K,
                "act": rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), "bias": rng.random() < 0.6,
                "residual": rng.random() < 0.6, "out": rng.choice(("bf16", "bf16", "f32"))}
    V = rng.choice((2048, 32000, 128256, 152064, _log(rng, 100, 150000)))
    if op == "softmax":
        return {"op": op, "R": _log(rng, 1, min(1024, (320 * 128256) // V)), "V": V, "T": rng.choice((1.0, 0.7, 1.5))}
    K = _log(rng, 1, 12)
    return {"op": op, "N": _log(rng, 1, max(1, min(128, (320 * 128256) // (V * (K + 1))))), "K": K, "V": V,
            "near": rng.choice((0.3, 0.7, 1.5)), "point": rng.random() < 0.25}


def _contexts(c):
    """The requests' lengths: evenly spaced quantiles of a lognormal law, so that their sum goes by the case alone."""
    n = c["N"]
    z = [statistics.NormalDist().inv_cdf((i + 0.5) / n) for i in range(n)]
    return [max(c["lo"], min(c["hi"], int(round(c["median"] * math.exp(c["sigma"] * v))))) for v in z]


def work(c):
    if c["op"] == "attn":
        pairs = sum(min(x + c["K"] - 1, c["cap"] - 1) + 1 for x in _contexts(c)[:c["N"] - _pads(c)])
        kv = pairs * c["Hkv"] * c["hd"] * 2 * 2
        qo = 2 * c["N"] * c["K"] * c["Hq"] * c["hd"] * 2
        return {"bytes": kv + qo, "flops": 4 * pairs * c["K"] * c["Hq"] * c["hd"]}
    if c["op"] == "write":
        return {"bytes": 2 * c["N"] * c["K"] * (c["Hq"] + 2 * c["Hkv"]) * c["hd"] * 2, "flops": 0}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        size = 2 if c["out"] == "bf16" else 4
        return {"bytes": 2 * (M * K + N * K) + M * N * (size + (2 if c["residual"] else 0)) + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "softmax":
        return {"bytes": 8 * c["R"] * c["V"], "flops": 0}
    # one row of the target for each request, and the draft's where a token was rejected (nearly always, in four)
    return {"bytes": c["N"] * c["V"] * 4 * (1 if c["point"] else 2), "flops": 0}


def _pads(c):
    return min(c.get("pad", 0), c["N"] - 1)


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _pages(c, g, rng):
    """A pool of pages in random order, the table that names them, and the rows' slots and positions."""
    N, K, page = c["N"], c["K"], c["page"]
    ctx = _contexts(c)
    free = _pads(c)
    keep = ctx[:N - free]
    rng.shuffle(keep)
    last = [min(x + K - 1, c["cap"] - 1) for x in keep]
    wide = c["cap"] // page
    need = sum(x // page + 1 for x in last)
    order = list(range(need + 3))
    rng.shuffle(order)
    table, at = [], 0
    for x in last:
        n = x // page + 1
        table.append(order[at:at + n] + [-1] * (wide - n))
        at += n
    table += [[-1] * wide] * free
    first = [x - (K - 1) for x in last]
    pos = [[f + j for j in range(K)] for f in first] + [[-1] * K] * free
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    slot = [[r] * K for r in range(N)]
    pool = (len(order), c["Hkv"], page, c["hd"])
    return {"k_pages": _normal(g, pool), "v_pages": _normal(g, pool), "page_table": i32(table),
            "row_slot": i32(slot).reshape(-1), "row_pos": i32(pos).reshape(-1)}


def prepare(case, seed):
    c, g, rng = case, _generator(seed), random.Random(seed)
    if c["op"] == "attn":
        s = _pages(c, g, rng)
        # keys of norm sqrt(hd) and queries a little longer: scores of the size that trained heads have
        s["q"] = _normal(g, (c["N"] * c["K"], c["Hq"], c["hd"]), 1.5)
        s["o"] = torch.empty_like(s["q"])
    elif c["op"] == "write":
        s = _pages(c, g, rng)
        W = c["N"] * c["K"]
        s["qkv"] = _normal(g, (W, (c["Hq"] + 2 * c["Hkv"]) * c["hd"]))
        s["q_out"] = torch.empty(W, c["Hq"], c["hd"], dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s = {"A": _normal(g, (M, K)), "B": _normal(g, (N, K), K ** -0.5), "bias": None, "residual": None}
        if c["bias"]:
            s["bias"] = _normal(g, (N,), 0.5)
        if c["residual"]:
            s["residual"] = _normal(g, (M, N))
        s["C"] = torch.empty(M, N, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device="cuda")
    elif c["op"] == "softmax":
        s = {"logits": _logits(g, c["R"], c["V"])}
        s["probs"] = torch.empty_like(s["logits"])
    else:
        N, K, V = c["N"], c["K"], c["V"]
        z = _logits(g, N * (K + 1), V)
        s = {"target": torch.softmax(z, 1)}
        if c["point"]:
            s["draft_probs"] = None
            q = s["target"].view(N, K + 1, V)[:, :K].reshape(N * K, V)
        else:
            y = z.view(N, K + 1, V)[:, :K].reshape(N * K, V)
            q = s["draft_probs"] = torch.softmax(y + _normal(g, (N * K, V), c["near"], torch.float32), 1)
        s["draft"] = torch.multinomial(q, 1, generator=g).to(torch.int32).view(N, K)
        s["u_accept"] = torch.rand(N, K, generator=g, device="cuda")
        s["u_sample"] = torch.rand(N, generator=g, device="cuda")
        s["p0"] = torch.randint(1, 4096, (N,), generator=g, device="cuda", dtype=torch.int32)
        s["tokens"] = torch.empty(N, K + 1, dtype=torch.int32, device="cuda")
        s["accept_len"] = torch.empty(N, dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty(N, dtype=torch.int32, device="cuda")
    s["case"] = c
    return s


def _logits(g, R, V):
    """Rows as a language model's head gives them: a wide floor and a few likely tokens far above it."""
    z = torch.randn(R, V, generator=g, device="cuda", dtype=torch.float32) * 2.0
    top = torch.randint(0, V, (R, min(8, V)), generator=g, device="cuda")
    return z.scatter_add_(1, top, 6.0 + 6.0 * torch.rand(top.shape, generator=g, device="cuda"))


# ------------------------------------------------------------- plain forms
def _gathered(pages, table, dtype):
    """[N, Hkv, cap, hd] of a pool and the requests' tables; unnamed pages give page 0, which the mask leaves out."""
    x = pages[table.clamp(min=0).long()]
    n, p, h, s, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, p * s, d).to(dtype)


def _plain_attn(s):
    c = s["case"]
    N, K, Hkv, hd = c["N"], c["K"], c["Hkv"], c["hd"]
    G = c["Hq"] // Hkv
    k, v = _gathered(s["k_pages"], s["page_table"], torch.float32), _gathered(s["v_pages"], s["page_table"], torch.float32)
    q = s["q"].float().view(N, K, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(N, Hkv, K * G, hd)
    pos = s["row_pos"].view(N, 1, K, 1)
    z = torch.matmul(q, k.transpose(2, 3)) * hd ** -0.5
    seen = torch.arange(z.shape[-1], device="cuda") <= pos
    seen = seen[:, :, :, None, :].expand(N, 1, K, G, z.shape[-1]).reshape(N, 1, K * G, z.shape[-1])
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    return o.view(N, Hkv, K, G, hd).permute(0, 2, 1, 3, 4).reshape(N * K, c["Hq"], hd).to(torch.bfloat16)


def _plain_write(s):
    c = s["case"]
    Hq, Hkv, hd, page = c["Hq"], c["Hkv"], c["hd"], c["page"]
    W = c["N"] * c["K"]
    x = s["qkv"].float().view(W, Hq + 2 * Hkv, hd)
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    angle = s["row_pos"].double()[:, None] * torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device="cuda"), -2 * i / hd)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[:, :Hq + Hkv, :hd // 2], x[:, :Hq + Hkv, hd // 2:]
    turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)
    slot, pos = s["row_slot"].long(), s["row_pos"].long()
    at = s["page_table"][slot, pos // page].long()
    s["k_pages"][at, :, pos % page] = turned[:, Hq:]
    s["v_pages"][at, :, pos % page] = x[:, Hq + Hkv:].to(torch.bfloat16)
    return {"q": turned[:, :Hq], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x


def _plain_gemm(s):
    x = torch.matmul(s["A"].float(), s["B"].float().t())
    if s["bias"] is not None:
        x = x + s["bias"].float()
    x = _act(x, s["case"]["act"])
    if s["residual"] is not None:
        x = x + s["residual"].float()
    return x.to(s["C"].dtype)


def _plain_softmax(s):
    x = s["logits"]
    e = torch.exp((x - x.amax(1, keepdim=True)) / s["case"]["T"])
    return e / e.sum(1, keepdim=True)


def _plain_verify(s):
    c = s["case"]
    N, K, V = c["N"], c["K"], c["V"]
    p, d = s["target"].view(N, K + 1, V), s["draft"].long()
    # products of two 24-bit numbers are exact in 64 bits
    pd = p[:, :K].gather(2, d[:, :, None])[:, :, 0].double()
    qd = 1.0 if c["point"] else s["draft_probs"].view(N, K, V).gather(2, d[:, :, None])[:, :, 0].double()
    n = (s["u_accept"].double() * qd < pd).int().cumprod(1).sum(1)
    r = torch.arange(N, device="cuda")
    j = n.clamp(max=K - 1)
    pn = p[r, n]
    if c["point"]:
        w = pn.clone()
        w[r, d[r, j]] = torch.where(n < K, 0.0, w[r, d[r, j]])
    else:
        qn = torch.where((n < K)[:, None], s["draft_probs"].view(N, K, V)[r, j], 0.0)
        w = torch.where(pn > qn, pn - qn, 0.0)
    w = torch.where((w.sum(1) > 0)[:, None], w, pn)
    # sums of many small numbers next to a border: 64 bits
    cs = w.double().cumsum(1)
    token = (cs <= s["u_sample"].double()[:, None] * cs[:, -1:]).sum(1).clamp(max=V - 1)
    at = torch.arange(K + 1, device="cuda")
    tokens = torch.where(at < n[:, None], torch.cat([d, d[:, :1]], 1), -1)
    tokens = torch.where(at == n[:, None], token[:, None], tokens)
    return {"tokens": tokens.int(), "accept_len": (n + 1).int(), "new_len": (s["p0"] + n + 1).int()}


_PLAIN = {"attn": _plain_attn, "write": _plain_write, "gemm": _plain_gemm, "softmax": _plain_softmax,
          "verify": _plain_verify}


# ------------------------------------------------------- the library's calls
def _own_attn(s):
    from invariant_verify_gb300 import abi as B
    if "workspace" not in s:
        # one for each batch shape and stream, as a server keeps it: a call owns its workspace until it is done
        W, Hq, hd = s["q"].shape
        n = B.biv_decode_attn_paged_workspace_size(W, Hq, hd, s["page_table"].shape[1], s["k_pages"].shape[2])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    B.biv_decode_attn_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["row_slot"], s["row_pos"], s["o"],
                            s["case"]["K"], s["workspace"])
    return s["o"]


def _own_write(s):
    from invariant_verify_gb300 import abi as B
    B.biv_rope_kv_write_paged(s["qkv"], s["q_out"], s["k_pages"], s["v_pages"], s["page_table"], s["row_slot"],
                              s["row_pos"], s["case"]["theta"], s["case"]["K"])
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_gemm(s):
    from invariant_verify_gb300 import abi as B
    B.biv_gemm_bias_act(s["A"], s["B"], s["C"], bias=s["bias"], residual=s["residual"], act=s["case"]["act"])
    return s["C"]


def _own_softmax(s):
    from invariant_verify_gb300 import abi as B
    B.biv_softmax(s["logits"], s["probs"], s["case"]["T"])
    return s["probs"]


def _own_verify(s):
    from invariant_verify_gb300 import abi as B
    B.biv_verify_sample(s["target"], s["draft_probs"], s["draft"], s["u_accept"], s["u_sample"], s["p0"], s["tokens"],
                        s["accept_len"], s["new_len"])
    return {"tokens": s["tokens"], "accept_len": s["accept_len"], "new_len": s["new_len"]}


_OWN = {"attn": _own_attn, "write": _own_write, "gemm": _own_gemm, "softmax": _own_softmax, "verify": _own_verify}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "attn":
        N, K, Hq, Hkv, hd, page = (c[k] for k in ("N", "K", "Hq", "Hkv", "hd", "page"))
        out = torch.zeros(N * K, Hq, hd, dtype=torch.float64, device="cuda")
        table, pos = s["page_table"].tolist(), s["row_pos"].tolist()
        for r in range(N):
            for j in range(K):
                n = pos[r * K + j] + 1
                if n <= 0:
                    continue
                at = table[r][:-(-n // page)]
                for h in range(Hkv):
                    k = s["k_pages"][at, h].reshape(-1, hd)[:n].double()
                    v = s["v_pages"][at, h].reshape(-1, hd)[:n].double()
                    lo, hi = h * (Hq // Hkv), (h + 1) * (Hq // Hkv)
                    p = torch.softmax(s["q"][r * K + j, lo:hi].double() @ k.T / math.sqrt(hd), 1)
                    out[r * K + j, lo:hi] = p @ v
        return out
    if c["op"] == "write":
        Hq, Hkv, hd, page = c["Hq"], c["Hkv"], c["hd"], c["page"]
        x = s["qkv"].double().view(-1, Hq + 2 * Hkv, hd)
        half = torch.complex(x[:, :Hq + Hkv, :hd // 2], x[:, :Hq + Hkv, hd // 2:])
        freq = torch.tensor([c["theta"] ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device="cuda")
        angle = torch.outer(s["row_pos"].double(), freq)[:, None]
        half = half * torch.complex(angle.cos(), angle.sin())
        y = torch.cat([half.real, half.imag], -1)
        k, v = s["k_pages"].double(), s["v_pages"].double()
        slot, pos = s["row_slot"].long(), s["row_pos"].long()
        for h in range(Hkv):
            at = (s["page_table"][slot, pos // page].long(), pos % page)
            k[:, h][at] = y[:, Hq + h]
            v[:, h][at] = x[:, Hq + Hkv + h]
        return {"q": y[:, :Hq].contiguous(), "k_pages": k, "v_pages": v}
    if c["op"] == "gemm":
        x = s["A"].double() @ s["B"].double().T
        if c["bias"]:
            x += s["bias"].double()
        if c["act"] == "relu":
            x = x.clamp(min=0)
        elif c["act"] == "gelu":
            x = x * torch.special.ndtr(x)
        elif c["act"] == "gelu_tanh":
            x = x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
        elif c["act"] == "silu":
            x = x * torch.sigmoid(x)
        return x + s["residual"].double() if c["residual"] else x
    if c["op"] == "softmax":
        return torch.softmax(s["logits"].double() / c["T"], 1)
    return None
