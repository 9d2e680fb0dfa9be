"""What a decoding step held in 8 bits asks of libbiv, as measured cases.

Four operators that a server uses together once weights and cache are e4m3: the
quantisation of activations (a scale for 128 values of a row) and of weights (a
scale for 128 x 128), the matrix product of the two, the rotation of new rows with
their write into a paged cache whose blocks of 16 positions have a scale for each
head, and the attention over that cache.

A block of 16 positions goes into the pages when its last position is written; the
rows of the blocks before that stay in bf16 in a ring of ``tail`` positions a slot.
So a row at position p attends to positions below 16 floor(p / 16) in 8 bits and to
the rest, up to its own, in bf16, whatever else is in the batch.

With ``own`` false, run() computes each of them in plain torch; with ``own`` true
it calls the library.  exact() gives the same outputs in 64 bits.
"""
import math
import random
import statistics

import torch

own = False

BLOCK = 16             # positions of a block of the cache
GROUP = 128            # values of a row that share a scale in the matrix product
TOP = 448.0            # the largest e4m3 number
LEAST = 2.0 ** -100    # the smallest scale: a block of zeros has it


# ----------------------------------------------------------------- cases
def listed():
    return [
        # the hidden states of a small batch before a projection: nothing but latency
        {"name": "quant 64 x 4096", "op": "quant", "rows": 64, "K": 4096, "block": 1},
        # a stacked gate and up weight when a model is loaded
        {"name": "quant weights 28672 x 4096", "op": "quant", "rows": 28672, "K": 4096, "block": 128},
        # the query, key and value projection of eight requests, one token each
        {"name": "gemm qkv 8 rows", "op": "gemm", "M": 8, "N": 6144, "K": 4096, "act": "none", "bias": True,
         "residual": False, "out": "bf16"},
        # the down projection of a batch: the weights stream once
        {"name": "gemm down 64 rows", "op": "gemm", "M": 64, "N": 4096, "K": 14336, "act": "none", "bias": False,
         "residual": True, "out": "bf16"},
        # the head's logits for 64 windows of five rows
        {"name": "gemm head 320 rows", "op": "gemm", "M": 320, "N": 128256, "K": 4096, "act": "none", "bias": False,
         "residual": False, "out": "f32"},
        # an MLP's first projection over a prompt: bound by the matrix product
        {"name": "gemm up silu 1023 rows", "op": "gemm", "M": 1023, "N": 14336, "K": 4096, "act": "silu", "bias": False,
         "residual": False, "out": "bf16"},
        # the rows of one decoding step of the small decoder: one of them fills its block
        {"name": "write 8 rows", "op": "write", "N": 8, "K": 1, "Hq": 8, "Hkv": 2, "hd": 128, "page": 16, "tail": 32,
         "median": 703, "sigma": 1.0, "lo": 1, "hi": 2048, "cap": 2304, "theta": 10000.0},
        # a part of a prompt
        {"name": "write prompt of 2047", "op": "write", "N": 1, "K": 2047, "Hq": 32, "Hkv": 8, "hd": 128, "page": 64,
         "tail": 2064, "median": 5, "sigma": 0.0, "lo": 5, "hi": 5, "cap": 8192, "theta": 500000.0},
        # one user, a short conversation, the small decoder: nothing but latency
        {"name": "attn 1 request ctx 700", "op": "attn", "N": 1, "K": 1, "Hq": 8, "Hkv": 2, "hd": 128, "page": 16,
         "tail": 32, "median": 700, "sigma": 0.0, "lo": 1, "hi": 2303, "cap": 2304, "pad": 0},
        # a batch in service: 64 requests of very different length, one new token each, two seats of the batch free
        {"name": "attn 64 requests", "op": "attn", "N": 64, "K": 1, "Hq": 32, "Hkv": 8, "hd": 128, "page": 64,
         "tail": 32, "median": 1024, "sigma": 1.0, "lo": 256, "hi": 8192, "cap": 8448, "pad": 2},
        # one request with a very long context
        {"name": "attn 1 request ctx 131071", "op": "attn", "N": 1, "K": 1, "Hq": 32, "Hkv": 8, "hd": 128,
         "page": 256, "tail": 32, "median": 131071, "sigma": 0.0, "lo": 1, "hi": 131071, "cap": 131072, "pad": 0},
        # a verify window: four drafts and the last token of each of 32 requests
        {"name": "attn 32 windows of 5", "op": "attn", "N": 32, "K": 5, "Hq": 32, "Hkv": 8, "hd": 128, "page": 32,
         "tail": 32, "median": 1024, "sigma": 1.0, "lo": 256, "hi": 8192, "cap": 8448, "pad": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _tail(K):
    return BLOCK * -(-(K + BLOCK - 1) // BLOCK)


def draw(rng):
    op = rng.choice(("attn", "attn", "write", "gemm", "gemm", "quant"))
    if op in ("attn", "write"):
        Hq, Hkv = rng.choice(((8, 2), (32, 8), (8, 1), (12, 4), (16, 16), (40, 8), (32, 2)))
        hd, page = rng.choice((128, 128, 64)), rng.choice((16, 32, 64, 128, 256))
    if op == "attn":
        N, K = _log(rng, 1, 96), rng.choice((1, 1, 1, _log(rng, 2, 16)))
        # the keys and values of all requests together stay below the long request's
        most = min(131071, (1 << 27) // (N * Hkv * hd))
        median = _log(rng, 16, max(17, most // 4))
        hi = min(most, 8 * median)
        return {"op": op, "N": N, "K": K, "Hq": Hq, "Hkv": Hkv, "hd": hd, "page": page,
                "tail": _tail(K) + rng.choice((0, 16, 48)), "median": median, "sigma": rng.choice((0.0, 0.5, 1.0)),
                "lo": 1, "hi": hi, "cap": page * -(-(hi + K) // page), "pad": rng.choice((0, 0, 1, 3))}
    if op == "write":
        K = rng.choice((1, _log(rng, 2, 16), _log(rng, 64, 2047)))
        N = _log(rng, 1, max(1, min(256, 2047 // K)))
        return {"op": op, "N": N, "K": K, "Hq": Hq, "Hkv": Hkv, "hd": hd, "page": page,
                "tail": _tail(K) + rng.choice((0, 16, 48)), "median": _log(rng, 1, 2048), "sigma": 0.5, "lo": 1,
                "hi": 4096, "cap": page * -(-(K + 4096) // page), "theta": rng.choice((10000.0, 500000.0))}
    if op == "gemm":
        N, K = rng.choice(((1024, 1024), (1024, 2816), (5632, 1024), (4096, 4096), (4096, 14336), (14336, 4096),
                           (6144, 4096), (8 * _log(rng, 1, 1024), 16 * _log(rng, 1, 512))))
        return {"op": op, "M": _log(rng, 1, 1023), "N": N, "K": K,
                "act": rng.choice(("none", "none", "relu", "gelu", "gelu_tanh", "silu")), "bias": rng.random() < 0.6,
                "residual": rng.random() < 0.6, "out": rng.choice(("bf16", "bf16", "f32"))}
    return {"op": op, "rows": _log(rng, 1, 4096), "K": 16 * _log(rng, 1, 1024), "block": rng.choice((1, 1, 128))}


def _contexts(c):
    """The requests' lengths: evenly spaced quantiles of a lognormal law, so that their sum goes by the case alone."""
    n = c["N"]
    z = [statistics.NormalDist().inv_cdf((i + 0.5) / n) for i in range(n)]
    return [max(c["lo"], min(c["hi"], int(round(c["median"] * math.exp(c["sigma"] * v))))) for v in z]


def _windows(c):
    """First position of every request's rows; the last ones of the batch have none."""
    last = [min(x + c["K"] - 1, c["cap"] - 1) for x in _contexts(c)[:c["N"] - min(c.get("pad", 0), c["N"] - 1)]]
    return [x - (c["K"] - 1) for x in last]


def work(c):
    if c["op"] == "quant":
        n = -(-c["rows"] // c["block"]) * -(-c["K"] // GROUP)
        return {"bytes": 3 * c["rows"] * c["K"] + 4 * n, "flops": 0}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        size = (2 if c["out"] == "bf16" else 4) + (2 if c["residual"] else 0)
        scales = 4 * -(-K // GROUP) * (M + -(-N // GROUP))
        return {"bytes": M * K + N * K + scales + M * N * size + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    K, head = c["K"], c["Hkv"] * c["hd"]
    if c["op"] == "write":
        rows = c["N"] * K
        blocks = sum((p + K) // BLOCK - p // BLOCK for p in _windows(c))
        before = sum(p % BLOCK for p in _windows(c) if (p + K) // BLOCK > p // BLOCK)    # of the first block that is filled
        # the rows in, q and the ring's rows out; for a filled block its e4m3 values and a scale for each head
        return {"bytes": 2 * 2 * rows * (c["Hq"] * c["hd"] + 2 * head) + 2 * 2 * before * head
                + 2 * blocks * (BLOCK * head + 2 * c["Hkv"]), "flops": 0}
    held = sum(BLOCK * (p // BLOCK) for p in _windows(c))          # positions that the first rows read in 8 bits
    near = sum(p % BLOCK + K for p in _windows(c))                 # and those in bf16
    held += sum(BLOCK * ((p + K - 1) // BLOCK - p // BLOCK) for p in _windows(c))
    pairs = sum(p + j + 1 for p in _windows(c) for j in range(K))
    return {"bytes": 2 * held * (head + c["Hkv"] / 8) + 4 * near * head + 4 * c["N"] * K * c["Hq"] * c["hd"],
            "flops": 4 * pairs * c["Hq"] * c["hd"]}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _scale(top):
    """top / 448, rounded once (by a number on the host the division would be a product with its inverse)."""
    return (top / top.new_full((), TOP)).clamp(min=LEAST)


def _held_blocks(x):
    """(e4m3, scales) of blocks x [..., BLOCK, hd]: the scale is the next bf16 number from max |x| / 448 on."""
    s = _scale(x.float().abs().amax((-2, -1)))
    up = ((s.view(torch.int32) + 0xffff) & -65536).view(torch.float32)
    return (x.float() / up[..., None, None]).to(torch.float8_e4m3fn), up.to(torch.bfloat16)


def _cache(c, g, rng):
    """Pages in random order with what earlier steps have left in them, the table that names them, the ring, and the rows' slots and positions."""
    N, K, Hkv, hd, page = c["N"], c["K"], c["Hkv"], c["hd"], c["page"]
    first = _windows(c)
    rng.shuffle(first)
    wide = c["cap"] // page
    need = [(p + K - 1) // page + 1 for p in first]
    order = list(range(sum(need) + 3))
    rng.shuffle(order)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (wide - n))
        at += n
    table += [[-1] * wide] * (N - len(first))
    pos = [[p + j for j in range(K)] for p in first] + [[-1] * K] * (N - len(first))
    s = {"page_table": _i32(table), "row_slot": _i32([[r] * K for r in range(N)]).view(-1), "row_pos": _i32(pos).view(-1)}
    for x in "kv":
        blocks, scales = _held_blocks(_normal(g, (len(order), Hkv, page // BLOCK, BLOCK, hd)))
        s[x + "_pages"], s[x + "_scales"] = blocks.view(len(order), Hkv, page, hd), scales
        s[x + "_tail"] = _normal(g, (N, Hkv, c["tail"], hd))
    # the blocks that the rows fill, as (slot, block): the program knows its requests' lengths
    s["filled"] = _i32([[r, b] for r, p in enumerate(first) for b in range(p // BLOCK, (p + K) // BLOCK)]).view(-1, 2).long()
    return s


def prepare(case, seed):
    c, g, rng = case, _generator(seed), random.Random(seed)
    if c["op"] == "quant":
        x = _normal(g, (c["rows"], c["K"]), 1.0 if c["block"] == 1 else c["K"] ** -0.5)
        groups = -(-c["K"] // GROUP)
        shape = (groups, c["rows"]) if c["block"] == 1 else (-(-c["rows"] // GROUP), groups)
        s = {"x": x, "q": torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"),
             "scales": torch.empty(shape, device="cuda")}
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s = {"bias": None, "residual": None}
        s["A"], s["a_scales"] = _plain_quant({"x": _normal(g, (M, K)), "case": {"block": 1}}).values()
        s["B"], s["b_scales"] = _plain_quant({"x": _normal(g, (N, K), K ** -0.5), "case": {"block": 128}}).values()
        if c["bias"]:
            s["bias"] = _normal(g, (N,), 0.5)
        if c["residual"]:
            s["residual"] = _normal(g, (M, N))
        s["C"] = torch.empty(M, N, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device="cuda")
    else:
        s = _cache(c, g, rng)
        W = c["N"] * c["K"]
        if c["op"] == "attn":
            # keys of norm sqrt(hd) and queries a little longer: scores of the size that trained heads have
            s["q"] = _normal(g, (W, c["Hq"], c["hd"]), 1.5)
            s["o"] = torch.empty_like(s["q"])
        else:
            s["qkv"] = _normal(g, (W, (c["Hq"] + 2 * c["Hkv"]) * c["hd"]))
            s["q_out"] = torch.empty(W, c["Hq"], c["hd"], dtype=torch.bfloat16, device="cuda")
    s["case"] = c
    return s


# ------------------------------------------------------------- plain forms
def _groups(x, block):
    """x [rows, K] as [row blocks, block, groups, GROUP], zeros where it ends."""
    rows, K = x.shape
    up = torch.nn.functional.pad(x, (0, -K % GROUP, 0, -rows % block))
    return up.view(up.shape[0] // block, block, up.shape[1] // GROUP, GROUP)


def _plain_quant(s):
    x, block = s["x"], s["case"]["block"]
    rows, K = x.shape
    y = _groups(x.float(), block)
    scale = _scale(y.abs().amax((1, 3)))                               # [row blocks, groups]
    q = (y / scale[:, None, :, None]).view(y.shape[0] * block, -1)[:rows, :K].to(torch.float8_e4m3fn)
    return {"q": q, "scales": scale.t().contiguous() if block == 1 else scale}


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
    M, K = s["A"].shape
    N = s["B"].shape[0]
    A = (_groups(s["A"].float(), 1) * s["a_scales"].t()[:, None, :, None]).view(M, -1)
    B = (_groups(s["B"].float(), GROUP) * s["b_scales"][:, None, :, None]).view(-1, A.shape[1])[:N]
    x = torch.matmul(A, B.t())
    if s["bias"] is not None:
        x = x + s["bias"].float()
    x = _act(x, s["case"]["act"])
    if s["residual"] is not None:
        x = x + s["residual"].float()
    return x.to(s["C"].dtype)


def _plain_write(s):
    c = s["case"]
    N, K, Hq, Hkv, hd, page, tail = (c[k] for k in ("N", "K", "Hq", "Hkv", "hd", "page", "tail"))
    x = s["qkv"].float().view(N * K, Hq + 2 * Hkv, hd)
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    # angles of far positions: 64 bits
    angle = s["row_pos"].double()[:, None] * torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device="cuda"), -2 * i / hd)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[:, :Hq + Hkv, :hd // 2], x[:, :Hq + Hkv, hd // 2:]
    turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)
    slot, pos = s["row_slot"].long(), s["row_pos"].long()
    s["k_tail"][slot, :, pos % tail] = turned[:, Hq:]
    s["v_tail"][slot, :, pos % tail] = x[:, Hq + Hkv:].to(torch.bfloat16)
    slot, block = s["filled"][:, 0], s["filled"][:, 1]
    from_ring = (block[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")) % tail
    at = s["page_table"][slot, block * BLOCK // page].long()
    place = block % (page // BLOCK)
    q8, scale = _held_blocks(s["k_tail"][slot[:, None], :, from_ring].transpose(1, 2))
    s["k_pages"].view(torch.uint8).view(-1, Hkv, page // BLOCK, BLOCK, hd)[at, :, place] = q8.view(torch.uint8)
    s["k_scales"][at, :, place] = scale
    q8, scale = _held_blocks(s["v_tail"][slot[:, None], :, from_ring].transpose(1, 2))
    s["v_pages"].view(torch.uint8).view(-1, Hkv, page // BLOCK, BLOCK, hd)[at, :, place] = q8.view(torch.uint8)
    s["v_scales"][at, :, place] = scale
    return {"q": turned[:, :Hq], **{k: s[k] for k in ("k_pages", "v_pages", "k_scales", "v_scales", "k_tail", "v_tail")}}


def _gathered(pages, scales, table):
    """fp32 [N, Hkv, cap, hd] of a pool and the requests' tables; unnamed pages give page 0, which the mask leaves out."""
    at = table.clamp(min=0).long()
    x, s = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float(), scales[at].float()
    n, p, h, t, d = x.shape
    x = x.view(n, p, h, t // BLOCK, BLOCK, d) * s[..., None, None]
    return x.permute(0, 2, 1, 3, 4, 5).reshape(n, h, p * t, d)


def _plain_attn(s):
    c = s["case"]
    N, K, Hkv, hd, tail = c["N"], c["K"], c["Hkv"], c["hd"], c["tail"]
    G = c["Hq"] // Hkv
    k = _gathered(s["k_pages"], s["k_scales"], s["page_table"])
    q = s["q"].float().view(N, K, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(N, Hkv, K * G, hd)
    pos = s["row_pos"].view(N, 1, K, 1, 1).expand(N, 1, K, G, 1).reshape(N, 1, K * G, 1)
    start = pos.clamp(min=0) // BLOCK * BLOCK                          # of the row's own block
    z = torch.matmul(q, k.transpose(2, 3)) * hd ** -0.5
    z = torch.where(torch.arange(z.shape[-1], device="cuda") < torch.where(pos < 0, 0, start), z, -math.inf)
    del k
    # place j of the ring holds position start + (j - start) mod tail, as far as the row's block goes
    ahead = (torch.arange(tail, device="cuda") - start) % tail
    near = torch.matmul(q, s["k_tail"].float().transpose(2, 3)) * hd ** -0.5
    near = torch.where(start + ahead <= pos, near, -math.inf)
    m = torch.maximum(z.amax(-1, keepdim=True), near.amax(-1, keepdim=True))
    m = torch.where(m == -math.inf, 0.0, m)
    z, near = torch.exp(z - m), torch.exp(near - m)
    total = z.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
    o = torch.matmul(z, _gathered(s["v_pages"], s["v_scales"], s["page_table"])) + torch.matmul(near, s["v_tail"].float())
    o = o / torch.where(total == 0, 1.0, total)
    return o.view(N, Hkv, K, G, hd).permute(0, 2, 1, 3, 4).reshape(N * K, c["Hq"], hd).to(torch.bfloat16)


_PLAIN = {"quant": _plain_quant, "gemm": _plain_gemm, "write": _plain_write, "attn": _plain_attn}


# ------------------------------------------------------- the library's calls
def _own_quant(s):
    from invariant_verify_gb300 import abi as B
    B.biv_quant_e4m3(s["x"], s["q"], s["scales"], s["case"]["block"])
    return {"q": s["q"], "scales": s["scales"]}


def _own_gemm(s):
    from invariant_verify_gb300 import abi as B
    B.biv_gemm_e4m3(s["A"], s["a_scales"], s["B"], s["b_scales"], s["C"], bias=s["bias"], residual=s["residual"],
                    act=s["case"]["act"])
    return s["C"]


def _own_write(s):
    from invariant_verify_gb300 import abi as B
    B.biv_rope_kv_write_paged_e4m3(s["qkv"], s["q_out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                   s["k_tail"], s["v_tail"], s["page_table"], s["row_slot"], s["row_pos"],
                                   s["case"]["theta"], s["case"]["K"])
    return {"q": s["q_out"], **{k: s[k] for k in ("k_pages", "v_pages", "k_scales", "v_scales", "k_tail", "v_tail")}}


def _own_attn(s):
    from invariant_verify_gb300 import abi as B
    if "workspace" not in s:
        # one for each batch shape and stream, as a server keeps it: a call owns its workspace until it is done
        W, Hq, hd = s["q"].shape
        n = B.biv_decode_attn_paged_workspace_size(W, Hq, hd, s["page_table"].shape[1], s["k_pages"].shape[2])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    B.biv_decode_attn_paged_e4m3(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["k_tail"], s["v_tail"],
                                 s["page_table"], s["row_slot"], s["row_pos"], s["o"], s["case"]["K"], s["workspace"])
    return s["o"]


_OWN = {"quant": _own_quant, "gemm": _own_gemm, "write": _own_write, "attn": _own_attn}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------- in 64 bits
def _scale64(top):
    """The next number of 8 bits from top / 448 on."""
    m, e = torch.frexp(torch.clamp(top / TOP, min=LEAST))
    return torch.ldexp(torch.ceil(m * 256) / 256, e)


def exact(case, seed):
    """What is held in e4m3 comes back as the quotient by its scale, not rounded."""
    s, c = prepare(case, seed), case
    if c["op"] == "quant":
        x = s["x"].double()
        cols = [x[:, a:a + GROUP] for a in range(0, c["K"], GROUP)]
        if c["block"] == 1:
            scales = torch.stack([torch.linalg.vector_norm(y, math.inf, 1) for y in cols]) / TOP
            each = scales.t().repeat_interleave(GROUP, 1)[:, :c["K"]]
        else:
            scales = torch.stack([torch.stack([y[r:r + 128].abs().max() for r in range(0, c["rows"], 128)]) for y in cols], 1) / TOP
            each = scales.repeat_interleave(128, 0)[:c["rows"]].repeat_interleave(GROUP, 1)[:, :c["K"]]
        return {"q": x / each, "scales": scales}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        x = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for i, a in enumerate(range(0, K, GROUP)):
            part = s["A"][:, a:a + GROUP].double() @ s["B"][:, a:a + GROUP].double().T
            x += part.mul_(s["a_scales"][i].double()[:, None]).mul_(s["b_scales"][:, i].double().repeat_interleave(128)[:N])
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
    N, K, Hq, Hkv, hd, page, tail = (c[k] for k in ("N", "K", "Hq", "Hkv", "hd", "page", "tail"))
    table, pos = s["page_table"].tolist(), s["row_pos"].tolist()
    if c["op"] == "write":
        x = s["qkv"].double().view(-1, Hq + 2 * Hkv, hd)
        half = torch.complex(x[:, :Hq + Hkv, :hd // 2], x[:, :Hq + Hkv, hd // 2:])
        freq = torch.tensor([c["theta"] ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device="cuda")
        half = half * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(s["row_pos"].double(), freq))[:, None]
        y = torch.cat([half.real, half.imag], -1)
        out = {"q": y[:, :Hq].contiguous()}
        for name, rows in (("k", y[:, Hq:]), ("v", x[:, Hq + Hkv:])):
            pages, scales, ring = (s[name + t].double() for t in ("_pages", "_scales", "_tail"))
            ring = ring.transpose(1, 2).contiguous()                   # [N, tail, Hkv, hd]
            ring[s["row_slot"].long(), s["row_pos"].long() % tail] = rows
            for r in range(N):
                p = pos[r * K]
                for b in range(p // BLOCK, (p + K) // BLOCK):
                    held = ring[r, b * BLOCK % tail:b * BLOCK % tail + BLOCK].transpose(0, 1)      # [Hkv, BLOCK, hd]
                    # the block's largest is a bf16 number of the ring
                    scale = _scale64(held.abs().amax((1, 2)).bfloat16().double())
                    i, t = table[r][b * BLOCK // page], b * BLOCK % page
                    pages[i, :, t:t + BLOCK] = held / scale[:, None, None]
                    scales[i, :, t // BLOCK] = scale
            out |= {name + "_pages": pages, name + "_scales": scales, name + "_tail": ring.transpose(1, 2).contiguous()}
        return out
    out = torch.zeros(N * K, Hq, hd, dtype=torch.float64, device="cuda")
    G = Hq // Hkv
    for r in range(N):
        n = max(pos[r * K:(r + 1) * K]) // BLOCK * BLOCK               # held in 8 bits for the last row
        at = table[r][:-(-n // page)]
        for h in range(Hkv):
            held = [(s[x + "_pages"][at, h].double().view(-1, BLOCK, hd) * s[x + "_scales"][at, h].double().reshape(-1, 1, 1)).view(-1, hd)
                    for x in "kv"] if at else [torch.zeros(0, hd, dtype=torch.float64, device="cuda")] * 2
            for j in range(K):
                p = pos[r * K + j]
                if p < 0:
                    continue
                a = p // BLOCK * BLOCK
                ring = slice(a % tail, a % tail + p - a + 1)
                k, v = (torch.cat([y[:a], s[x + "_tail"][r, h, ring].double()]) for x, y in zip("kv", held))
                w = torch.softmax(s["q"][r * K + j, h * G:(h + 1) * G].double() @ k.T / math.sqrt(hd), 1)
                out[r * K + j, h * G:(h + 1) * G] = w @ v
    return out
