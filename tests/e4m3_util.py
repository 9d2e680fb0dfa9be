"""Plain 64-bit forms of the operators on e4m3 numbers, for their tests (torch on
the CPU; no code of the package)."""
import torch

from paged_util import HALF_STEP, bf16, gen, rope  # noqa: F401

E4M3 = torch.float8_e4m3fn
BLOCK, TOP, LEAST = 16, 448.0, 2.0 ** -100
F32_STEP = 2.0 ** -24
LARGEST = float(torch.finfo(torch.bfloat16).max)


def top(x, dims):
    """max |x| as the scale counts it: a NaN is nothing, an infinity the largest bf16 number."""
    return torch.where(x.isnan(), 0.0, x.double().abs()).clamp(max=LARGEST).amax(dims)


def scale(t):
    """The fp32 scale of values up to t: a quotient of two numbers of at most 8 bits, rounded once."""
    return (t / TOP).clamp(min=LEAST).float()


def scale_up(t):
    """The next bf16 number."""
    bits = (scale(t).view(torch.int32) + 0xffff) & -65536
    return bits.view(torch.float32).to(torch.bfloat16)


def assert_nearest(q, x, s):
    """q (e4m3) is x / s rounded to nearest: at most half a step away, which is 2^-4 of the
    value, or half of the smallest number's 2^-9.  The quotient that is rounded may be off by
    2^-23 of itself."""
    want = x.double() / s.double()
    got = q.float().double()
    fine = x.double().isfinite()
    assert got[~fine].isnan().all() and not got[fine].isnan().any()
    err, tol = (got - want).abs(), torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) * (1 + 2.0 ** -18)
    bad = fine & (err > tol)
    assert not bad.any(), (int(bad.sum()), x[bad][:4], got[bad][:4], want[bad][:4])


def quant(x, block):
    """(e4m3 values, scales in the kernels' layout, scales of every element) of x [rows, K]."""
    rows, K = x.shape
    groups = -(-K // 128)
    up = torch.zeros(-(-rows // block) * block, groups * 128, dtype=torch.float64)
    up[:rows, :K] = torch.where(x.isnan(), 0.0, x.double())
    t = top(up.view(-1, block, groups, 128), (1, 3))
    s = scale(t)
    each = s.repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :K]
    q = (x.double() / each.double()).float().to(E4M3)
    return q, (s.t().contiguous() if block == 1 else s), each


def gemm(A, each_a, B, each_b):
    """(A B^T, sum of the products' sizes) in 64 bits."""
    a, b = A.float().double() * each_a.double(), B.float().double() * each_b.double()
    return a @ b.t(), a.abs() @ b.abs().t()


def gemm_tolerance(size, K):
    """What a sum may be off by: a tensor core's MMA of 32 terms cuts each of up to 33 addends by at most
    2^-23 of the largest, four of them a block; fp32 roundings of scales (2), block and sum."""
    return size * (4 * 33 * 2.0 ** -23 + (-(-K // 128) + 4) * F32_STEP)


class HeldPool:
    """Requests of the given lengths (positions 0..n-1 hold keys), their full blocks in e4m3 in
    shuffled pages, the last `tail` rows of each in its ring; what lies elsewhere is NaN."""

    def __init__(self, lengths, Hkv, hd, page, seed, tail=32, spare=3, cap=None, rows_seed=None):
        g = gen(seed)
        nan = float("nan")
        self.lengths, self.page, self.tail = list(lengths), page, tail
        need = [-(-n // page) for n in self.lengths]
        wide = max([1, *need]) if cap is None else -(-cap // page)
        total = sum(need) + spare
        order = torch.randperm(total, generator=g).tolist()
        self.table = torch.full((len(self.lengths), wide), -1, dtype=torch.int32)
        shape = (total, Hkv, page // BLOCK, BLOCK, hd)
        self.pages = [torch.full(shape, nan).to(E4M3) for _ in "kv"]
        self.scales = [torch.full(shape[:3], nan, dtype=torch.bfloat16) for _ in "kv"]
        self.tails = [torch.full((len(self.lengths), Hkv, tail, hd), nan, dtype=torch.bfloat16) for _ in "kv"]
        self.rows, self.held = [], []                    # (k, v) [Hkv, n, hd] of each request: bf16, and as held
        at = 0
        if rows_seed is not None:
            g = gen(rows_seed)
        for r, n in enumerate(self.lengths):
            ids = order[at:at + need[r]]
            at += need[r]
            self.table[r, :need[r]] = torch.tensor(ids, dtype=torch.int32)
            rows, held = [], []
            for x in range(2):
                y = bf16(g, Hkv, n, hd, std=1.0 + 2.0 * x)
                full = n // BLOCK
                blocks = y[:, :full * BLOCK].reshape(Hkv, full, BLOCK, hd)
                s = scale_up(top(blocks, (2, 3))) if full else torch.zeros(Hkv, 0, dtype=torch.bfloat16)
                q = (blocks.double() / s.double()[..., None, None]).float().to(E4M3)
                for b in range(full):
                    p, i = ids[b * BLOCK // page], b % (page // BLOCK)
                    self.pages[x][p, :, i] = q[:, b]
                    self.scales[x][p, :, i] = s[:, b]
                for t in range(max(0, n - tail), n):
                    self.tails[x][r, :, t % tail] = y[:, t]
                rows.append(y)
                held.append((q.float().double() * s.double()[..., None, None]).reshape(Hkv, full * BLOCK, hd))
            self.rows.append(rows)
            self.held.append(held)
        self.pages = [p.view(total, Hkv, page, hd) for p in self.pages]

    def on(self, device="cuda"):
        """The call's tensors: k_pages, v_pages, k_scales, v_scales, k_tail, v_tail, page_table."""
        return [t.to(device) for t in (*self.pages, *self.scales, *self.tails, self.table)]


def seen(pool, r, p):
    """(k, v) in 64 bits that a row at position p of request r reads."""
    a = p // BLOCK * BLOCK
    return [torch.cat([h[:, :a], y[:, a:p + 1].double()], 1) for h, y in zip(pool.held[r], pool.rows[r])]


def attention(q, pool, slot, pos):
    """(o, tolerance) in 64 bits.  The tolerance: half a bf16 step of o; fp32 scores (sums of hd products,
    each partial sum within 2^-23, and the products with the row's and the block's scales) move every weight by
    at most twice that relative error; a weight rounded to 11 bits moves o by at most 2^-12 of sum p |v| itself and
    as much by the sum that it is in; the exponential, the sums and weights below fp16's normal numbers
    stay below 2^-14 of it."""
    W, Hq, hd = q.shape
    o = torch.zeros(W, Hq, hd, dtype=torch.float64)
    tol = torch.zeros_like(o)
    for w in range(W):
        if pos[w] < 0:
            continue
        k, v = seen(pool, int(slot[w]), int(pos[w]))
        G = Hq // k.shape[0]
        for h in range(Hq):
            qh, kh, vh = q[w, h].double(), k[h // G], v[h // G]
            p = torch.softmax(kh @ qh * hd ** -0.5, 0)
            o[w, h] = p @ vh
            ds = (kh.abs() @ qh.abs()).max() * hd ** -0.5 * (hd + 4) * 2.0 ** -23
            tol[w, h] = HALF_STEP[torch.bfloat16] * o[w, h].abs() + (2 * ds + 2.0 ** -11 + 2.0 ** -14) * (p @ vh.abs())
    return o, tol
