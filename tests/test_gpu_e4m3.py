"""A decoding step held in 8 bits: quantisation, the product of e4m3 matrices, the
write into a cache held in e4m3 and the attention over it, against 64 bits."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean(gpu):
    B.biv_device_error()
    yield
    torch.cuda.synchronize()


def no_error():
    assert B.biv_device_error() == 0


def raw(t):
    return t.view(torch.uint8) if t.dtype == E.E4M3 else t


# ------------------------------------------------------------ quantisation
def quantised(x, block):
    rows, K = x.shape
    q = torch.empty(rows, K, dtype=E.E4M3, device="cuda")
    groups = -(-K // 128)
    s = torch.full((groups, rows) if block == 1 else (-(-rows // 128), groups), float("nan"), device="cuda")
    B.biv_quant_e4m3(x, q, s, block)
    return q, s


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (127, 256), (128, 1040), (129, 112), (300, 4096), (2049, 2048)])
def test_quant(rows, K, block):
    x = U.bf16(U.gen(rows + K), rows, K)
    x[0, :16] = torch.tensor([0, -0.0, 448, 1e-30, 3e38, -3e38, 1, 2, 3, -5, 7, 1e-40, 0.1, -448, 447, 0.5])
    if rows > 2:
        x[1] = 0                                            # nothing but zeros
        x[2] *= 1e-38
    q, s = quantised(x.cuda(), block)
    _, want, each = E.quant(x, block)
    assert torch.equal(s.cpu(), want)
    E.assert_nearest(q.cpu(), x, each)
    no_error()


def test_quant_of_what_is_not_finite():
    x = U.bf16(U.gen(1), 4, 256)
    x[0, 3], x[1, 200], x[2, 7], x[2, 9] = float("nan"), float("inf"), float("-inf"), float("nan")
    q, s = quantised(x.cuda(), 1)
    _, want, each = E.quant(x, 1)
    assert torch.equal(s.cpu(), want)
    E.assert_nearest(q.cpu(), x, each)


def test_quant_of_strided_rows():
    x = U.bf16(U.gen(2), 33, 520).cuda()
    a, b = quantised(x[:, 8:280], 1), quantised(x[:, 8:280].contiguous(), 1)
    assert all(torch.equal(raw(y), raw(z)) for y, z in zip(a, b))


def test_quant_rows_do_not_depend_on_others():
    x = U.bf16(U.gen(3), 1500, 4096).cuda()
    q, s = quantised(x, 1)
    q1, s1 = quantised(x[777:778], 1)
    assert torch.equal(raw(q[777:778]), raw(q1)) and torch.equal(s[:, 777:778], s1)


# ------------------------------------------------------------------- GEMM
def matrices(M, N, K, seed):
    g = U.gen(seed)
    qa, sa, ea = E.quant(U.bf16(g, M, K), 1)
    qb, sb, eb = E.quant(U.bf16(g, N, K, std=K ** -0.5), 128)
    return (qa, sa, ea), (qb, sb, eb), U.bf16(g, N, std=0.5), U.bf16(g, M, N)


def product(A, Bm, out, **kw):
    C = torch.full((A[0].shape[0], Bm[0].shape[0]), float("nan"), dtype=out, device="cuda")
    B.biv_gemm_e4m3(A[0].cuda(), A[1].cuda(), Bm[0].cuda(), Bm[1].cuda(), C, **kw)
    return C


# both forms; widths of one tile, of several, of a last one that is not full; k-blocks that fill sets and stages
# and that do not; K that is no multiple of 128
SHAPES = [(1, 8, 16), (1, 64, 128), (3, 136, 272), (8, 6144, 1024), (31, 200, 640), (33, 4096, 384), (64, 2048, 5120), (100, 1000, 896),
          (128, 256, 2048), (129, 256, 128), (160, 136, 208), (255, 1024, 1024), (300, 520, 1152), (320, 2560, 512), (513, 264, 400), (500, 28672, 144)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, out):
    A, Bm, _, _ = matrices(M, N, K, M + N + K)
    C = product(A, Bm, out).cpu().double()
    want, size = E.gemm(A[0], A[2], Bm[0], Bm[2])
    tol = E.gemm_tolerance(size, K) + want.abs() * U.HALF_STEP[out]
    bad = ~((C - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), ((C - want).abs() / tol).max())
    no_error()


@pytest.mark.parametrize("M,N,K", [(70, 12000, 400), (97, 12000, 400), (128, 19200, 640), (128, 12000, 128), (256, 8192, 272), (300, 12904, 528), (128, 24000, 272)])
def test_gemm_of_middle_widths(M, N, K):
    """Tiles of 65 to 192 columns, on both sides of the row count that chooses their form; two of them to a CTA; odd numbers of k-blocks."""
    A, Bm, bias, res = matrices(M, N, K, 9)
    C = product(A, Bm, torch.float32, bias=bias.cuda(), residual=res.cuda()).cpu().double()
    want, size = E.gemm(A[0], A[2], Bm[0], Bm[2])
    y = want + bias.double() + res.double()
    tol = E.gemm_tolerance(size, K) + (want.abs() + 2 * (want + bias.double()).abs() + 2 * y.abs()) * E.F32_STEP
    bad = ~((C - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), ((C - y).abs() / tol).max())
    rows = slice(3, 40)                                     # another form, the same bits
    few = product([x[rows] if x.shape[0] == M else x[:, rows] for x in A], Bm, torch.float32, bias=bias.cuda(), residual=res[rows].cuda())
    assert same_bits(few.cpu().double(), C[rows])
    no_error()


@pytest.mark.parametrize("M,N,K", [(5, 136, 272), (70, 264, 384), (200, 264, 400)])
@pytest.mark.parametrize("act", list(B.ACTS))
def test_gemm_tail(M, N, K, act):
    """Bias, activation and residual; tolerance: the sum's, carried through an activation whose slope is
    at most 1.13, plus the activation's (24 + 4 y) 2^-24 with y <= 40 here and the residual's rounding."""
    A, Bm, bias, res = matrices(M, N, K, M + N)
    want, size = E.gemm(A[0], A[2], Bm[0], Bm[2])
    x = want + bias.double()
    y = U.act(x, act) + res.double()
    tol = 1.13 * (E.gemm_tolerance(size, K) + x.abs() * E.F32_STEP) + (184 * x.abs() + 2 * y.abs()) * E.F32_STEP
    for out in (torch.bfloat16, torch.float32):
        C = product(A, Bm, out, bias=bias.cuda(), residual=res.cuda(), act=act).cpu().double()
        assert ((C - y).abs() <= tol + y.abs() * U.HALF_STEP[out]).all()


@pytest.mark.parametrize("M", [7, 190])
def test_gemm_onto_its_residual(M):
    A, Bm, _, res = matrices(M, 264, 256, 4)
    x = res.cuda()
    want = product(A, Bm, torch.bfloat16, residual=x)
    B.biv_gemm_e4m3(A[0].cuda(), A[1].cuda(), Bm[0].cuda(), Bm[1].cuda(), x, residual=x)
    assert same_bits(x, want)


@pytest.mark.parametrize("M,N,K,out", [(5, 72, 144, torch.float32), (130, 304, 256, torch.bfloat16), (70, 96, 256, torch.float32), (9, 1040, 128, torch.bfloat16)])
def test_gemm_into_rows_of_16_bytes(M, N, K, out):
    """C sixteen bytes off a 32-byte boundary: the bits that it has on one, and nothing beside it."""
    A, Bm, bias, res = matrices(M, N, K, 3)
    on = torch.zeros(M, N, dtype=out, device="cuda")
    room = torch.full((M * N + 64,), 7.0, dtype=out, device="cuda")
    step = 16 // on.element_size()
    off = room[step:step + M * N].view(M, N)
    assert on.data_ptr() % 32 == 0 and off.data_ptr() % 32 == 16
    for C in (on, off):
        B.biv_gemm_e4m3(A[0].cuda(), A[1].cuda(), Bm[0].cuda(), Bm[1].cuda(), C, bias=bias.cuda(), residual=res.cuda(), act="gelu")
    assert same_bits(on, off)
    assert (room[:step] == 7).all() and (room[step + M * N:] == 7).all()
    no_error()


# 28672: 256 columns a tile, pairs of CTAs where the number of 128-row tiles is even
@pytest.mark.parametrize("N,K", [(520, 1040), (4096, 1408), (28672, 400)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm_rows_do_not_depend_on_m(N, K, out):
    A, Bm, bias, res = matrices(600, N, K, 9)
    full = product(A, Bm, out, bias=bias.cuda(), residual=res.cuda())
    for M in (1, 2, 7, 33, 64, 127, 128, 129, 161, 256, 257, 333, 512):
        for first in (0, 600 - M):
            part = (A[0][first:first + M], A[1][:, first:first + M].contiguous(), None)
            got = product(part, Bm, out, bias=bias.cuda(), residual=res[first:first + M].cuda())
            assert same_bits(got, full[first:first + M]), (M, first)


def test_gemm_with_what_is_not_finite():
    """A NaN stays in its row, or its column; zeros times it are NaN there and nowhere else."""
    for M in (40, 200):
        A, Bm, _, _ = matrices(M, 256, 256, 5)
        A[0][3, 100] = float("nan")
        Bm[0][77, 9] = float("nan")
        C = product(A, Bm, torch.float32).cpu()
        bad = torch.zeros(M, 256, dtype=torch.bool)
        bad[3], bad[:, 77] = True, True
        assert torch.equal(C.isnan(), bad)


# ------------------------------------------------------------------ write
class Cache:
    """An empty cache on the GPU: everything NaN, pages of the slots in order behind one that nobody has."""

    def __init__(self, slots, Hkv, hd, page, tail, max_pages):
        nan = float("nan")
        n = slots * max_pages + 1
        self.page, self.tail, self.Hkv, self.hd = page, tail, Hkv, hd
        self.pages = [torch.full((n, Hkv, page, hd), nan).to(E.E4M3).cuda() for _ in "kv"]
        self.scales = [torch.full((n, Hkv, page // 16), nan, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        self.tails = [torch.full((slots, Hkv, tail, hd), nan, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        self.table = torch.arange(1, n, dtype=torch.int32, device="cuda").view(slots, max_pages)
        self.cap = page * max_pages

    def args(self):
        return (*self.pages, *self.scales, *self.tails, self.table)

    def write(self, qkv, slot, pos, Hq, theta, K, keep=None):
        q = torch.full((len(slot), Hq, self.hd), float("nan"), dtype=torch.bfloat16, device="cuda")
        i32 = lambda v: torch.as_tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        B.biv_rope_kv_write_paged_e4m3(qkv.cuda(), q, *self.args(), i32(slot), i32(pos), theta, K,
                                       rows_keep=None if keep is None else i32(keep))
        return q

    def state(self):
        return [raw(t).clone() for t in (*self.pages, *self.scales, *self.tails)]


def check_rows(got, want, a, b):
    """bf16 of a rotation: half a step and the fp32 roundings of its two products, their sum, sine and cosine."""
    tol = want.abs() * U.HALF_STEP[torch.bfloat16] + (a.abs() + b.abs()) * 8 * E.F32_STEP
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), int(bad.sum())


def rotated(x, pos, theta):
    y = U.rope(x, pos, theta)
    hd = x.shape[-1]
    return y, x.double().roll(hd // 2, -1)


def check_write(cache, qkv, slot, pos, Hq, theta, q, before):
    """Rows against 64 bits; the blocks in the pages against the ring's own rows; nothing else has changed."""
    Hkv, hd, tail, page = cache.Hkv, cache.hd, cache.tail, cache.page
    x = qkv.view(len(slot), Hq + 2 * Hkv, hd)
    pos_t = torch.tensor(pos)
    y, other = rotated(x[:, :Hq + Hkv], pos_t, theta)
    check_rows(q.cpu(), y[:, :Hq], x[:, :Hq].double(), other[:, :Hq])
    want = [t.cpu().clone() for t in before]
    filled = set()
    for w, (s, p) in enumerate(zip(slot, pos)):
        if p < 0:
            continue
        got_k, got_v = (cache.tails[i][s, :, p % tail].cpu() for i in range(2))
        check_rows(got_k, y[w, Hq:], x[w, Hq:Hq + Hkv].double(), other[w, Hq:])
        assert same_bits(got_v, x[w, Hq + Hkv:])
        want[4][s, :, p % tail], want[5][s, :, p % tail] = got_k, got_v
        if p % 16 == 15:
            filled.add((s, p // 16))
    for s, b in filled:
        at, i = int(cache.table[s, b * 16 // page]), b % (page // 16)
        for n in range(2):
            rows = cache.tails[n][s, :, b * 16 % tail:b * 16 % tail + 16].cpu()        # [Hkv, 16, hd]
            scale = E.scale_up(E.top(rows, (1, 2)))
            assert same_bits(cache.scales[n][at, :, i].cpu(), scale)
            got = cache.pages[n][at, :, 16 * i:16 * i + 16].cpu()
            E.assert_nearest(got, rows, scale.double()[:, None, None])
            want[n][at, :, 16 * i:16 * i + 16], want[2 + n][at, :, i] = got.view(torch.uint8), scale
    for got, w in zip(cache.state(), want):
        g, w = got.cpu(), w
        assert torch.equal(g.view(torch.int16) if g.dtype == torch.bfloat16 else g, w.view(torch.int16) if w.dtype == torch.bfloat16 else w)
    return filled


@pytest.mark.parametrize("Hq,Hkv,hd,page,K,tail", [(8, 2, 128, 16, 1, 16), (4, 4, 64, 32, 1, 48), (32, 8, 128, 64, 5, 32), (8, 1, 64, 16, 16, 32),
                                                    (12, 4, 128, 256, 33, 48), (8, 2, 128, 128, 200, 224)])
def test_write(Hq, Hkv, hd, page, K, tail):
    """Windows one after the other, from positions that fill blocks, cross pages and wrap the ring; seats
    without a request, and a window that ends early."""
    theta, slots = 10000.0, 3
    cache = Cache(slots, Hkv, hd, page, tail, -(-(6 * K + 700) // page))
    g = U.gen(K + hd)
    at = [0, 13, 5 * 16 + 15]
    for i in range(3):                                      # rows of the started blocks
        if at[i] % 16:
            for t in cache.tails:
                for p in range(at[i] // 16 * 16, at[i]):
                    t[i, :, p % tail] = U.bf16(g, Hkv, hd).cuda()
    total = 0
    for step in range(5):
        slot, pos = [], []
        for i in (2, 0, 1):
            n = 0 if (step + i) % 4 == 3 else K if step % 2 == 0 else (K + 1) // 2       # rows of this window
            slot += [i] * K
            pos += [at[i] + j if j < n else -1 for j in range(K)]
            at[i] += n
        qkv = U.bf16(g, 3 * K, (Hq + 2 * Hkv) * hd)
        before = cache.state()
        q = cache.write(qkv, slot, pos, Hq, theta, K)
        total += len(check_write(cache, qkv, slot, pos, Hq, theta, q, before))
    no_error()
    assert K < 5 or total > 0


def test_write_far_positions():
    cache = Cache(1, 2, 128, 256, 32, 1 << 14)
    g = U.gen(8)
    for p in (4194302, 4194303):
        qkv, before = U.bf16(g, 1, 8 * 128), cache.state()
        for t in cache.tails:
            t[0] = 1.0
        before = cache.state()
        q = cache.write(qkv, [0], [p], 4, 500000.0, 1)
        check_write(cache, qkv, [0], [p], 4, 500000.0, q, before)
    no_error()


def test_write_does_not_depend_on_the_window():
    """One row at a time, in windows of 7, at once, or with rejected drafts in between: the same cache."""
    n, Hq, Hkv, hd = 70, 4, 2, 64
    g = U.gen(9)
    qkv, wrong = U.bf16(g, n, (Hq + 2 * Hkv) * hd), U.bf16(g, n + 7, (Hq + 2 * Hkv) * hd, std=9.0)
    states = []
    for kind in ("rows", "windows", "once", "drafts"):
        cache = Cache(1, Hkv, hd, 32, 96, 4)
        K = {"rows": 1, "windows": 7, "once": n, "drafts": 7}[kind]
        at = 0
        while at < n:
            take = 3 if kind == "drafts" else K
            take = min(take, n - at)
            x = torch.cat([qkv[at:at + take], wrong[at:at + K - take]])
            pos = [at + j if kind == "drafts" or j < take else -1 for j in range(K)]
            cache.write(x, [0] * K, pos, Hq, 1e4, K)
            at += take
        if kind == "drafts":                                # the last window's drafts are in the ring: overwrite none of them
            cache.tails = [t.clone() for t in cache.tails]
            for t in cache.tails:
                t[0, :, n:] = float("nan")
        states.append([*cache.pages, *cache.scales, *cache.tails])
    for other in states[1:]:
        for i, (a, b) in enumerate(zip(states[0], other)):
            if i < 4:                                       # blocks that are full
                a, b = (raw(t)[1:3] if i < 2 else t[1:3] for t in (a, b))
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    no_error()


def test_write_keeps_rows():
    """Rows past rows_keep are rotated only, and do not fill a block."""
    Hq, Hkv, hd, K = 4, 2, 128, 8
    g = U.gen(10)
    qkv = U.bf16(g, 2 * K, (Hq + 2 * Hkv) * hd)
    slot, pos = [0] * K + [1] * K, [8 + j for j in range(K)] * 2
    cache = Cache(2, Hkv, hd, 16, 32, 4)
    for t in cache.tails:
        t[:, :, :8] = 1.0
    before = cache.state()
    q = cache.write(qkv, slot, pos, Hq, 1e4, K, keep=[8, 7])
    kept = [p if w < K or w % K < 7 else -1 for w, p in enumerate(pos)]
    y, other = rotated(qkv.view(2 * K, -1, hd)[:, :Hq], torch.tensor(pos), 1e4)
    check_rows(q.cpu(), y, qkv.view(2 * K, -1, hd)[:, :Hq].double(), other)
    rows = torch.tensor(kept) >= 0
    q2 = q.clone()
    q2[~rows.cuda()] = 0
    x = qkv.clone()
    x[~rows] = 0
    assert check_write(cache, x, slot, kept, Hq, 1e4, q2, before) == {(0, 0)}
    no_error()


@pytest.mark.parametrize("groups", [2, 300])
def test_write_of_a_slot_by_two_groups(groups):
    """Neither would see the other's rows when it fills a block: the error word says so.  Empty groups, and those that keep
    no row, may name any slot."""
    K, Hq, Hkv, hd = 4, 2, 1, 64
    cache = Cache(groups, Hkv, hd, 16, 32, 2)
    qkv = U.bf16(U.gen(1), groups * K, (Hq + 2 * Hkv) * hd)
    pos = [j for _ in range(groups) for j in range(K)]
    slots = list(range(groups))
    slots[-1] = 0
    rows = lambda s: [x for x in s for _ in range(K)]  # noqa: E731
    cache.write(qkv, rows(range(groups)), pos, Hq, 1e4, K)
    no_error()
    cache.write(qkv, rows(slots), pos[:-K] + [-1] * K, Hq, 1e4, K)
    no_error()
    cache.write(qkv, rows(slots), pos, Hq, 1e4, K, keep=[K] * (groups - 1) + [0])
    no_error()
    cache.write(qkv, rows(slots), pos, Hq, 1e4, K)
    torch.cuda.synchronize()
    assert B.biv_device_error() == B.DEVERR_GROUP


@pytest.mark.parametrize("fault,bit", [("slot", B.DEVERR_INDEX), ("far", B.DEVERR_INDEX), ("negative", B.DEVERR_INDEX), ("page", B.DEVERR_INDEX),
                                       ("gap", B.DEVERR_GROUP), ("jump", B.DEVERR_GROUP), ("other", B.DEVERR_GROUP)])
def test_write_faults(fault, bit):
    """A row at fault is not written and no block with it is; rows before it are."""
    Hq, Hkv, hd, K = 4, 2, 64, 16
    cache = Cache(2, Hkv, hd, 16, 32, 4)
    slot, pos = [1] * K, list(range(16, 32))
    if fault == "slot":
        slot = [7] * K
    if fault == "far":
        pos = list(range(64, 80))
    if fault == "negative":
        pos = list(range(-48, -32))
    if fault == "page":
        cache.table[1, 1] = 9
    if fault == "gap":
        pos[5] = -1
    if fault == "jump":
        pos[9] = 40
    if fault == "other":
        slot[9] = 0
    before = cache.state()
    qkv = U.bf16(U.gen(11), K, (Hq + 2 * Hkv) * hd)
    q = cache.write(qkv, slot, pos, Hq, 1e4, K)
    y, other = rotated(qkv.view(K, -1, hd)[:, :Hq], torch.tensor(pos), 1e4)
    check_rows(q.cpu(), y, qkv.view(K, -1, hd)[:, :Hq].double(), other)
    assert B.biv_device_error() == bit
    after = cache.state()
    for i in range(4):
        assert torch.equal(before[i].view(torch.uint8), after[i].view(torch.uint8))
    written = [i for i in range(2) if not torch.equal(before[4][i].view(torch.int16), after[4][i].view(torch.int16))]
    assert written == ([] if bit == B.DEVERR_INDEX and fault != "page" else [1])


# -------------------------------------------------------------- attention
def attend(pool, q, slot, pos, rpg, o=None):
    W, Hq, hd = q.shape
    t = pool.on()
    ws = torch.full((B.biv_decode_attn_paged_workspace_size(W, Hq, hd, pool.table.shape[1], pool.page),), 255, dtype=torch.uint8, device="cuda")
    o = torch.full((W, Hq, hd), float("nan"), dtype=torch.bfloat16, device="cuda") if o is None else o
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    B.biv_decode_attn_paged_e4m3(q.cuda(), *t, i32(slot), i32(pos), o, rpg, ws)
    return o


def check_attention(o, q, pool, slot, pos):
    want, tol = E.attention(q, pool, slot, pos)
    bad = ~((o.cpu().double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((o.cpu().double() - want).abs() / tol.clamp(min=1e-30)).max()))


@pytest.mark.parametrize("Hq,Hkv,hd,page", [(8, 2, 128, 16), (32, 8, 64, 64), (8, 8, 128, 256), (16, 1, 64, 32), (6, 2, 128, 128), (8, 1, 128, 16)])
def test_attention_single_tokens(Hq, Hkv, hd, page):
    lengths = [1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257, 272, 511, 512, 513, 700, 1025]
    pool = E.HeldPool(lengths, Hkv, hd, page, seed=hd + Hq)
    q = U.bf16(U.gen(1), len(lengths), Hq, hd, std=1.5)
    slot, pos = list(range(len(lengths))), [n - 1 for n in lengths]
    o = attend(pool, q, slot, pos, 1)
    check_attention(o, q, pool, slot, pos)
    no_error()
    for r in (0, 5, 16):                                    # a row alone: the same bits
        assert same_bits(attend(pool, q[r:r + 1], [r], [pos[r]], 1), o[r:r + 1])


@pytest.mark.parametrize("Hq,Hkv,hd,page,K", [(8, 2, 128, 16, 5), (32, 8, 64, 64, 2), (8, 8, 128, 32, 16), (16, 2, 64, 128, 4), (8, 1, 128, 256, 5),
                                               (4, 2, 128, 16, 33)])
def test_attention_windows(Hq, Hkv, hd, page, K):
    """Windows whose rows lie in one block, in two, in many; each row has the bits that it has alone."""
    lengths = [K, K + 1, 16 + K // 2, 250 + K, 257 + K, 530 + K, 1023 + K]
    pool = E.HeldPool(lengths, Hkv, hd, page, seed=K, tail=16 * -(-(K + 15) // 16))
    N = len(lengths)
    q = U.bf16(U.gen(2), N * K, Hq, hd, std=1.5)
    slot = [r for r in range(N) for _ in range(K)]
    pos = [n - K + j for n in lengths for j in range(K)]
    pos[K - 1] = -1                                         # an empty seat in the first window
    o = attend(pool, q, slot, pos, K)
    check_attention(o, q, pool, slot, pos)
    no_error()
    assert same_bits(attend(pool, q, slot, pos, 1), o)
    half = (N // 2) * K
    assert same_bits(attend(pool, q[half:], slot[half:], pos[half:], K), o[half:])


def test_attention_of_a_long_context():
    pool = E.HeldPool([20011], 2, 128, 256, seed=3)
    q = U.bf16(U.gen(3), 1, 8, 128, std=1.5)
    check_attention(attend(pool, q, [0], [20010], 1), q, pool, [0], [20010])
    no_error()


@pytest.mark.parametrize("N,K", [(1100, 1), (150, 4)])
def test_attention_of_many_rows(N, K):
    """More rows, and more groups, than a CTA keeps a table of; requests share slots."""
    lengths = [4, 40, 515, 77]
    pool = E.HeldPool(lengths, 1, 64, 16, seed=7)
    q = U.bf16(U.gen(8), N * K, 2, 64, std=1.5)
    slot = [r % 4 for r in range(N) for _ in range(K)]
    pos = [lengths[r % 4] - K + j for r in range(N) for j in range(K)]
    for w in range(0, N * K, 37):
        pos[w] = -1
    o = attend(pool, q, slot, pos, K)
    check_attention(o, q, pool, slot, pos)
    some = slice(5 * K, 9 * K)
    assert same_bits(attend(pool, q[some], slot[some], pos[some], K), o[some])
    no_error()


@pytest.mark.parametrize("K,hd,Hq,Hkv", [(1, 128, 8, 2), (5, 128, 8, 2), (3, 64, 16, 1)])
@pytest.mark.parametrize("cap", [512, 1024, 2048, 4096])
def test_attention_does_not_depend_on_the_tables_width(K, hd, Hq, Hkv, cap):
    """A table's width says how a call is split among CTAs, no more: tables of one to eight splits and of twenty."""
    lengths = [n for n in (K, 16, 100, 511, 512, 513, 528, 1000, 1537, 2048, 3100, 4096) if n <= cap]
    q, outs = U.bf16(U.gen(4), len(lengths) * K, Hq, hd, std=1.5), []
    slot = [r for r in range(len(lengths)) for _ in range(K)]
    pos = [n - K + j for n in lengths for j in range(K)]
    pos[2 * K] = -1
    for wide in (cap, 10240):
        pool = E.HeldPool(lengths, Hkv, hd, 16, seed=5, cap=wide)
        outs.append(attend(pool, q, slot, pos, K))
    if K == 1:
        check_attention(outs[0], q, pool, slot, pos)
    assert same_bits(outs[0], outs[1])
    no_error()


def test_attention_does_not_depend_on_pages():
    """Page size, ring and the pages' order are where keys lie, no more."""
    q, outs = U.bf16(U.gen(4), 2, 8, 64), []
    for page, tail, spare in ((16, 16, 3), (64, 48, 0), (256, 32, 7)):
        pool = E.HeldPool([300, 77], 2, 64, page, seed=5, tail=tail, spare=spare, rows_seed=6)
        outs.append(attend(pool, q, [0, 1], [299, 76], 1))
    assert same_bits(outs[0], outs[1]) and same_bits(outs[0], outs[2])


@pytest.mark.parametrize("std", [1e-4, 30.0, 3e4])
def test_attention_of_extreme_queries(std):
    """Rows of very small and very large queries (one key takes all of the weight), and a row of zeros."""
    pool = E.HeldPool([200, 333, 64], 2, 128, 32, seed=6)
    q = U.bf16(U.gen(5), 3, 4, 128, std=std)
    q[0, 0] = 0
    q[1, 1, 5] = 1e30 if std > 1e4 else q[1, 1, 5]
    slot, pos = [0, 1, 2], [199, 332, 63]
    o = attend(pool, q, slot, pos, 1).cpu()
    assert o.float().isfinite().all()
    if std < 1e4:
        want, tol = E.attention(q, pool, slot, pos)
        bad = ~((o.double() - want).abs() <= tol)
        assert not bad.any()


def test_attention_rows_without_a_result():
    """Empty seats, slots and positions out of range, rows of another slot than their group's, pages out of range."""
    lengths = [100, 200, 300, 40]
    pool = E.HeldPool(lengths, 2, 64, 16, seed=7)
    q = U.bf16(U.gen(6), 4, 4, 64)
    zero = torch.zeros(4, 64)
    o = attend(pool, q, [0, 1, 2, 3], [99, -1, 299, 39], 1)
    assert torch.equal(o[1].cpu().float(), zero)
    no_error()
    for slot, pos, bit in (([0, 9, 2, 3], [99, 199, 299, 39], B.DEVERR_INDEX), ([0, 1, 2, 3], [99, 16 * pool.table.shape[1], 299, 39], B.DEVERR_INDEX),
                           ([0, 1, 2, 3], [99, -7, 299, 39], B.DEVERR_INDEX)):
        got = attend(pool, q, slot, pos, 1)
        assert torch.equal(got[1].cpu().float(), zero) and same_bits(got[[0, 2, 3]], o[[0, 2, 3]])
        assert B.biv_device_error() == bit
    got = attend(pool, q, [0, 1, 2, 3], [99, 199, 299, 39], 2)
    assert torch.equal(got[1].cpu().float(), zero) and torch.equal(got[3].cpu().float(), zero)
    assert same_bits(got[[0, 2]], o[[0, 2]])
    assert B.biv_device_error() == B.DEVERR_GROUP


@pytest.mark.parametrize("K", [1, 3])
def test_attention_pages_out_of_range(K):
    """Rows that reach such a page come back as zeros; the others, in the same window too, do not see it.  The page
    of a row's own block is not read."""
    pool = E.HeldPool([67, 150], 2, 64, 16, seed=8)
    pool.table[0, 4] = 99                                   # positions 64..79: no row of this window has them held
    pool.table[1, 8] = -1                                   # 128..143: held for rows from 144 on
    first = [64, 142] if K == 3 else [66, 149]
    q = U.bf16(U.gen(7), 2 * K, 4, 64)
    slot, pos = [0] * K + [1] * K, [p + j for p in first for j in range(K)]
    o = attend(pool, q, slot, pos, K)
    assert B.biv_device_error() == B.DEVERR_INDEX
    want, tol = E.attention(q, pool, slot, pos)
    gone = [w for w in range(2 * K) if slot[w] == 1 and pos[w] >= 144]
    for w in range(2 * K):
        if w in gone:
            assert (o[w] == 0).all()
        else:
            assert ((o[w].cpu().double() - want[w]).abs() <= tol[w]).all(), w


def test_attention_on_a_captured_graph_and_another_stream():
    pool = E.HeldPool([600, 1000], 2, 128, 64, seed=9)
    q = U.bf16(U.gen(8), 2, 8, 128).cuda()
    want = attend(pool, q, [0, 1], [599, 999], 1)
    t = pool.on()
    slot, pos = torch.tensor([0, 1]).int().cuda(), torch.tensor([599, 999]).int().cuda()
    n = B.biv_decode_attn_paged_workspace_size(2, 8, 128, pool.table.shape[1], 64)
    ws, o = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.biv_decode_attn_paged_e4m3(q, *t, slot, pos, o, 1, ws)
    s.synchronize()
    assert same_bits(o, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biv_decode_attn_paged_e4m3(q, *t, slot, pos, o, 1, ws)
    o.zero_()
    ws.fill_(255)
    g.replay()
    torch.cuda.synchronize()
    assert same_bits(o, want)


# --------------------------------------------------------------- together
def test_a_step_of_single_tokens_is_a_window():
    """Write and attention one row at a time, in windows, and over a whole prompt: the same rows out."""
    n, Hq, Hkv, hd = 75, 8, 2, 64
    qkv = U.bf16(U.gen(12), n, (Hq + 2 * Hkv) * hd)
    outs = []
    for K in (1, 5, n):
        cache = Cache(1, Hkv, hd, 16, 16 * -(-(K + 15) // 16), 5)
        rows = []
        for a in range(0, n, K):
            pos = torch.arange(a, a + K, dtype=torch.int32)
            q = cache.write(qkv[a:a + K], [0] * K, pos, Hq, 1e4, K)
            o = torch.empty_like(q)
            ws = torch.empty(B.biv_decode_attn_paged_workspace_size(K, Hq, hd, 5, 16), dtype=torch.uint8, device="cuda")
            B.biv_decode_attn_paged_e4m3(q, *cache.args(), torch.zeros(K, dtype=torch.int32, device="cuda"), pos.cuda(), o, K, ws)
            rows.append(o)
        outs.append(torch.cat(rows))
    assert same_bits(outs[0], outs[1]) and same_bits(outs[0], outs[2])
    no_error()


# ------------------------------------------------- the binding's way and abi.py's
def calls(seed=0):
    """name -> arguments, and the indexes of the outputs and of the tensors whose last dimension is theirs to choose."""
    g = U.gen(seed)
    b = lambda *shape: U.bf16(g, *shape).cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    A, Bm, bias, res = matrices(5, 72, 144, seed)
    x = b(40, 272)
    cache = Cache(2, 2, 64, 16, 32, 3)
    for t in (*cache.pages, *cache.scales, *cache.tails):
        t.view(torch.uint8).zero_()
    ws = torch.empty(B.biv_decode_attn_paged_workspace_size(2, 4, 64, 3, 16), dtype=torch.uint8, device="cuda")
    slot, pos = i32([0, 1]), i32([15, 40])
    return {
        "biv_quant_e4m3": ([x, torch.zeros(40, 272, device="cuda").to(E.E4M3), torch.zeros(3, 40, device="cuda")], (1, 2), ()),
        "biv_gemm_e4m3": ([A[0].cuda(), A[1].cuda(), Bm[0].cuda(), Bm[1].cuda(), torch.zeros(5, 72, device="cuda"), bias.cuda(), res.cuda()], (4,), ()),
        "biv_rope_kv_write_paged_e4m3": ([b(2, 8 * 64), torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), *cache.args(), slot, pos, 1e4, 1],
                                         (1, 2, 3, 4, 5, 6, 7), (8,)),
        "biv_decode_attn_paged_e4m3": ([b(2, 4, 64), *[b(*t.shape).to(t.dtype) for t in cache.args()[:6]], cache.table, slot, pos,
                                        torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), 1, ws], (10,), (7, 12)),
    }


NAMES = ["biv_quant_e4m3", "biv_gemm_e4m3", "biv_rope_kv_write_paged_e4m3", "biv_decode_attn_paged_e4m3"]


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_agree(name):
    def run(**kw):
        args, out, _ = calls()[name]
        torch.cuda.synchronize()
        getattr(B, name)(*args, **kw)
        torch.cuda.synchronize()
        no_error()
        return [raw(args[i]).clone() for i in out]

    direct = run()
    assert all(bool((x != 0).any()) for x in direct[:2])
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream().cuda_stream):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(direct, run(stream=stream)))


@pytest.mark.parametrize("fault", ["type", "shape", "stride", "device"])
@pytest.mark.parametrize("name", NAMES)
def test_a_fault_has_its_status(name, fault):
    good, _, own = calls()[name]
    for at, x in enumerate(good):
        if not isinstance(x, torch.Tensor) or at in own:
            continue
        if fault == "type":
            bad, status = x.to(torch.float64), 4
        elif fault == "device":
            bad, status = x.cpu(), 7
        elif fault == "stride":
            bad, status = torch.zeros(*x.shape, 2, device="cuda").to(x.dtype)[..., 0], 2
        else:
            bad, status = torch.zeros(*x.shape[:-1], x.shape[-1] + 16, device="cuda").to(x.dtype), 2
        args = list(good)
        args[at] = bad
        with pytest.raises(B.BivError) as e:
            getattr(B, name)(*args)
        assert e.value.status == status, (at, str(e.value))
