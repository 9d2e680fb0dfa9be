"""The paged cache write, the paged attention and the bias/activation/residual
GEMM against plain 64-bit forms, and what must not change a row's bits."""
import pytest
import torch

import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu

BIG = 1e30


def within(got, ref, tol, what=""):
    err = (got.detach().double().cpu() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).nan_to_num(nan=torch.inf).max()):.3g} of the tolerance"


def nan_like(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def attend(q, pool, slot, pos, rpg=1, ws_fill=255, **kw):
    """The call with an output of NaN and a workspace full of rubbish."""
    W, Hq, hd = q.shape
    k, v, table = (kw.get(n, getattr(pool, n)).cuda() for n in ("k", "v", "table"))
    n = B.biv_decode_attn_paged_workspace_size(W, Hq, hd, table.shape[1], pool.page)
    ws = torch.full((max(n, 16),), ws_fill, dtype=torch.uint8, device="cuda")
    o = nan_like(W, Hq, hd)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    B.biv_decode_attn_paged(q.cuda(), k, v, table, i32(slot), i32(pos), o, rpg, ws)
    torch.cuda.synchronize()
    return o


def wide(pool):
    """The pool's table with columns for 5000 more keys: too many splits for the one-launch form."""
    return torch.cat([pool.table, torch.full((pool.table.shape[0], -(-5000 // pool.page)), -1, dtype=torch.int32)], 1)


LENGTHS = [1, 2, 15, 16, 17, 255, 256, 257, 700, 1030]


@pytest.mark.parametrize("Hq,Hkv,hd", [(8, 2, 128), (4, 4, 64), (32, 2, 128), (12, 4, 64), (17, 1, 128), (40, 8, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attention_single_rows(Hq, Hkv, hd, page):
    pool = U.Pool(LENGTHS, Hkv, hd, page, seed=page + Hq)      # NaN wherever no key lies
    N = len(LENGTHS)
    q = U.bf16(U.gen(7), N, Hq, hd, std=1.5)
    pos = [n - 1 for n in LENGTHS]
    o = attend(q, pool, range(N), pos)
    assert B.biv_device_error() == 0
    within(o, *U.attention(q, pool.rows, range(N), pos))


@pytest.mark.parametrize("K", [2, 3, 5, 16, 33])
@pytest.mark.parametrize("hd,Hq,Hkv", [(128, 8, 2), (64, 6, 2), (128, 3, 3)])
def test_attention_windows(K, hd, Hq, Hkv):
    lengths = [max(n, K) for n in (K, 40, 257, 600)]
    pool = U.Pool(lengths, Hkv, hd, 32, seed=K)
    N = len(lengths)
    q = U.bf16(U.gen(9), N * K, Hq, hd, std=1.5)
    slot = [r for r in range(N) for _ in range(K)]
    pos = [n - K + j for n in lengths for j in range(K)]
    o = attend(q, pool, slot, pos, rpg=K)
    assert B.biv_device_error() == 0
    within(o, *U.attention(q, pool.rows, slot, pos))
    assert same_bits(attend(q, pool, slot, pos, rpg=K, table=wide(pool)), o)
    # the same rows one at a time, in another order: the same bits
    perm = torch.randperm(N * K, generator=U.gen(K)).tolist()
    o1 = attend(q[perm], pool, [slot[i] for i in perm], [pos[i] for i in perm], rpg=1)
    assert same_bits(o[perm], o1)


@pytest.mark.parametrize("hd", [64, 128])
def test_attention_long_rows_alone_and_among_many(hd):
    """More splits than one warp joins (64), in calls of few and of very many rows."""
    n = 18001
    pool = U.Pool([n, 300], 1, hd, 256, seed=15)
    q = U.bf16(U.gen(16), 1300, 2, hd)
    slot, pos = [0, 1, 0, 0], [n - 1, 299, 16384, 16383]
    o = attend(q[:4], pool, slot, pos)
    assert B.biv_device_error() == 0
    within(o, *U.attention(q[:4], pool.rows, slot, pos))
    many = attend(q, pool, slot + [1] * 1296, pos + [r % 300 for r in range(1296)])
    assert same_bits(many[:4], o)
    table = pool.table.clone()
    table[0, 70] = -1                                      # page 70 starts at key 17920
    bad = attend(q[:4], pool, slot, pos, table=table)
    assert B.biv_device_error() == 2
    assert bool((bad[0] == 0).all()) and same_bits(bad[1:], o[1:])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hd,G,K", [(128, 4, 5), (64, 4, 5), (128, 8, 4), (64, 2, 40)])
def test_attention_windows_over_pages(page, hd, G, K):
    """Windows of every page size end inside a page, a round of 64 keys and a split."""
    lengths = [K, 66, 259, 530, 1000]
    pool = U.Pool(lengths, 2, hd, page, seed=page + K)
    N, Hq = len(lengths), 2 * G
    q = U.bf16(U.gen(14), N * K, Hq, hd)
    slot = [r for r in range(N) for _ in range(K)]
    pos = [n - K + j for n in lengths for j in range(K)]
    pos[0] = -1                                            # an empty seat within a window
    o = attend(q, pool, slot, pos, rpg=K)
    assert B.biv_device_error() == 0
    within(o, *U.attention(q, pool.rows, slot, pos))
    assert same_bits(attend(q, pool, slot, pos, rpg=K, table=wide(pool)), o)
    assert same_bits(attend(q, pool, slot, pos, rpg=1), o)
    assert same_bits(attend(q[:-2], pool, slot[:-2], pos[:-2], rpg=K, table=wide(pool)), o[:-2])     # a last window that is not full
    assert same_bits(attend(q[:-2], pool, slot[:-2], pos[:-2], rpg=K), o[:-2])
    # twice the requests: clusters of four where eight do not fit one round
    assert same_bits(attend(torch.cat([q, q]), pool, slot + slot, pos + pos, rpg=K), torch.cat([o, o]))
    assert B.biv_device_error() == 0


def test_attention_does_not_depend_on_batch_pages_or_workspace():
    lengths, Hq, Hkv, hd = [900, 33, 511, 2000], 8, 2, 128
    q = U.bf16(U.gen(3), 4, Hq, hd)
    base = None
    for page in (16, 32, 64, 128, 256):
        pool = U.Pool(lengths, Hkv, hd, page, seed=5, fill=BIG if page == 64 else float("inf"))
        # the same keys in other pages: the pools draw them from the same seed after the order
        if base is not None:
            for r, (k, v) in enumerate(base_rows):
                for i in range(-(-lengths[r] // page)):
                    m = min(page, lengths[r] - i * page)
                    pool.k[pool.table[r, i], :, :m] = k[:, i * page:i * page + m]
                    pool.v[pool.table[r, i], :, :m] = v[:, i * page:i * page + m]
        o = attend(q, pool, range(4), [n - 1 for n in lengths], ws_fill=page % 251)
        if base is None:
            base, base_rows = o, pool.rows
        assert same_bits(o, base), page
        for r in range(4):
            alone = attend(q[r:r + 1], pool, [r], [lengths[r] - 1])
            assert same_bits(alone[0], base[r])
        wide = torch.cat([pool.table, torch.full((4, 40), -1, dtype=torch.int32)], 1)
        assert same_bits(attend(q, pool, range(4), [n - 1 for n in lengths], table=wide), base)


def test_attention_more_rows_than_the_tables_hold():
    """Thousands of single rows, and one prompt's rows as a single group (their first
    ones see one key, their last ones all)."""
    Hq, Hkv, hd, page = 4, 2, 64, 16
    W = 2600
    lengths = [1 + (37 * r) % 90 for r in range(W)]
    pool = U.Pool(lengths, Hkv, hd, page, seed=6)
    q = U.bf16(U.gen(7), W, Hq, hd)
    pos = [n - 1 for n in lengths]
    o = attend(q, pool, range(W), pos)
    some = list(range(0, W, 131))
    within(o[some], *U.attention(q[some], pool.rows, some, [pos[r] for r in some]))
    assert same_bits(attend(q[some], pool, some, [pos[r] for r in some]), o[some])
    pool = U.Pool([W], Hkv, hd, page, seed=8)
    pos, slot = list(range(W)), [0] * W
    o = attend(q, pool, slot, pos, rpg=W)
    some = [0, 1, 15, 16, 255, 256, 257, 1000, 2047, 2048, W - 1]
    within(o[some], *U.attention(q[some], pool.rows, [0] * len(some), some))
    assert same_bits(attend(q[some], pool, [0] * len(some), some), o[some])
    assert B.biv_device_error() == 0


def test_attention_widest_table():
    """A table for every position below 2^31: nothing but its width is large."""
    small = U.Pool([300], 1, 64, 16, seed=3)
    wide = (1 << 27) - 1
    table = torch.full((1, wide), -1, dtype=torch.int32, device="cuda")
    table[0, :small.table.shape[1]] = small.table[0].cuda()
    q = U.bf16(U.gen(2), 1, 1, 64)
    o = attend(q, small, [0], [299], table=table)
    assert B.biv_device_error() == 0 and same_bits(o, attend(q, small, [0], [299]))


def test_attention_shared_prefix_pages():
    """Two slots that name the same pages read the same keys."""
    pool = U.Pool([300, 300], 2, 128, 64, seed=1)
    table = pool.table.clone()
    table[1] = table[0]
    q = U.bf16(U.gen(2), 1, 8, 128).expand(2, 8, 128).contiguous()
    o = attend(q, pool, [0, 1], [299, 299], table=table)
    assert same_bits(o[0], o[1])


def test_attention_empty_rows_and_rows_out_of_range():
    lengths = [300, 40, 500]
    pool = U.Pool(lengths, 2, 128, 64, seed=4)
    q = U.bf16(U.gen(2), 6, 8, 128)
    slot, pos = [0, 1, -7, 2, 99, 0], [299, 39, -1, 499, -1, 10]
    o = attend(q, pool, slot, pos)
    assert B.biv_device_error() == 0                       # empty seats are no error, whatever slot they name
    within(o, *U.attention(q, pool.rows, slot, pos))
    assert bool((o[[2, 4]] == 0).all())
    cap = pool.table.shape[1] * 64
    for bad_slot, bad_pos, bits in ((3, 10, 2), (-1, 10, 2), (0, cap, 2), (0, -2, 2)):
        o2 = attend(q, pool, slot[:5] + [bad_slot], pos[:5] + [bad_pos])
        assert B.biv_device_error() == bits
        assert same_bits(o2[:5], o[:5]) and bool((o2[5] == 0).all())
    # a row of another slot in a group: zeros, the other rows as they were
    o3 = attend(q, pool, [0, 0, 1, 1, 2, 0], [299, 10, 39, 5, 499, 3], rpg=2)
    assert B.biv_device_error() == 4
    assert bool((o3[5] == 0).all())
    within(o3[:5], *U.attention(q[:5], pool.rows, [0, 0, 1, 1, 2], [299, 10, 39, 5, 499]))
    # a last group that is not full
    o4 = attend(q[:5], pool, [0, 0, 1, 1, 2], [299, 10, 39, 5, 499], rpg=2)
    assert B.biv_device_error() == 0 and same_bits(o4, o3[:5])


def test_attention_page_ids_out_of_range():
    lengths = [300, 700, 90]
    pool = U.Pool(lengths, 2, 128, 64, seed=4)
    q = U.bf16(U.gen(2), 3, 8, 128)
    pos = [n - 1 for n in lengths]
    good = attend(q, pool, range(3), pos)
    assert B.biv_device_error() == 0
    for row, entry, bad in ((0, 1, -1), (1, 10, pool.k.shape[0]), (1, 0, 1 << 30), (2, 0, -5)):
        table = pool.table.clone()
        table[row, entry] = bad
        o = attend(q, pool, range(3), pos, table=table)
        assert B.biv_device_error() == 2
        assert bool((o[row] == 0).all())
        keep = [r for r in range(3) if r != row]
        assert same_bits(o[keep], good[keep])


@pytest.mark.parametrize("path", ["one launch", "one launch, tiles", "direct", "staged"])
def test_attention_page_out_of_range_for_some_rows_of_a_window(path):
    """Rows that do not reach the bad page are computed, whatever page 0 holds."""
    G, K = (4, 5) if path in ("staged", "one launch, tiles") else (2, 4)
    pool = U.Pool([34], 1, 128, 16, seed=13)
    nan = torch.full_like(pool.k[:1], float("nan"))
    pool.k, pool.v, pool.table = torch.cat([nan, pool.k]), torch.cat([nan, pool.v]), pool.table + 1
    if path in ("direct", "staged"):
        pool.table = wide(pool)
    q = U.bf16(U.gen(2), K, G, 128)
    pos = [30, 31, 32, 33, 33][:K]
    table = pool.table.clone()
    table[0, 2] = -3
    o = attend(q, pool, [0] * K, pos, rpg=K, table=table)
    assert B.biv_device_error() == 2
    within(o[:2], *U.attention(q[:2], pool.rows, [0, 0], pos[:2]))
    assert bool((o[2:] == 0).all())


def test_attention_extreme_scores():
    """One key far above the others, far below, and scores of a thousand."""
    pool = U.Pool([600], 1, 128, 64, seed=8)
    k, v = pool.rows[0]
    q = U.bf16(U.gen(1), 3, 4, 128)
    for at, size in ((599, 40.0), (0, 40.0), (300, -300.0)):
        k[:, at] = (q[0, :1] * size).to(torch.bfloat16)
        page, off = int(pool.table[0, at // 64]), at % 64
        pool.k[page, :, off] = k[:, at]
    o = attend(q, pool, [0, 0, 0], [599, 598, 300])
    assert bool(o.isfinite().all())
    # the scores reach a thousand: fp32 leaves them 1e-4, which the tolerance has from the largest |q||k|
    within(o, *U.attention(q, pool.rows, [0, 0, 0], [599, 598, 300]))


@pytest.mark.parametrize("slope", [0.05, 0.4, 3.0, -0.4])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_scores_that_rise_or_fall(slope, hd):
    """Scores that grow from key to key by little (a row's reference stays behind its
    maximum for a while) or much (it moves on in every step), for some heads only."""
    lengths, Hq, Hkv, page, K = [700, 90], 4, 2, 32, 5
    pool = U.Pool(lengths, Hkv, hd, page, seed=11)
    for r, (k, v) in enumerate(pool.rows):
        # head 0 of every KV head's two: dim 0 of q is 4, of the keys the trend (in units of ln 2)
        k[:, :, 0] = (torch.arange(lengths[r]) * (slope * 0.6931 * hd ** 0.5 / 4)).to(torch.bfloat16)
        for i in range(-(-lengths[r] // page)):
            m = min(page, lengths[r] - i * page)
            pool.k[pool.table[r, i], :, :m] = k[:, i * page:i * page + m]
    q = U.bf16(U.gen(12), 2 * K, Hq, hd)
    q[:, :, 0] = torch.tensor([4.0, 0.0, 4.0, 0.0])
    slot = [r for r in range(2) for _ in range(K)]
    pos = [n - K + j for n in lengths for j in range(K)]
    o = attend(q, pool, slot, pos, rpg=K)
    assert B.biv_device_error() == 0
    within(o, *U.attention(q, pool.rows, slot, pos))
    assert same_bits(attend(q, pool, slot, pos, rpg=1), o)
    assert same_bits(attend(q, pool, slot, pos, rpg=K, table=wide(pool)), o)
    for w in (0, 3, 9):
        assert same_bits(attend(q[w:w + 1], pool, [slot[w]], [pos[w]])[0], o[w])


def test_attention_pool_past_two_gib_of_elements():
    """Pages whose offsets pass 32 bits."""
    page, Hkv, hd = 256, 8, 128
    n = (1 << 32) // (page * Hkv * hd * 2) + 3             # bytes past 2^32, elements past 2^31
    kp = torch.zeros(n * 2, Hkv, page, hd, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    small = U.Pool([400], Hkv, hd, page, seed=3)
    table = torch.tensor([[2 * n - 1, 2 * n - 2]], dtype=torch.int32)
    for i in range(2):
        kp[int(table[0, i])] = small.k[int(small.table[0, i])].cuda()
        vp[int(table[0, i])] = small.v[int(small.table[0, i])].cuda()
    q = U.bf16(U.gen(2), 1, 8, hd)
    assert same_bits(attend(q, small, [0], [399], k=kp, v=vp, table=table), attend(q, small, [0], [399]))
    window = U.bf16(U.gen(5), 5, 32, hd), small, [0] * 5, [395, 396, 397, 398, 399], 5
    assert same_bits(attend(*window, k=kp, v=vp, table=table), attend(*window))
    far = torch.cat([table, torch.full((1, 20), -1, dtype=torch.int32)], 1)
    assert same_bits(attend(*window, k=kp, v=vp, table=far), attend(*window))
    qkv = U.bf16(U.gen(4), 1, (8 + 2 * Hkv) * hd).cuda()
    q_out = nan_like(1, 8, hd)
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    B.biv_rope_kv_write_paged(qkv, q_out, kp, vp, table.cuda(), i32(0), i32(401), 1e4, 1)
    assert same_bits(vp[2 * n - 2, :, 401 - 256].cpu(), qkv.cpu().view(-1, hd)[8 + Hkv:])


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("Hq,Hkv,hd,page,K,N", [(8, 2, 128, 16, 1, 5), (4, 4, 64, 64, 3, 4), (6, 2, 256, 32, 1, 3),
                                                 (32, 8, 128, 128, 700, 1), (5, 1, 16, 256, 2, 2), (3, 3, 48, 16, 2, 3),
                                                 (7, 1, 80, 32, 4, 200)])
def test_rope_write(Hq, Hkv, hd, page, K, N):
    starts = [3 + 37 * r for r in range(N)]
    pool = U.Pool([s + K for s in starts], Hkv, hd, page, seed=K)
    W, theta = N * K, 500000.0
    qkv = U.bf16(U.gen(5), W, (Hq + 2 * Hkv) * hd)
    slot = torch.arange(N, dtype=torch.int32).repeat_interleave(K)
    pos = (torch.tensor(starts).repeat_interleave(K) + torch.arange(K).repeat(N)).int()
    kp, vp, q_out = pool.k.cuda(), pool.v.cuda(), nan_like(W, Hq, hd)
    keep = torch.tensor([max(0, K - r) for r in range(N)], dtype=torch.int32)
    B.biv_rope_kv_write_paged(qkv.cuda(), q_out, kp, vp, pool.table.cuda(), slot.cuda(), pos.cuda(), theta, K,
                              rows_keep=keep.cuda())
    assert B.biv_device_error() == 0
    x = qkv.view(W, Hq + 2 * Hkv, hd)
    turned = U.rope(x[:, :Hq + Hkv], pos, theta)
    # half a bf16 step, and fp32 sines, products and the sum: 2^-21 of the pair's length
    size = x[:, :Hq + Hkv].double().abs().amax()
    tol = U.HALF_STEP[torch.bfloat16] * turned.abs() + 2.0 ** -20 * size
    within(q_out, turned[:, :Hq], tol[:, :Hq], "q")
    written = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for w in range(W):
        if w % K >= int(keep[w // K]):
            continue
        p, off = int(pool.table[int(slot[w]), int(pos[w]) // page]), int(pos[w]) % page
        written[p, off] = True
        within(kp[p, :, off], turned[w, Hq:], tol[w, Hq:], "k")
        assert same_bits(vp[p, :, off].cpu(), x[w, Hq + Hkv:])
    # everything else as it was
    rest = ~written[:, None, :, None].expand(kp.shape)
    assert torch.equal(kp.cpu().view(torch.int16)[rest], pool.k.view(torch.int16)[rest])
    assert torch.equal(vp.cpu().view(torch.int16)[rest], pool.v.view(torch.int16)[rest])


def test_rope_write_far_positions_and_batch():
    """Angles of positions near 2^31 lose nothing, and a row does not depend on the batch."""
    Hq, Hkv, hd, page = 4, 2, 128, 256
    W = 700                                              # past the one-row-per-CTA launches
    cap = (1 << 31) - 256
    qkv = U.bf16(U.gen(5), W, (Hq + 2 * Hkv) * hd).cuda()
    pos = torch.randint(0, 1 << 20, (W,), generator=U.gen(6)).int()
    kp = torch.zeros(4, Hkv, page, hd, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, (1 << 20) // page, dtype=torch.int32, device="cuda")
    zero = torch.zeros(W, dtype=torch.int32, device="cuda")
    none = torch.zeros(W, dtype=torch.int32, device="cuda")
    run = lambda rows, p, K=1: (out := nan_like(len(rows), Hq, hd), B.biv_rope_kv_write_paged(  # noqa: E731
        qkv[rows].contiguous(), out, kp, kp.clone(), table, zero[rows], p[rows].cuda(), 1e4, K, rows_keep=none[rows]))[0]
    every = list(range(W))
    q = run(every, pos)
    x = qkv.cpu().view(W, -1, hd)[:, :Hq]
    ref = U.rope(x, pos, 1e4)
    within(q, ref, U.HALF_STEP[torch.bfloat16] * ref.abs() + 2.0 ** -20 * x.double().abs().amax())
    assert same_bits(run([5], pos), q[5:6]) and same_bits(run([699, 3], pos), q[[699, 3]])
    far = torch.full((W,), cap - 1, dtype=torch.int32)
    qf = run([0], far)                                   # q turns by any position; rows_keep 0 writes nothing
    within(qf, U.rope(x[:1], far[:1], 1e4), U.HALF_STEP[torch.bfloat16] * U.rope(x[:1], far[:1], 1e4).abs() + 2.0 ** -18 * x.double().abs().amax())
    assert B.biv_device_error() == 0 and bool((kp == 0).all())


def test_rope_write_seats_and_bad_indexes():
    Hq, Hkv, hd, page = 4, 2, 64, 16
    pool = U.Pool([20, 20], Hkv, hd, page, seed=1)
    W = 4
    qkv = U.bf16(U.gen(5), W, (Hq + 2 * Hkv) * hd).cuda()

    def run(slot, pos, table=None):
        kp, vp, q_out = pool.k.cuda(), pool.v.cuda(), nan_like(W, Hq, hd)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        B.biv_rope_kv_write_paged(qkv, q_out, kp, vp, (pool.table if table is None else table).cuda(), i32(slot),
                                  i32(pos), 1e4, 1)
        bits = B.biv_device_error()
        changed = (kp.cpu().view(torch.int16) != pool.k.view(torch.int16)).any(-1).any(1)
        return bits, changed, q_out

    bits, changed, q = run([0, 7, -3, 1], [2, -1, -1, 17])
    assert bits == 0 and int(changed.sum()) == 2 and bool(q[[0, 3]].isfinite().all())
    for slot, pos in ((2, 3), (-1, 3), (0, 32), (0, -2)):
        bits, changed, _ = run([0, slot, -3, 1], [2, pos, -1, 17])
        assert bits == 2 and int(changed.sum()) == 2
    table = pool.table.clone()
    table[1, 1] = pool.k.shape[0]
    bits, changed, _ = run([0, 7, -3, 1], [2, -1, -1, 17], table)
    assert bits == 2 and int(changed.sum()) == 1


# ------------------------------------------------------------------- GEMM
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (3, 1024, 2816), (64, 200, 64), (65, 72, 200), (128, 512, 128),
                                    (129, 520, 192), (300, 1000, 1024), (513, 64, 64)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_gemm_bias_act(M, N, K, act):
    g = U.gen(M + N)
    A, W = U.bf16(g, M, K), U.bf16(g, N, K, std=K ** -0.5)
    bias, res = U.bf16(g, N), U.bf16(g, M, N)
    s = A.double() @ W.double().T
    # fp32 accumulation in the tensor core: K partial sums, each within 2^-23 of sum |a b|
    acc = K * 2.0 ** -23 * (A.double().abs() @ W.double().abs().T)
    for b, r, dt in ((bias, res, torch.bfloat16), (None, res, torch.bfloat16), (bias, None, torch.float32),
                     (None, None, torch.bfloat16), (bias, res, torch.float32)):
        C = nan_like(M, N, dtype=dt)
        B.biv_gemm_bias_act(A.cuda(), W.cuda(), C, bias=None if b is None else b.cuda(),
                            residual=None if r is None else r.cuda(), act=act)
        x = s if b is None else s + b.double()
        ref = U.act(x, act)
        if r is not None:
            ref = ref + r.double()
        # the activations' slopes stay below 1.13; their own fp32 arithmetic within 2^-20 of |x| + 1
        tol = 1.13 * acc + U.HALF_STEP[dt] * ref.abs() + 2.0 ** -20 * (x.abs() + 1 + (0 if r is None else r.double().abs()))
        within(C, ref, tol, f"{act} {b is not None} {r is not None}")
    assert B.biv_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(7, 1024, 1024), (64, 4096, 512), (300, 512, 256), (48, 2056, 8192), (65, 2048, 6400),
                                    (127, 9728, 4096), (128, 4104, 2976), (300, 264, 2000), (700, 512, 4096)])
def test_gemm_bias_act_bits(M, N, K):
    """No bias, activation or residual, bf16: the plain GEMM's bits; in place over the
    residual the same as apart; a row does not depend on M, in either type."""
    g = U.gen(M)
    A, W = U.bf16(g, M, K).cuda(), U.bf16(g, N, K, std=0.05).cuda()
    bias, res = U.bf16(g, N).cuda(), U.bf16(g, M, N).cuda()
    a, b = nan_like(M, N), nan_like(M, N)
    B.biv_gemm_bias_act(A, W, a)
    B.biv_gemm_nosplitk(A, W, b)
    assert same_bits(a, b)
    full = nan_like(M, N, dtype=torch.float32)
    B.biv_gemm_bias_act(A, W, full, bias=bias, residual=res)
    # fp32 sums: blocks of 768 terms cut in the tensor core (48 additions, 2^-23 each at
    # most), then at most K / 768 + 1 rounded additions
    s = A.double() @ W.double().T
    tol = (48 * 2.0 ** -23 + (K / 768 + 5) * 2.0 ** -24) * (A.double().abs() @ W.double().abs().T + bias.double().abs() + res.double().abs())
    within(full, (s + bias.double() + res.double()).cpu(), tol.cpu(), "fp32")
    apart, over = nan_like(M, N), res.clone()
    B.biv_gemm_bias_act(A, W, apart, bias=bias, residual=res, act="gelu")
    B.biv_gemm_bias_act(A, W, over, bias=bias, residual=over, act="gelu")
    assert same_bits(apart, over)
    for rows in ([0], list(range(M // 2)), [M - 1, 0]):
        few = nan_like(len(rows), N)
        B.biv_gemm_bias_act(A[rows].contiguous(), W, few, bias=bias, residual=res[rows].contiguous(), act="gelu")
        assert same_bits(few, apart[rows])
        few = nan_like(len(rows), N, dtype=torch.float32)
        B.biv_gemm_bias_act(A[rows].contiguous(), W, few, bias=bias, residual=res[rows].contiguous())
        assert same_bits(few, full[rows])


def test_gemm_bias_act_not_a_number():
    """A NaN stays in its row and column, through every activation."""
    for act in B.ACTS:
        A, W = torch.ones(5, 64, dtype=torch.bfloat16), torch.ones(64, 64, dtype=torch.bfloat16)
        A[2, 3] = float("nan")
        bias = torch.zeros(64, dtype=torch.bfloat16)
        bias[7] = float("nan")
        C = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
        B.biv_gemm_bias_act(A.cuda(), W.cuda(), C, bias=bias.cuda(), act=act)
        nan = C.isnan().cpu()
        want = torch.zeros(5, 64, dtype=torch.bool)
        want[2] = True
        want[:, 7] = True
        assert torch.equal(nan, want), act


# --------------------------------------------------- streams and graphs
def test_paged_step_in_a_graph():
    """Write and attention of a step captured once and replayed on new inputs,
    beside an eager call that uses a workspace of its own."""
    Hq, Hkv, hd, page, N = 8, 2, 128, 64, 3
    lengths = [300, 20, 1000]
    pool = U.Pool([n + 8 for n in lengths], Hkv, hd, page, seed=2, fill=0.0)
    kp, vp, table = pool.k.cuda(), pool.v.cuda(), pool.table.cuda()
    ke, ve = kp.clone(), vp.clone()
    slot = torch.arange(N, dtype=torch.int32, device="cuda")
    pos = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    qkv = U.bf16(U.gen(1), N, (Hq + 2 * Hkv) * hd).cuda()
    ws = lambda: torch.empty(B.biv_decode_attn_paged_workspace_size(N, Hq, hd, table.shape[1], page),  # noqa: E731
                             dtype=torch.uint8, device="cuda")
    w1, w2 = ws(), ws()
    q, o, qe, oe = (nan_like(N, Hq, hd) for _ in range(4))

    def step(q, o, k, v, w):
        B.biv_rope_kv_write_paged(qkv, q, k, v, table, slot, pos, 1e4, 1)
        B.biv_decode_attn_paged(q, k, v, table, slot, pos, o, 1, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, o, kp, vp, w1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q, o, kp, vp, w1)
    for i in range(4):
        qkv.copy_(U.bf16(U.gen(10 + i), *qkv.shape))
        graph.replay()
        step(qe, oe, ke, ve, w2)
        assert same_bits(o, oe) and same_bits(q, qe) and same_bits(kp, ke) and same_bits(vp, ve)
        pos += 1
    assert B.biv_device_error() == 0
