"""A page id out of range in a window over a cache held in e4m3: what page 0, read in its place, holds and is scaled by
reaches no row."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("cap", [160, 10240])               # a call of one launch, one of two
@pytest.mark.parametrize("K,Hq", [(3, 2), (3, 8), (12, 8)])  # one head a KV head: a tile of eight query rows has rows of both kinds
def test_rows_that_end_before_the_page(gpu, K, Hq, cap, junk, hd):
    """Rows up to 143 do not reach the block at 128 in the pages; those from 144 on do, and come back as zeros."""
    B.biv_device_error()
    pool = E.HeldPool([67, 160], 2, hd, 16, seed=1, cap=cap, tail=32)
    assert not (pool.table == 0).any()                      # page 0 is nobody's
    for s in pool.scales:
        s[0] = junk
    pool.table[1, 8] = -1
    first = [64 - K, 145 - K if K == 3 else 140]
    q = U.bf16(U.gen(7), 2 * K, Hq, hd, std=1.5)
    slot, pos = [0] * K + [1] * K, [p + j for p in first for j in range(K)]
    o = torch.full((2 * K, Hq, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.biv_decode_attn_paged_workspace_size(2 * K, Hq, hd, pool.table.shape[1], 16), dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B.biv_decode_attn_paged_e4m3(q.cuda(), *pool.on(), i32(slot), i32(pos), o, K, ws)
    assert B.biv_device_error() == B.DEVERR_INDEX
    want, tol = E.attention(q, pool, slot, pos)
    gone = [slot[w] == 1 and pos[w] >= 144 for w in range(2 * K)]
    assert any(gone) and not all(gone[K:])
    for w in range(2 * K):
        if gone[w]:
            assert (o[w] == 0).all(), pos[w]
        else:
            assert ((o[w].cpu().double() - want[w]).abs() <= tol[w]).all(), (slot[w], pos[w])
