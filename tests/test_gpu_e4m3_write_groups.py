"""Groups of the write into a cache held in e4m3 whose first row has no position."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,bits", [(-1, B.DEVERR_GROUP), (-5, B.DEVERR_GROUP | B.DEVERR_INDEX)])
@pytest.mark.parametrize("K", [2, 17, 40, 64])
def test_rows_behind_a_first_row_without_a_position(gpu, K, first, bits):
    """Such rows raise the group's bit and nothing of them is written, whatever they count on from; a group that is as it
    should be, in the same call, is written."""
    B.biv_device_error()
    Hq, Hkv, hd, page, tail, wide = 4, 2, 64, 16, 96, 8
    n = 2 * wide + 1
    nan = float("nan")
    pools = [*[torch.full((n, Hkv, page, hd), nan, device="cuda").to(E.E4M3) for _ in "kv"],
             *[torch.full((n, Hkv, 1), nan, dtype=torch.bfloat16, device="cuda") for _ in "kv"],
             *[torch.full((2, Hkv, tail, hd), nan, dtype=torch.bfloat16, device="cuda") for _ in "kv"]]
    table = torch.arange(1, n, dtype=torch.int32, device="cuda").view(2, wide)
    qkv = U.bf16(U.gen(K), 2 * K, (Hq + 2 * Hkv) * hd).cuda()
    q = torch.empty(2 * K, Hq, hd, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([0] * K + [1] * K, dtype=torch.int32, device="cuda")
    pos = torch.tensor([first + j for j in range(K)] + list(range(K)), dtype=torch.int32, device="cuda")
    B.biv_rope_kv_write_paged_e4m3(qkv, q, *pools, table, slot, pos, 1e4, K)
    got = B.biv_device_error()
    assert got == (bits if K > -first else B.DEVERR_INDEX)
    mine = table[0].long()
    for t in pools[:4]:
        assert t[mine].float().isnan().all()                # no page, no scale of the first group's slot
    assert all(t[0].isnan().all() for t in pools[4:])
    assert all(t[1, :, :K].isfinite().all() and t[1, :, K:].isnan().all() for t in pools[4:])
    full = K // page
    for t in pools[:4]:
        assert t[table[1, :full].long()].float().isfinite().all() and t[table[1, full:].long()].float().isnan().all()
