"""Groups of the write into a cache held in e4m3 that name one slot, of which at most one writes."""
import pytest
import torch

import e4m3_util as E
import paged_util as U
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots,first", [([7, 7], [0, 0]), ([-3, -3], [0, 16]), ([1, 1], [16, 64]), ([1, 1], [2 ** 31 - 5, 16])])
def test_groups_at_fault_write_no_slot(gpu, slots, first):
    """Slots and positions out of range raise the index bit, not the group's: nobody else's rows are at stake."""
    B.biv_device_error()
    K, Hq, Hkv, hd, page = 4, 2, 1, 64, 16
    pools = [*[torch.zeros(9, Hkv, page, hd, dtype=torch.uint8, device="cuda").view(E.E4M3) for _ in "kv"],
             *[torch.zeros(9, Hkv, 1, dtype=torch.bfloat16, device="cuda") for _ in "kv"],
             *[torch.zeros(2, Hkv, 32, hd, dtype=torch.bfloat16, device="cuda") for _ in "kv"]]
    table = torch.arange(1, 9, dtype=torch.int32, device="cuda").view(2, 4)      # positions below 64
    qkv = U.bf16(U.gen(1), 2 * K, (Hq + 2 * Hkv) * hd).cuda()
    q = torch.empty(2 * K, Hq, hd, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([s for s in slots for _ in range(K)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([p + j for p in first for j in range(K)], dtype=torch.int32, device="cuda")
    B.biv_rope_kv_write_paged_e4m3(qkv, q, *pools, table, slot, pos, 1e4, K)
    assert B.biv_device_error() == B.DEVERR_INDEX
    good = [i for i in range(2) if slots[i] == 1 and first[i] == 16]
    for t, at in zip(pools[4:], (Hq + Hkv - 1, Hq + Hkv)):
        rows = t[1, 0, 16:16 + K]
        assert (rows != 0).any() == bool(good)
        if good and at == Hq + Hkv:
            assert torch.equal(rows, qkv[good[0] * K:good[0] * K + K].view(K, -1, hd)[:, at])
