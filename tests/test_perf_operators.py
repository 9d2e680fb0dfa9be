"""The measured cases' calls: each prepared state owns the workspace that its attention uses (host only)."""
import importlib.util
import os

import pytest
import torch

from invariant_verify_gb300 import abi as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def cases():
    spec = importlib.util.spec_from_file_location("measured_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_states_do_not_share_a_workspace(cases, monkeypatch):
    """Two of them may run on two streams, or be captured into two graphs."""
    used = []
    monkeypatch.setattr(B, "biv_decode_attn_paged_workspace_size", lambda W, Hq, hd, pages, page: 1000 * W)
    monkeypatch.setattr(B, "biv_decode_attn_paged", lambda *a: used.append((a[8].data_ptr(), a[8].numel())))
    monkeypatch.setattr(cases, "own", True)
    q, i = torch.zeros(2, 4, 64), torch.zeros(2, 3, dtype=torch.int32)
    states = [dict(q=q, o=q, k_pages=q[None], v_pages=q[None], page_table=i, row_slot=i, row_pos=i, case={"op": "attn", "K": 1})
              for _ in range(2)]
    for s in (0, 1, 1, 0):
        cases.run(states[s])
    assert all(n >= 2000 for _, n in used)
    assert used[0] == used[3] and used[1] == used[2] and used[0][0] != used[1][0]
