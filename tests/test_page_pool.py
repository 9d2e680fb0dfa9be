"""The page pool's bookkeeping (host only)."""
import pytest

from invariant_verify_gb300.paged import PagePool


def pool():
    return PagePool(n_pages=10, page_size=16, layers=2, Hkv=1, hd=16, n_slots=3, max_pages=6, device="cpu")


def test_reserve_and_release():
    p = pool()
    p.reserve(0, 1)
    p.reserve(1, 33)
    p.reserve(0, 16)
    assert [len(x) for x in p.pages] == [1, 3, 0] and len(p.free) == 6
    held = p.pages[0] + p.pages[1]
    assert len(set(held)) == 4 and not set(held) & set(p.free)
    for s in range(3):
        assert p.table[s].tolist() == p.pages[s] + [-1] * (6 - len(p.pages[s]))
    p.reserve(0, 17)
    assert p.pages[0][0] == held[0] and len(p.pages[0]) == 2      # a request keeps the pages it has
    p.release(1)
    assert p.table[1].tolist() == [-1] * 6 and len(p.free) == 8
    p.reserve(0, 3)                                                # shorter: nothing changes
    assert len(p.pages[0]) == 2


def test_refusals_change_nothing():
    p = pool()
    p.reserve(0, 96)
    with pytest.raises(ValueError, match="table holds 6"):
        p.reserve(0, 97)
    with pytest.raises(ValueError, match="4 free"):
        p.reserve(1, 80)
    assert [len(x) for x in p.pages] == [6, 0, 0] and len(p.free) == 4
    assert p.table[1].tolist() == [-1] * 6
