"""The groups that a verifier's forward takes (host only: refused before any kernel)."""
import pytest

from invariant_verify_gb300.paged import PagedVerifier


@pytest.mark.parametrize("group", [0, -5, 3, 7, 41, 80])
def test_groups_that_would_leave_rows_unwritten(group):
    """Rows behind the last whole group would be attended to without having been written."""
    ver = object.__new__(PagedVerifier)
    ver.W, ver.rows = 40, 5
    with pytest.raises(ValueError, match="40 rows"):
        ver.forward(group)
