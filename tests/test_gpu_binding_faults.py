"""Each fault of a tensor is named by its own status, and the binding of the small calls is the one that runs."""
import pytest
import torch

from invariant_verify_gb300 import abi as B
from test_gpu_binding import OUTPUTS, calls

pytestmark = pytest.mark.gpu

TYPE, SHAPE, DEVICE = 4, 2, 7


# arguments whose last dimension is theirs to choose (tables, rows of a wider matrix, the vocabulary)
OWN_WIDTH = {("biv_rope_kv_write_paged", 4), ("biv_decode_attn_paged", 3), ("biv_softmax", 0), ("biv_softmax", 1),
             ("biv_verify_sample", 0)}


def test_the_binding_is_loaded():
    B.lib()
    assert B._fast.__name__.endswith("_biv_torch") and B._fast.__file__.endswith(".so")


@pytest.mark.parametrize("fault", ["type", "shape", "stride", "device"])
@pytest.mark.parametrize("name", OUTPUTS)
def test_a_fault_has_its_status(name, fault):
    good = calls()[name]
    seen = 0
    for at, x in enumerate(good):
        if not isinstance(x, torch.Tensor) or (name == "biv_decode_attn_paged" and at == 8):
            continue                               # a workspace may have any type and shape
        if fault == "type":
            bad, status = x.to(torch.float64), TYPE
        elif fault == "device":
            bad, status = x.cpu(), DEVICE
        elif fault == "stride":
            bad, status = torch.zeros(*x.shape, 2, dtype=x.dtype, device="cuda")[..., 0], SHAPE
        else:
            bad, status = torch.zeros(*x.shape[:-1], x.shape[-1] + 1, dtype=x.dtype, device="cuda"), SHAPE
            if (name, at) in OWN_WIDTH:
                if name.endswith("paged"):
                    continue
                bad = x[:-1]                       # a row less than the others have
        args = list(good)
        args[at] = bad
        with pytest.raises(B.BivError) as e:
            getattr(B, name)(*args)
        assert e.value.status == status, (at, str(e.value))
        seen += 1
    assert seen >= 2
    torch.cuda.synchronize()
    assert B.biv_device_error() == 0
