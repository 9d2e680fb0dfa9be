"""The Python binding of the small calls: the same results whichever way a call goes
(its own checks of the tensors, or abi.py's), faults that are named, the caller's stream."""
import threading

import pytest
import torch

import paged_util as U
from gpu_util import same_bits
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


def calls(seed=0):
    """name -> (function, arguments, indexes of the outputs)."""
    g = U.gen(seed)
    W, Hq, Hkv, hd, page = 3, 4, 2, 64, 16
    f = lambda *shape: torch.rand(*shape, generator=g).cuda()  # noqa: E731
    b = lambda *shape: U.bf16(g, *shape).cuda()  # noqa: E731
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = b(9, Hkv, page, hd), b(9, Hkv, page, hd)
    table, slot, pos = i([[0, 1, 2], [3, 4, 5], [6, 7, 8]]), i([0, 1, 2]), i([5, 40, 17])
    ws = torch.empty(B.biv_decode_attn_paged_workspace_size(W, Hq, hd, 3, page), dtype=torch.uint8, device="cuda")
    p = f(4, 100)
    return {
        "biv_rope_kv_write_paged": [b(W, (Hq + 2 * Hkv) * hd), torch.zeros(W, Hq, hd, dtype=torch.bfloat16, device="cuda"), k.clone(),
                                    v.clone(), table, slot, pos, 1e4, 1],
        "biv_decode_attn_paged": [b(W, Hq, hd), k, v, table, slot, pos, torch.zeros(W, Hq, hd, dtype=torch.bfloat16, device="cuda"), 1, ws],
        "biv_gemm_bias_act": [b(5, 64), b(72, 64), torch.zeros(5, 72, device="cuda"), b(72), b(5, 72), "gelu"],
        "biv_softmax": [f(4, 100), torch.zeros(4, 100, device="cuda"), 0.5],
        "biv_verify_sample": [p / p.sum(1, keepdim=True), None, i([[3], [4]]), f(2, 1), f(2), i([7, 8]),
                              torch.zeros(2, 2, dtype=torch.int32, device="cuda"), i([0, 0]), i([0, 0])],
    }


OUTPUTS = {"biv_rope_kv_write_paged": (1, 2, 3), "biv_decode_attn_paged": (6,), "biv_gemm_bias_act": (2,), "biv_softmax": (1,),
           "biv_verify_sample": (6, 7, 8)}


def run(name, args, **kw):
    torch.cuda.synchronize()                               # the arguments were filled on the current stream
    getattr(B, name)(*args, **kw)
    torch.cuda.synchronize()
    assert B.biv_device_error() == 0
    return [args[i].clone() for i in OUTPUTS[name]]


def same(a, b):
    return all(same_bits(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", OUTPUTS)
def test_both_ways_agree(name):
    direct = run(name, calls()[name])
    assert any(bool((x != 0).any()) for x in direct)
    # a stream that is named goes through abi.py's own checks and call
    assert same(direct, run(name, calls()[name], stream=torch.cuda.current_stream()))
    side = torch.cuda.Stream()
    assert same(direct, run(name, calls()[name], stream=side.cuda_stream))
    # the current stream of a side stream's context, and of another thread
    args = calls()[name]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        getattr(B, name)(*args)
    side.synchronize()
    assert same(direct, [args[i] for i in OUTPUTS[name]])
    got = []
    t = threading.Thread(target=lambda: got.append(run(name, calls()[name])))
    t.start()
    t.join()
    assert same(direct, got[0])


@pytest.mark.parametrize("name", OUTPUTS)
def test_faults_are_named(name):
    """Each tensor in turn of another type, shape, stride or device."""
    good = calls()[name]
    for at, x in enumerate(good):
        if not isinstance(x, torch.Tensor) or x is good[-1] and name == "biv_decode_attn_paged":
            continue
        wide = torch.zeros(*x.shape, 2, dtype=x.dtype, device="cuda")[..., 0]
        for bad, status in ((x.to(torch.float64), 4), (x[..., :-1], 2), (wide, 2), (x.cpu(), 7)):
            if name == "biv_gemm_bias_act" and at in (0, 1) and bad.shape != x.shape:
                bad = x[..., :-8].contiguous()             # another K than the other operand's
            if name == "biv_softmax" and bad.shape != x.shape and at == 0:
                continue                                   # fewer columns of a wider matrix are allowed
            if name == "biv_verify_sample" and at == 0 and bad.shape != x.shape:
                bad = x[:-1]
            args = list(good)
            args[at] = bad
            if bad is wide and (x.numel() < 2 or x.shape == (1,)):
                continue
            with pytest.raises((B.BivError, ValueError)) as e:
                getattr(B, name)(*args)
            assert not isinstance(e.value, B.BivError) or e.value.status in (status, 2, 4), (at, e.value)
    torch.cuda.synchronize()
    assert B.biv_device_error() == 0


def test_arguments_the_binding_leaves_to_the_other_way():
    args = calls()["biv_rope_kv_write_paged"]
    B.biv_rope_kv_write_paged(*args, rows_keep=torch.ones(3, dtype=torch.int32, device="cuda"))
    assert same([args[i] for i in (1, 2, 3)], run("biv_rope_kv_write_paged", calls()["biv_rope_kv_write_paged"]))
    args = calls()["biv_rope_kv_write_paged"]
    args[7] = 10000                                        # an integer theta
    assert same([args[1]], run("biv_rope_kv_write_paged", args)[:1])
    x = torch.rand(3, 40, device="cuda")
    p = torch.zeros(3, 40, device="cuda")
    B.biv_softmax(x, p, 1)
    q = torch.zeros(3, 40, device="cuda")
    B.biv_softmax(x, q, 1.0)
    assert same_bits(p, q)
    B.biv_softmax(torch.zeros(0, 40, device="cuda"), torch.zeros(0, 40, device="cuda"), 1.0)
    with pytest.raises(B.BivError):
        B.biv_softmax(x, p, -1.0)
    with pytest.raises(B.BivError):
        B.biv_gemm_bias_act(*calls()["biv_gemm_bias_act"][:5], act="tanh")
    with pytest.raises((B.BivError, TypeError, AttributeError)):
        B.biv_verify_sample(*[None] * 9)
