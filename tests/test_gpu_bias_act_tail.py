"""Activations where they are small: relative errors over the whole range of x."""
import math

import pytest
import torch

import paged_util as U
from invariant_verify_gb300 import abi as B

pytestmark = pytest.mark.gpu


def exact(x, act):
    """The activation of a float in 64 bits, without cancellation."""
    if act == "gelu":
        return 0.5 * x * math.erfc(-x / math.sqrt(2))
    y = x if act == "silu" else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return x / (1 + math.exp(-y)) if y > -700 else 0.0


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [37, 64, 300])
def test_relative_error_of_an_activation(act, dtype, M):
    """One product a sum (A holds x, B a power of two), so that the activation's argument is
    exact: 16384 values from -12.5 to 12.5, and tiny and huge ones.

    Tolerance: half a step of C's type; the exponential's argument y (x^2 / 2, or the
    sigmoid's) passes three roundings and the exponential and the quotient two units of 2^-23
    each; what the polynomial of erfc and its evaluation add stays below 16 roundings:
    (24 + 4 |y|) 2^-24 of the value, and 2^-126 |x| where the exponential is below the
    smallest normal number."""
    N, K = 2048, 6400                              # M = 64: two CTAs share the row tile
    x = torch.linspace(-12.5, 12.5, 16384).to(torch.bfloat16).unique()
    x = torch.cat([x, torch.tensor([0.0, 2.0 ** -60, -2.0 ** -60, 1e4, -1e4, 3e38, -3e38], dtype=torch.bfloat16)])
    x = x.repeat(-(-M * 8 // len(x)))[:M * 8] if len(x) < M * 8 else x[torch.randperm(len(x), generator=U.gen(1))[:M * 8]]
    if M < 300:                                    # fewer values than there are: the tail first
        x[:M * 4] = torch.linspace(-12.5, -2.0, M * 4).to(torch.bfloat16)
    A, W = torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(N, K, dtype=torch.bfloat16)
    A[:, :8] = x.view(M, 8)
    W[torch.arange(N), torch.arange(N) % 8] = 1.0
    C = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    B.biv_gemm_bias_act(A.cuda(), W.cuda(), C, act=act)
    arg = x.view(M, 8).double()
    ref = torch.tensor([exact(v, act) for v in arg.view(-1).tolist()], dtype=torch.float64).view(M, 8)
    y = (arg ** 2 / 2 if act == "gelu" else arg.abs() if act == "silu" else 1.6 * (arg.abs() + 0.044715 * arg.abs() ** 3)).clamp(max=200)
    tol = ref.abs() * (U.HALF_STEP[dtype] + (24 + 4 * y) * 2.0 ** -24) + 2.0 ** -126 * arg.abs()
    err = (C.double().cpu().view(M, N // 8, 8) - ref[:, None]).abs()
    bad = (err > tol[:, None]).any(1)
    assert not bool(bad.any()), [(float(a), float(r), float(e)) for a, r, e in zip(arg[bad], ref[bad], err.amax(1)[bad])][:8]
    assert B.biv_device_error() == 0
