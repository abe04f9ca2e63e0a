"""moe_linear on values that are not finite: an activation passes on what its
formula gives, NaN above all, so that a fault upstream stays visible.

x has one non-zero column and w a single 1 in each row, so the product of a row
is its value exactly (0 * 0 elsewhere); every expected value is the activation's
own in 64 bits, and finite ones are compared as in test_linear.py: one rounding,
e/2, on top of 2^-19 of its argument for the activation's arithmetic.
"""
import math

import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _formula(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return torch.relu(z) if act == "relu" else z


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [6, 300])  # few rows' kernel, many rows'
@pytest.mark.parametrize("act", sorted(ops.ACTIVATIONS))
def test_activations_pass_on_what_is_not_finite(act, M, dtype):
    values = torch.tensor([NAN, INF, -INF, -2.0, 0.0, 3.0], dtype=torch.float64)
    z = values.repeat(-(-M // 6))[:M].cuda()
    N = 72
    x = torch.zeros((M, 64), device="cuda", dtype=dtype)
    w = torch.zeros((N, 64), device="cuda", dtype=dtype)
    bias = torch.zeros(N, device="cuda", dtype=dtype)
    # the values come through the bias's columns where a product would make inf * 0
    x[:, 5] = 1
    res = torch.zeros((M, N), device="cuda", dtype=dtype)
    ws = ops.Workspace(ops.STATUS_BYTES)
    for i, v in enumerate(values.tolist()):
        bias.fill_(v)
        y = ops.linear(x, w, ws, bias=bias, activation=act, residual=res).double()
        want = _formula(values[i], act).item()
        if math.isnan(want):
            assert bool(torch.isnan(y).all()), (act, v)
        elif math.isinf(want):
            assert bool((y == want).all()), (act, v)
        else:
            assert (y - want).abs().max() <= torch.finfo(dtype).eps / 2 * abs(want) + 2.0 ** -19 * abs(v), (act, v)
    # a NaN of the product itself: one row's x
    x[:, 5] = z.to(dtype).nan_to_num(0.0, 0.0, 0.0)
    x[0, 5] = NAN
    w[:, 5] = 1
    y = ops.linear(x, w, ws, activation=act)
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isfinite(y[1:]).all())
