"""moe_linear: refusals on the host (no GPU), and on the GPU every output
against the formula in 64 bits.

Tolerance, derived: with z = x W^T + b and e = eps of the type, the product is
a sum of K exact products in fp32 (tensor cores may truncate: 2^-23 a step,
relative to S = sum|x w| + |b|), the activations' slopes are at most 1.13 and
their own error below 2^-20 of |z|, and the result is rounded once:
  e/2 |y| + (K + 4) 2^-22 S + 2^-19 |z| + 2^-22 |r| (+ 2^-25 in f16).
"""
import math

import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ refusals (no GPU)

def _call(**kw):
    a = dict(x=1 << 20, xs=64, M=4, K=64, w=2 << 20, N=128, dtype=0, bias=None, act=0, res=None, rs=0, y=3 << 20,
             ys=128, ws=4 << 20, wb=1 << 40)
    a.update(kw)
    return ops.lib().moe_linear(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), ops.MOE_ERR_INVALID_ARG), (dict(N=0), ops.MOE_ERR_INVALID_ARG), (dict(K=0), ops.MOE_ERR_INVALID_ARG),
    (dict(dtype=2), ops.MOE_ERR_INVALID_ARG), (dict(act=5), ops.MOE_ERR_INVALID_ARG),
    (dict(act=-1), ops.MOE_ERR_INVALID_ARG), (dict(x=None), ops.MOE_ERR_INVALID_ARG),
    (dict(w=None), ops.MOE_ERR_INVALID_ARG), (dict(y=None), ops.MOE_ERR_INVALID_ARG),
    (dict(y=1 << 20), ops.MOE_ERR_INVALID_ARG), (dict(y=2 << 20), ops.MOE_ERR_INVALID_ARG),
    (dict(ys=120), ops.MOE_ERR_INVALID_ARG), (dict(xs=56), ops.MOE_ERR_INVALID_ARG),
    (dict(res=3 << 20, rs=256), ops.MOE_ERR_INVALID_ARG), (dict(x=(1 << 20) + 8), ops.MOE_ERR_INVALID_ARG),
    (dict(bias=(5 << 20) + 2), ops.MOE_ERR_INVALID_ARG), (dict(res=5 << 20, rs=-128), ops.MOE_ERR_INVALID_ARG),
    (dict(K=60), ops.MOE_ERR_UNSUPPORTED), (dict(N=100), ops.MOE_ERR_UNSUPPORTED),
    (dict(xs=68), ops.MOE_ERR_UNSUPPORTED), (dict(ys=132), ops.MOE_ERR_UNSUPPORTED),
    (dict(res=5 << 20, rs=132), ops.MOE_ERR_UNSUPPORTED), (dict(M=(1 << 20) + 1), ops.MOE_ERR_UNSUPPORTED),
    (dict(ws=None), ops.MOE_ERR_WORKSPACE), (dict(ws=(4 << 20) + 16), ops.MOE_ERR_WORKSPACE),
    (dict(wb=128), ops.MOE_ERR_WORKSPACE), (dict(M=0, x=None, ws=None), ops.MOE_OK),
])
def test_refusals(change, status):
    assert _call(**change) == status


def test_workspace_query():
    assert ops.lib().moe_linear_workspace_bytes(4, 128, 64) >= ops.STATUS_BYTES
    for bad in ((-1, 128, 64), (4, 100, 64), (4, 128, 60), (4, 0, 64)):
        assert ops.lib().moe_linear_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ values (GPU)

def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z.clamp(min=0) if act == "relu" else z


def _check(x, w, bias, act, residual, y):
    K, e = x.shape[1], torch.finfo(x.dtype).eps
    z = x.double() @ w.double().t()
    S = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, S = z + bias.double(), S + bias.double().abs()
    want = _act(z, act)
    tol = (K + 4) * 2.0 ** -22 * S + 2.0 ** -19 * z.abs() + (2.0 ** -25 if x.dtype == HF else 0)
    if residual is not None:
        want = want + residual.double()
        tol = tol + 2.0 ** -22 * residual.double().abs()
    tol = tol + e / 2 * want.abs()
    off = (y.double() - want).abs()
    assert bool((off <= tol).all()), f"{(off > tol).sum().item()} outputs off by up to {(off / tol).max().item()} tol"
    # one rounding: uniform, at most e/2 relative, e/sqrt(12) in the 2-norm
    assert (y.double() - want).norm() <= 0.36 * e * want.norm() + 1e-30


def _inputs(M, K, N, dtype, bias, residual, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + K + N)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    return (normal(M, K), normal(N, K, std=K ** -0.5), normal(N) if bias else None,
            normal(M, N) if residual else None)


CASES = [
    # M, K, N, dtype, bias, activation, residual
    (1, 8, 8, BF, False, "none", False),
    (1, 4096, 4096, BF, False, "none", True),
    (9, 4096, 1024, BF, True, "silu", True),
    (16, 64, 128, HF, True, "relu", False),
    (17, 72, 136, HF, True, "gelu", True),
    (72, 4096, 6144, BF, True, "none", False),
    (72, 2056, 1000, HF, False, "gelu_tanh", True),
    (129, 512, 1000, BF, True, "gelu", True),
    (255, 1000, 264, HF, True, "silu", False),
    (256, 128, 128, BF, False, "relu", True),
    (257, 256, 384, BF, True, "gelu_tanh", True),
    (300, 4104, 520, HF, True, "none", True),
    (513, 192, 2048, BF, False, "none", True),
    (1001, 2056, 5000, HF, True, "silu", True),
    (1024, 1024, 4096, BF, True, "gelu", False),
    (2047, 520, 776, BF, True, "none", True),
    (5, 32768, 256, BF, False, "none", False),
    (40, 128, 40000, HF, True, "none", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,dtype,bias,act,residual", CASES)
def test_against_formula(M, K, N, dtype, bias, act, residual):
    x, w, b, r = _inputs(M, K, N, dtype, bias, residual)
    ws = ops.Workspace(ops.linear_workspace_bytes(M, N, K))
    y = ops.linear(x, w, ws, bias=b, activation=act, residual=r)
    assert ws.device_status() == (ops.MOE_OK, 0)
    _check(x, w, b, act, r, y)
    assert torch.equal(ops.linear(x, w, ws, bias=b, activation=act, residual=r), y)  # the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("M", [7, 200, 700])
def test_strided_rows_in_place_and_guards(M):
    """Rows that lie apart; the residual updated in place; nothing outside the
    rows of y is written."""
    K, N = 264, 392
    x, w, b, r = _inputs(M, K + 24, N, BF, True, True, seed=3)
    x, w = x[:, 16:16 + K], w[:, :K].contiguous()
    full = torch.full((M + 2, N + 64), 7.0, device="cuda", dtype=BF)
    y = full[1:M + 1, 8:8 + N]
    y.copy_(r)
    ws = ops.Workspace(ops.linear_workspace_bytes(M, N, K))
    out = ops.linear(x, w, ws, bias=b, residual=y, y=y)
    assert out is y
    _check(x, w, b, "none", r, y)
    edge = full.clone()
    edge[1:M + 1, 8:8 + N] = 7.0
    assert bool((edge == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [9, 600])
def test_stream_and_graph(M):
    x, w, b, r = _inputs(M, 512, 768, HF, True, True, seed=5)
    ws = ops.Workspace(ops.linear_workspace_bytes(M, 768, 512))
    want = ops.linear(x, w, ws, bias=b, activation="silu", residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(want)
    ops.linear(x, w, ws, bias=b, activation="silu", residual=r, y=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = ops.linear(x, w, ws, bias=b, activation="silu", residual=r, y=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 400])
def test_chain_waits_for_its_input(M):
    """Back to back on one stream, each call reading the last one's output as
    its rows, its residual or its weights."""
    n = 512
    x, w, _, _ = _inputs(M, n, n, BF, False, False, seed=6)
    ws = ops.Workspace(ops.linear_workspace_bytes(max(M, n), n, n))
    a = ops.linear(x, w, ws)
    b = ops.linear(a, w, ws, residual=a)
    w2 = ops.linear(w, w, ws)
    c = ops.linear(b, w2, ws)
    torch.cuda.synchronize()
    _check(x, w, None, "none", None, a)
    _check(a, w, None, "none", a, b)
    _check(w, w, None, "none", None, w2)
    _check(b, w2, None, "none", None, c)


@pytest.mark.gpu
def test_tails_of_the_activations():
    """Large logits both ways: no overflow, no cancellation."""
    z = torch.tensor([-300.0, -40.0, -9.0, -3.0, -1e-3, 0.0, 1e-3, 3.0, 9.0, 40.0, 300.0, 1e4], device="cuda")
    M = z.numel()
    x = torch.zeros((M, 64), device="cuda", dtype=BF)
    x[:, 0] = z.to(BF)
    w = torch.zeros((8, 64), device="cuda", dtype=BF)
    w[:, 0] = 1
    ws = ops.Workspace(ops.STATUS_BYTES)
    for act in ops.ACTIVATIONS:
        y = ops.linear(x, w, ws, activation=act)
        assert bool(torch.isfinite(y).all())
        _check(x, w, None, act, None, y)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [19456, 12288, 8192, 6144, 264])
@pytest.mark.parametrize("M", [33, 48, 49, 64, 65, 80, 81, 96, 97, 112, 113, 128, 129])
def test_between_the_two_kernels(M, N):
    """On both sides of the number of rows at which the kernel changes, with
    the many rows' tiles less than half full."""
    K = 264
    x, w, b, r = _inputs(M, K, N, BF, True, True, seed=M)
    ws = ops.Workspace(ops.linear_workspace_bytes(M, N, K))
    y = ops.linear(x, w, ws, bias=b, activation="relu", residual=r)
    assert ws.device_status() == (ops.MOE_OK, 0)
    _check(x, w, b, "relu", r, y)
