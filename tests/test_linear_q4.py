"""moe_q4_prepare and moe_linear_q4: refusals on the host (no GPU), and on the GPU every
output against the formula in 64 bits.

Tolerance, derived: with z = x W^T + b, e = eps of the type and W the weights as they are
(no rounding), a group's sum is a sum of g exact products in fp32 (tensor cores may
truncate: 2^-23 a step, relative to its sum of magnitudes), times its scale, added in fp32;
all together at most (K + 8) 2^-22 S with S = sum|x w| + |b|; the activations' slopes are
at most 1.13 and their own error below 2^-20 of |z|; the result is rounded once:
  e/2 |y| + (K + 8) 2^-22 S + 2^-19 |z| + 2^-22 |r| (+ 2^-25 in f16).
"""
import math

import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

BF, HF = torch.bfloat16, torch.float16
INVALID, UNSUPPORTED, WORKSPACE = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ refusals (no GPU)

def _call(**kw):
    a = dict(x=1 << 30, xs=256, M=4, K=256, w=2 << 30, wb=1 << 20, N=128, group=64, zeros=1, dtype=0, bias=None, act=0,
             res=None, rs=0, y=3 << 30, ys=128, ws=4 << 30, wsb=1 << 20)
    a.update(kw)
    return ops.lib().moe_linear_q4(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(group=0), INVALID),
    (dict(dtype=2), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(zeros=2), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(y=1 << 30), INVALID),
    (dict(y=2 << 30), INVALID), (dict(ys=120), INVALID), (dict(xs=248), INVALID), (dict(res=3 << 30, rs=256), INVALID),
    (dict(x=(1 << 30) + 8), INVALID), (dict(w=(2 << 30) + 8), INVALID), (dict(bias=(5 << 30) + 2), INVALID),
    (dict(res=5 << 30, rs=-128), INVALID), (dict(wb=16384), INVALID), (dict(bias=3 << 30), INVALID),
    (dict(K=288), UNSUPPORTED), (dict(N=100), UNSUPPORTED), (dict(group=16, K=256), UNSUPPORTED),
    (dict(group=256), UNSUPPORTED), (dict(xs=260), UNSUPPORTED), (dict(ys=132), UNSUPPORTED),
    (dict(res=5 << 30, rs=132), UNSUPPORTED), (dict(M=(1 << 20) + 1), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=(4 << 30) + 16), WORKSPACE), (dict(wsb=128), WORKSPACE), (dict(M=0, x=None, ws=None), ops.MOE_OK),
])
def test_refusals(change, status):
    assert _call(**change) == status


def _prepare(**kw):
    a = dict(codes=1 << 30, scales=2 << 30, zeros=3 << 30, N=128, K=256, group=64, out=4 << 30, bytes=1 << 20)
    a.update(kw)
    return ops.lib().moe_q4_prepare(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-8), INVALID), (dict(K=0), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(out=None), INVALID), (dict(codes=(1 << 30) + 8), INVALID), (dict(out=(4 << 30) + 8), INVALID),
    (dict(out=1 << 30), INVALID), (dict(out=3 << 30), INVALID), (dict(N=12), UNSUPPORTED), (dict(K=96), UNSUPPORTED),
    (dict(group=48), UNSUPPORTED), (dict(bytes=1024), WORKSPACE)])
def test_prepare_refusals(change, status):
    assert _prepare(**change) == status


def test_size_queries():
    bytes_of = ops.lib().moe_q4_weight_bytes
    assert bytes_of(128, 128, 128, 0) == 8192 + 256 and bytes_of(128, 128, 32, 1) == 8192 + 4 * 384
    assert bytes_of(136, 160, 32, 0) == 4 * bytes_of(128, 128, 32, 0)
    for bad in ((0, 128, 64, 0), (12, 128, 64, 0), (128, 100, 64, 0), (128, 128, 16, 0)):
        assert bytes_of(*bad) == 0
    assert ops.lib().moe_linear_q4_workspace_bytes(4, 128, 64) >= ops.STATUS_BYTES
    for bad in ((-1, 128, 64), (4, 100, 64), (4, 128, 60), (4, 0, 64)):
        assert ops.lib().moe_linear_q4_workspace_bytes(*bad) == 0


def test_arguments_that_are_wrong():
    w = ops.Q4Weight(torch.zeros(1, dtype=torch.uint8), 128, 64, 32, BF, False)
    x = torch.zeros((2, 64), dtype=BF)
    for call, error in ((lambda: ops.linear_q4(x, w, None), ValueError),
                        (lambda: ops.linear_q4(x.half(), w, None), TypeError),
                        (lambda: ops.linear_q4(x, torch.zeros((128, 64)), None), TypeError),
                        (lambda: ops.linear_q4(x, w, None, activation="tanh"), ValueError),
                        (lambda: ops.q4_prepare(x, x), TypeError),
                        (lambda: ops.q4_prepare(torch.zeros((8, 16), dtype=torch.uint8), x), ValueError)):
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------ values (GPU)

def _act(z, act):
    return {"none": lambda v: v, "silu": lambda v: v * torch.sigmoid(v),
            "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
            "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))),
            "relu": lambda v: v.clamp(min=0)}[act](z)


class Case:
    def __init__(self, M, K, N, group, dtype=BF, zeros=True, bias=False, act="none", residual=False, seed=0, strided=False):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(dtype)
        self.codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = (normal(N, K // group).float() * 0.02).to(dtype)  # of both signs
        self.zeros = torch.randint(0, 16, (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
        self.x = normal(M, K + 24)[:, 16:16 + K] if strided else normal(M, K)
        self.bias = normal(N) if bias else None
        self.residual = (normal(M, N + 8)[:, :N] if strided else normal(M, N)) if residual else None
        self.act, self.group, self.M, self.K, self.N = act, group, M, K, N
        self.w = ops.q4_prepare(self.codes, self.scales, self.zeros)
        self.ws = ops.Workspace(ops.linear_q4_workspace_bytes(M, N, K))
        self.strided = strided

    def run(self, **kw):
        y = kw.pop("y", None)
        if y is None:
            y = torch.full((self.M, self.N + (16 if self.strided else 0)), 7.0, device="cuda", dtype=self.x.dtype)[:, :self.N]
        out = ops.linear_q4(self.x, self.w, self.ws, bias=self.bias, activation=self.act, residual=self.residual, y=y, **kw)
        assert out is y
        return y

    def exact(self):
        w = torch.stack([self.codes & 15, self.codes >> 4], dim=-1).flatten(1).double()
        z = 8.0 if self.zeros is None else self.zeros.double().repeat_interleave(self.group, dim=1)
        w = (w - z) * self.scales.double().repeat_interleave(self.group, dim=1)
        x = self.x.double()
        v, S = x @ w.t(), x.abs() @ w.abs().t()
        if self.bias is not None:
            v, S = v + self.bias.double(), S + self.bias.double().abs()
        y = _act(v, self.act)
        r = 0 if self.residual is None else self.residual.double()
        y = y + r
        tol = (torch.finfo(self.x.dtype).eps / 2 * y.abs() + (self.K + 8) * 2.0 ** -22 * S + 2.0 ** -19 * v.abs()
               + (2.0 ** -25 if self.x.dtype == HF else 0))
        return y, tol + (2.0 ** -22 * r.abs() if self.residual is not None else 0)

    def check(self):
        got = self.run()
        assert self.ws.device_status() == (ops.MOE_OK, 0)
        y, tol = self.exact()
        off = (got.double() - y).abs()
        assert bool((off <= tol).all()), f"{(off > tol).sum().item()} of {off.numel()}, worst {off.max().item()}"
        return got


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,group,kw", [
    (1, 32, 8, 32, {}), (1, 128, 128, 128, {}), (1, 4096, 4096, 128, dict(residual=True)),
    (1, 4096, 512, 64, dict(dtype=HF, zeros=False)), (2, 160, 136, 32, dict(dtype=HF, bias=True)),
    (9, 4096, 1024, 128, dict(bias=True, act="silu", residual=True)), (16, 1024, 264, 64, {}),
    (17, 2080, 1000, 32, dict(dtype=HF, bias=True, act="gelu", residual=True)), (31, 256, 8, 64, dict(zeros=False)),
    (33, 512, 4096, 128, dict(act="gelu_tanh")), (48, 384, 1032, 128, dict(dtype=HF, act="relu")),
    (65, 640, 392, 128, dict(bias=True)), (72, 4096, 6144, 128, dict(bias=True)),
    (100, 1024, 2048, 32, dict(zeros=False, residual=True)), (128, 256, 20480, 64, {}), (129, 256, 512, 128, {}),
    (300, 1056, 1160, 32, dict(dtype=HF, bias=True, act="silu", residual=True)),
    (1000, 512, 3000, 64, dict(act="gelu", zeros=False)), (2048, 1024, 4096, 128, {}), (1, 32, 40000, 32, {}),
    (3, 40960, 128, 128, {})])
def test_against_formula(M, K, N, group, kw):
    Case(M, K, N, group, seed=M + K, **kw).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_code_zero_and_place(dtype, group):
    """A one in each input in turn reads the weights back: code and zero of every value,
    every place of a block."""
    K, N = 256, 16
    c = Case(K, K, N, group, dtype=dtype, seed=group)
    c.x = torch.eye(K, device="cuda", dtype=dtype)
    c.scales = torch.full_like(c.scales, 0.5)
    c.w = ops.q4_prepare(c.codes, c.scales, c.zeros)
    y, _ = c.exact()
    assert torch.equal(c.run().double(), y)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 40, 200])
def test_rows_that_lie_apart(M):
    c = Case(M, 512, 640, 64, bias=True, residual=True, seed=4, strided=True)
    got = c.check()
    assert got.stride(0) == 656
    whole = got.as_strided((M, 656), (656, 1))
    assert bool((whole[:, 640:] == 7).all())


@pytest.mark.gpu
def test_residual_in_place_and_padded_rows():
    c = Case(20, 256, 512, 128, residual=True, seed=5)
    y, tol = c.exact()
    got = ops.linear_q4(c.x, c.w, c.ws, residual=c.residual, y=c.residual)
    assert bool(((got.double() - y).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 72, 500])
def test_same_bits_again_other_stream_and_graph(M):
    c = Case(M, 2048, 1536, 128, bias=True, seed=6)
    want = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ops.linear_q4(c.x, c.w, c.ws, bias=c.bias, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    y = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(y=y)
    graph.replay()
    assert torch.equal(y, want)
    c.x.mul_(-2)
    direct = c.run()
    graph.replay()
    assert torch.equal(y, direct) and not torch.equal(direct, want)
    assert c.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_what_is_not_finite():
    """Infinities and NaN of an input reach their own row, of a scale their own column."""
    for M in (4, 200):
        c = Case(M, 256, 256, 64, seed=7)
        want = c.run()
        c.x[1, 3] = float("nan")
        c.x[2, 255] = float("inf")
        got = c.run()
        assert got[1].isnan().all() and not torch.isfinite(got[2]).any()
        keep = torch.tensor([i for i in range(M) if i not in (1, 2)], device="cuda")
        assert torch.equal(got[keep], want[keep])
        c.scales[5, 1] = float("nan")
        c.w = ops.q4_prepare(c.codes, c.scales, c.zeros)
        got = c.run()
        assert got[:, 5].isnan().all() and torch.isfinite(got[0, 6:]).all() and torch.isfinite(got[0, :5]).all()


@pytest.mark.gpu
def test_nothing_outside():
    """Outputs next to y, and bytes behind the prepared weights, stay as they were."""
    for M, N in ((5, 40), (130, 1000)):
        c = Case(M, 288, N, 32, bias=True, seed=8)
        big = torch.full((M + 2, N), 3.0, device="cuda", dtype=BF)
        c.run(y=big[1:-1])
        assert bool((big[0] == 3).all()) and bool((big[-1] == 3).all())
        y, tol = c.exact()
        assert bool(((big[1:-1].double() - y).abs() <= tol).all())


@pytest.mark.gpu
def test_wrong_tensors():
    c = Case(4, 256, 128, 64, bias=True, residual=True)
    with pytest.raises(ValueError, match="x: expected"):
        ops.linear_q4(c.x[:, :128], c.w, c.ws)
    with pytest.raises(ValueError, match="y"):
        ops.linear_q4(c.x, c.w, c.ws, y=torch.empty((4, 136), device="cuda", dtype=BF))
    with pytest.raises(ValueError, match="bias"):
        ops.linear_q4(c.x, c.w, c.ws, bias=c.bias[:64])
    with pytest.raises(TypeError, match="residual"):
        ops.linear_q4(c.x, c.w, c.ws, residual=c.residual.half())
    with pytest.raises(ops.MoeError):
        ops.linear_q4(c.x, c.w, ops.Workspace(256), y=c.x.as_strided((4, 128), (256, 1)))
    with pytest.raises(ValueError, match="scales"):
        ops.q4_prepare(c.codes, c.scales[:, :3].contiguous())
    empty = ops.linear_q4(c.x[:0], c.w, c.ws)
    assert empty.shape == (0, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 24, 25, 40])
@pytest.mark.parametrize("dtype,low,high,x", [(HF, 2.0 ** -24, 40, 256.0), (HF, 2.0 ** -14, 1, 1.0), (HF, 4096.0, 1, 2.0 ** -12),
                                              (BF, 2.0 ** -100, 1, 1.0), (BF, 2.0 ** 100, 1, 1.0)])
def test_scales_at_the_ends_of_the_range(M, dtype, low, high, x):
    """Subnormal, smallest and largest scales; the tolerance of the other tests (f16 outputs
    may be subnormal: half of 2^-24)."""
    c = Case(M, 256, 136, 32, dtype=dtype, seed=M)
    g = torch.Generator(device="cuda").manual_seed(7)
    odd = torch.randint(1, 1 + high, c.scales.shape, generator=g, device="cuda") if high > 1 else 1 - torch.rand(
        c.scales.shape, generator=g, device="cuda") * 0.49
    c.scales = (odd.float() * low * (1 - 2 * (torch.rand(c.scales.shape, generator=g, device="cuda") < 0.5).float())).to(dtype)
    c.x = (c.x.float() * x).to(dtype)
    c.w = ops.q4_prepare(c.codes, c.scales, c.zeros)
    assert bool((c.scales != 0).all())
    c.check()


@pytest.mark.gpu
def test_both_kernels_agree_on_integers():
    """Scales of 1 and whole inputs: every sum is exact, whatever kernel takes it."""
    c = Case(40, 512, 264, 64, dtype=BF, seed=1)
    c.scales, c.x = torch.ones_like(c.scales), c.x.mul(2).round().clamp(-3, 3)
    c.w = ops.q4_prepare(c.codes, c.scales, c.zeros)
    whole = c.check()
    want = c.exact()[0]
    assert torch.equal(whole, want.to(BF))
    for a in range(0, 40, 10):
        part = ops.linear_q4(c.x[a:a + 10], c.w, c.ws)
        assert torch.equal(part, whole[a:a + 10])


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(128, 8192, 4096), (72, 8192, 4096), (256, 4096, 10240)])
def test_same_bits_from_cold_memory(M, K, N):
    """Copies that land late and in any order, with rings of three stages and more: call behind
    call, with what lies in L2 replaced between some of them."""
    c = Case(M, K, N, 128, seed=M)
    want = c.check().clone()
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for turn in range(60):
        if turn % 3 == 0:
            other.fill_(turn)
        differ += (c.run() != want).sum()
    assert differ.item() == 0
    assert c.ws.device_status() == (ops.MOE_OK, 0)
