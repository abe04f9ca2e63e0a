"""moe_qk_norm_rope beyond the rotated part of a head: an element there is
itself, times the norm's factor and weight if there is a norm, whatever its
neighbours hold.

Without a norm the bits are the input's (NaN apart).  With one, the expected
value is x * r * w with r = 1 / sqrt(mean(x^2) + eps): r = 0 where the row holds
an infinity, so finite elements are 0 there and infinite ones NaN.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _rows(T, H, D, dtype, rot):
    g = torch.Generator(device="cuda").manual_seed(D + rot)
    x = torch.randn((T, H, D), generator=g, device="cuda").to(dtype)
    # non-finite values and zeros of both signs among the unrotated elements of some rows, each next to and R/2 or
    # four places from finite ones
    x[0, :, rot:] = torch.tensor([0.0, -0.0], device="cuda").repeat((D - rot) // 2).to(dtype)
    x[1, :, rot + 1::8] = INF
    x[2, :, rot + 4::8] = -INF
    x[3, :, rot + 6::8] = NAN
    return x


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,rot", [(64, 32), (64, 16), (128, 64), (256, 96), (128, 0)])
def test_unrotated_elements(D, rot, dtype, interleaved):
    T, Hq, Hkv = 5, 3, 2
    q, k = _rows(T, Hq, D, dtype, rot), _rows(T, Hkv, D, dtype, rot)
    table = ops.rope_table(8, rot) if rot else None
    pos = torch.tensor([0, 1, 7, 3, 2], device="cuda", dtype=torch.int32) if rot else None
    ws = ops.Workspace(ops.STATUS_BYTES)
    # no norm: the input's bits
    q_out, k_out, _ = ops.qk_norm_rope(q, k, None, pos, table, ws, interleaved=interleaved)
    for got, x in ((q_out, q), (k_out, k)):
        got, x = got[..., rot:], x[..., rot:]
        nan = torch.isnan(x)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(_bits(got)[~nan], _bits(x)[~nan])
    # a norm: every element by itself
    w = torch.linspace(0.5, 2, D, device="cuda").to(dtype)
    q_out, k_out, _ = ops.qk_norm_rope(q, k, None, pos, table, ws, q_weight=w, k_weight=w, interleaved=interleaved)
    for got, x in ((q_out, q), (k_out, k)):
        f = x.double()
        want = (f / (f.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double())[..., rot:]
        got = got[..., rot:].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want)
        # one rounding on top of 24 fp32 steps, as in test_qk_norm_rope.py
        tol = (torch.finfo(dtype).eps / 2 + 24 * 2.0 ** -24) * want.abs() + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert bool(((got - want).abs() <= tol)[ok].all())
    assert ws.device_status() == (ops.MOE_OK, 0)
