"""moe_prefix_attention in f16 where one key leads very many others: what the
others weigh together must not fall through the bottom of the type.

Tolerance: test_prefix_attention.py's, with the f16 term of a probability's
absolute rounding taken where it is.  A probability p (the row's largest is 1)
is held as 2^7 p, whose spacing at the bottom is 2^-24, so it is off by at most
2^-25 / 2^7 = 2^-32:  e/2 |o| + (e/2 + 2 ds + N 2^-22 + 2^-20) sum w|v| +
N 2^-32 max|v| + 2^-25.  The values are 0 for the leading key, so that the
output is what the others weigh.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nats", [8.0, 16.0, 17.0, 17.4, 19.0])
@pytest.mark.parametrize("lead", ["first", "last"])
def test_one_key_ahead_of_many(lead, nats, dtype):
    # as many row tiles as fill the GPU, so that one CTA walks all keys against the leading one
    N, H, D, page, T = 131072 + 1, 8, 64, 1024, 9728
    pages = -(-N // page)
    k = torch.zeros((pages, page, H, D), device="cuda", dtype=dtype)
    v = torch.ones((pages, page, H, D), device="cuda", dtype=dtype)
    rows_k, rows_v = k.view(-1, H, D), v.view(-1, H, D)
    rows_k[:N, :, 0] = -nats / 8
    at = 0 if lead == "first" else N - 1
    rows_k[at, :, 0] = 0
    rows_v[:N, :, 1] *= 3
    rows_v[at] = 0
    q = torch.zeros((T, H, D), device="cuda", dtype=dtype)
    q[0::2, :, 0] = 8
    q[1::2, :, 0] = 4

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = ops.Workspace(ops.prefix_attention_workspace_bytes(T, 1, H, H, D))
    lse = torch.zeros((T, H), device="cuda")
    out = ops.prefix_attention(q, k, v, i32(0, T), torch.arange(pages, dtype=torch.int32, device="cuda"), i32(N), None,
                               None, ws, scale=1.0, lse=lse)
    assert ws.device_status() == (ops.MOE_OK, 0)
    # the heads and the tokens of one parity are alike
    s = q[:2, 0].double() @ rows_k[:N, 0].double().t()
    vals = rows_v[:N, 0].double()
    want = torch.softmax(s, -1) @ vals
    eps = torch.finfo(dtype).eps
    half, bottom = (2.0 ** -25, 2.0 ** -32) if dtype == torch.float16 else (0.0, 0.0)
    ds = (D + 4) * 2.0 ** -24 * s.abs().amax(-1, keepdim=True)
    tol = (eps / 2 * want.abs() + (eps / 2 + 2 * ds + N * 2.0 ** -22 + 2.0 ** -20) * want
           + N * bottom * vals.amax(0) + half)
    off = (out.double().unflatten(0, (-1, 2)) - want[:, None]).abs().amax((0, 2))
    assert bool((off <= tol).all()), f"off by up to {(off / tol).max().item():.2f} of the tolerance"
    exact = torch.logsumexp(s, -1)
    off = (lse.double().unflatten(0, (-1, 2)) - exact[:, None]).abs().amax((0, 2))
    assert bool((off <= ds[:, 0] + N * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * exact.abs()).all())
