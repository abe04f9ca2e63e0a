"""Block starts out of order (moe_prefix_attention): recorded, and never more work
than the entry point allowed for, however the remaining blocks overlap."""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_prefix_attention import Batch

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _none_served(out, lse):
    return bool((out == 0).all()) and bool((lse == float("-inf")).all())


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
def test_other_requests_stay_right(causal):
    """Two bad requests in the middle, the others' blocks apart: those are right
    (test_prefix_attention.py's definition and tolerances)."""
    b = Batch(8, 2, 64, BF, 16, 70, [(4, 20), (2, 30), (0, 5), (3, 200)], seed=3)
    want, _ = b.run(causal)
    out, z, tol, tol_lse = b.exact(causal, 64 ** -0.5)
    assert b.start == [0, 4, 6, 6, 9]
    b.q_start = _i32([0, 4, -1, 6, 9])
    got, lse = b.run(causal)
    assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_STARTS)
    for t in (slice(0, 4), slice(6, 9)):
        assert bool(((got.double() - out).abs() <= tol)[t].all()) and bool(((lse.double() - z).abs() <= tol_lse)[t].all())
    b.q_start = _i32(b.start)
    again, _ = b.run(causal)
    assert torch.equal(again, want) and b.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [0, 9] * 40 + [0], [9, 0, 9, 0, 9]])
def test_overlapping_blocks_are_not_served(starts):
    B = len(starts) - 1
    b = Batch(8, 2, 64, BF, 16, 70, [(1, 20)] * min(B, 9) + [(0, 20)] * max(0, B - 9), seed=4, pad=(0, max(0, 9 - B)))
    assert b.q.shape[0] == 9
    b.q_start = _i32(starts)
    assert _none_served(*b.run(True))
    assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_STARTS)
    b.q_start = _i32(b.start)
    b.check(True)


@pytest.mark.gpu
def test_overlapping_blocks_past_the_counters():
    """65536 requests of which every other one claims all 16 tokens over 130944
    own keys: their units would pass 2^32."""
    T, B, Hq, Hkv, D, page = 16, 65536, 1024, 8, 64, 1024
    q = torch.ones((T, Hq, D), device="cuda", dtype=BF)
    k = torch.zeros((1, page, Hkv, D), device="cuda", dtype=BF)
    table = torch.zeros((B, 128), device="cuda", dtype=torch.int32)
    own = torch.full((B,), 1023 * 128, device="cuda", dtype=torch.int32)
    start = _i32([0, 16]).repeat(B // 2 + 1)[:B + 1].contiguous()
    ws = ops.Workspace(ops.prefix_attention_workspace_bytes(T, B, Hq, Hkv, D))
    lse = torch.zeros((T, Hq), device="cuda")
    for causal in (False, True):
        out = ops.prefix_attention(q, k, k, start, None, None, table, own, ws, causal=causal, lse=lse)
        assert _none_served(out, lse)
        assert ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_STARTS)
