"""moe_pages_resize: requests that need more pages in all than 32 bits count.  Those that the
free pages suffice for get theirs, the others are recorded and keep what they have.
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
def test_needs_past_32_bits():
    B, width, page, n_pages = 65536, 40000, 8, 100   # 2.6e9 pages wanted, a table of 10 GB
    def i32(shape, value):
        return torch.full(shape, value, dtype=torch.int32, device="cuda")
    refs, table, own = i32((n_pages,), 0), i32((B, width), -1), i32((B,), 0)
    pool = torch.zeros((n_pages, page, 8), dtype=torch.int16, device="cuda")
    ws = ops.Workspace(ops.pages_workspace_bytes(B, n_pages))
    new = i32((B,), width * page)
    new[0], new[1], new[2], new[B - 1] = 40, 0, 9 * page, 3
    ops.pages_resize(refs, table, own, new, page, ws, caches=[pool])
    assert ws.device_status() == (ops.MOE_ERR_DEVICE_POOL, ops.INFO_POOL)
    assert own[:4].tolist() == [40, 0, 72, 0] and not own[3:].any()
    assert table[0, :6].tolist() == [0, 1, 2, 3, 4, -1] and table[2, :10].tolist() == [*range(5, 14), -1]
    assert (table >= 0).sum().item() == 14 and refs.tolist() == [1] * 14 + [0] * 86
