"""moe_prefix_attention_kv4: blocks of few and of many rows in turn.  The rows of a softmax
group are 8 or 16 by the block, so that neighbouring blocks give a row to different groups,
of which one may be ahead by a block: nothing that it sets up may reach what another has
still to write.  Many blocks of each CTA, from the definition and repeated from cold memory.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_prefix_attention import BF, HF
from test_prefix_attention_kv4 import Batch4


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype,causal", [(128, BF, True), (64, HF, False)])
@pytest.mark.parametrize("short,long", [(3, 9), (8, 12), (2, 16)])
def test_rows_that_change_their_group(D, dtype, causal, short, long):
    """Four heads a key head: 8 to 32 rows, then 36 to 64, one to three tiles of keys each."""
    blocks = [((short, long)[i % 2], 16 + 37 * i % 340) for i in range(240)]
    b = Batch4(16, 4, D, dtype, 16, 70, blocks, seed=short)
    b.check(causal)
    want = [t.clone() for t in b.run(causal)]
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for turn in range(60):
        if turn % 3 == 0:
            other.fill_(turn)
        for got, w in zip(b.run(causal), want):
            differ += (got != w).sum()
    assert differ.item() == 0
    assert b.ws.device_status() == (ops.MOE_OK, 0)
