"""One workspace for the attention and the MoE FFN, call after call: the fixed
header, which the FFN's kernels count in, is whole, and every result has the bits
that it has from workspaces of its own."""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300 import synthetic as S
from moe_ffn_speculative_gb300.build import build
from test_prefix_attention import Batch


def _up(n):
    return (n + 255) // 256 * 256


# the status block; the router's counters of 4-token blocks of up to 65536 tokens and one more; the fused kernel's parity
# word and two sets of 4 + 512 + 17 x 128 counters (csrc/moe_internal.cuh)
HEADER = 256 + _up(4 * (65536 // 4 + 1)) + _up(4 * (1 + 2 * (4 + 512 + 17 * 128)))


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [(0, 0), (2, 3)])
def test_header_is_left_alone(pad):
    b = Batch(8, 2, 128, torch.bfloat16, 64, 500, [(4, 100), (4, 30)], seed=10, pad=pad)
    b.run(True)
    b.ws.buf.zero_()
    # where there is no counter at zero, a word of its own
    b.ws.buf[256:HEADER] = (torch.arange(HEADER - 256, device="cuda") % 251).to(torch.uint8)
    b.check(True)
    assert bool((b.ws.buf[:256] == 0).all())
    assert torch.equal(b.ws.buf[256:HEADER], (torch.arange(HEADER - 256, device="cuda") % 251).to(torch.uint8))
    assert bool((b.ws.buf[HEADER:] != 0).any())


@pytest.mark.gpu
def test_attention_and_both_schedules_of_the_ffn():
    cfg = S.LayerConfig("shared", T=24, H=1024, E=8, I=512, K=2, seed=21)
    d = S.make_inputs(cfg, "cuda")
    recipe = ops.Recipe.from_config(cfg)
    batches = [Batch(8, 2, 64, torch.bfloat16, 16, P, blocks, seed=s)
               for s, (P, blocks) in enumerate([(300, [(5, 40), (9, 9)]), (0, [(1, 700)] * 12), (64, [(24, 24)])])]
    ffn_bytes = max(ops.ffn_workspace_bytes(cfg.T, cfg.H, cfg.I, 0, recipe), HEADER)

    def forward(ws, schedule):
        ops.set_schedule(schedule)
        try:
            return ops.moe_ffn_forward(d["x"], d["gate"], d["w_gate_up"], d["w_down"], recipe, ws)
        finally:
            ops.set_schedule(ops.SCHEDULE_AUTO)
    want_ffn = {s: forward(ops.Workspace(ffn_bytes), s) for s in (ops.SCHEDULE_SLICE, ops.SCHEDULE_STREAM_K)}
    want = [b.run(True) for b in batches]
    shared = ops.Workspace(max([ffn_bytes] + [b.ws.nbytes for b in batches]))
    for b in batches:
        b.ws = shared
    for turn in range(3):
        for schedule in (ops.SCHEDULE_SLICE, ops.SCHEDULE_STREAM_K, ops.SCHEDULE_SLICE):
            for b, (out, lse) in zip(batches, want):
                got, z = b.run(True)
                assert torch.equal(got, out) and torch.equal(z, lse), turn
                assert torch.equal(forward(shared, schedule), want_ffn[schedule]), (turn, schedule)
    assert shared.device_status() == (ops.MOE_OK, 0)
