"""Launches of one stream that overlap: a kernel may let the next one start
early only where that cannot read too soon what the stream's kernels write.

The fused forward (the slice schedule) loads its first expert weights before it
waits for its predecessor, so nothing that writes a tensor a caller may use as
weights signals its dependents before it is complete.
"""
import os
import re

import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300 import synthetic as S
from moe_ffn_speculative_gb300.build import CSRC, build


def test_who_signals_early():
    """The fused forward itself (it writes y alone), and the attention kernel,
    whose dependent is its own joining launch, which does not signal."""
    signals = {}
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            with open(os.path.join(CSRC, name)) as f:
                text = re.sub(r"//[^\n]*", "", f.read())
            n = len(re.findall(r"griddep_launch_dependents\(\)|griddepcontrol\.launch_dependents", text))
            if n:
                signals[name] = n
    assert signals == {"prefix_attention.cu": 1, "slice.cu": 1}


@pytest.fixture(scope="module")
def _library():
    build()
    ops.lib()
    ops.set_schedule(ops.SCHEDULE_SLICE)
    yield
    ops.set_schedule(ops.SCHEDULE_AUTO)


def _merge(base, up, down, ws, y):
    """y = base + up down^T, the rows of all experts in one product."""
    ops.linear(up, down, ws, residual=base, y=y)


@pytest.mark.gpu
@pytest.mark.parametrize("between", [False, True])
def test_weights_made_by_linear_then_the_fused_forward(between, _library):
    """An adapter merged into the experts' weights right before the forward that
    uses them, with another small product between them or not: the same bits as
    when everything before the forward has ended."""
    cfg = S.LayerConfig("adapters", T=9, H=2048, E=8, I=512, K=2, seed=11)
    d = S.make_inputs(cfg, "cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    rank = 64

    def normal(*shape, std=0.05):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()
    base = d["w_gate_up"].clone()
    rows = base.flatten(0, 1)
    adapters = [(normal(rows.shape[0], rank), normal(cfg.H, rank)) for _ in range(4)]
    layer = ops.MoELayer(d, ops.Recipe.from_config(cfg), cfg.T)
    ws = ops.Workspace(ops.STATUS_BYTES)
    target = d["w_gate_up"].flatten(0, 1)
    small, scratch = normal(9, cfg.H, std=1.0), torch.empty((9, rows.shape[0]), device="cuda", dtype=torch.bfloat16)
    x = d["x"]

    def step(i, wait):
        _merge(rows, *adapters[i], ws, target)
        if between:
            ops.linear(small, rows, ws, y=scratch)
        if wait:
            torch.cuda.synchronize()
        return layer.forward(x).clone()
    want = [step(i, True) for i in range(4)]
    assert not torch.equal(want[0], want[1])
    for turn in range(25):
        for i in range(4):
            assert torch.equal(step(i, False), want[i]), (turn, i)
    assert layer.ws.device_status() == ws.device_status() == (ops.MOE_OK, 0)
