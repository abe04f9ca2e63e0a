"""The attention side's calls on a stream of their own: a buffer that a call makes
is not memory that the current stream's pending work still reads, and outlives
what the current stream does with it."""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _linear():
    x, w, ws = torch.ones((64, 64), device="cuda", dtype=BF), torch.ones((4096, 64), device="cuda", dtype=BF), ops.Workspace(256)
    return lambda stream: [ops.linear(x, w, ws, stream=stream)]


def _attention():
    q, k = torch.ones((64, 64, 64), device="cuda", dtype=BF), torch.ones((1, 64, 8, 64), device="cuda", dtype=BF)
    ws = ops.Workspace(ops.prefix_attention_workspace_bytes(64, 1, 64, 8, 64))
    start, pages, n = _i32(0, 64), _i32(0), _i32(64)
    return lambda stream: [ops.prefix_attention(q, k, k, start, pages, n, None, None, ws, stream=stream)]


def _rope():
    q, ws = torch.ones((64, 64, 64), device="cuda", dtype=BF), ops.Workspace(256)
    return lambda stream: list(ops.qk_norm_rope(q, q, q, None, None, ws, stream=stream))


@pytest.mark.gpu
@pytest.mark.parametrize("make", [_linear, _attention, _rope])
def test_made_buffers(make):
    call, stream = make(), torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    size = want[0].shape
    assert want[0].numel() == 64 * 4096
    kept = [torch.empty(size, device="cuda", dtype=BF) for _ in want]
    torch.cuda.synchronize()
    for turn in range(3):
        # blocks of the outputs' size that the current stream still reads, a while from now, are given back
        held = [torch.full(size, 7.0 + i, device="cuda", dtype=BF) for i in range(len(want))]
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        for a, b in zip(kept, held):
            a.copy_(b)
        where = {t.data_ptr() for t in held}
        del held, b
        made = call(stream)
        assert not where & {t.data_ptr() for t in made}
        stream.synchronize()
        torch.cuda.synchronize()
        for i, t in enumerate(kept):
            assert bool((t == 7.0 + i).all()), (turn, i)
        # read on the current stream, a while from now, then dropped: the next call on the stream leaves them alone
        torch.cuda._sleep(50_000_000)
        for a, b in zip(kept, made):
            a.copy_(b)
        where = {t.data_ptr() for t in made}
        del made, b
        again = call(stream)
        assert not where & {t.data_ptr() for t in again}
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
