"""The 4-bit operators' calls on a stream of their own, on the current device, and
without a GPU: a buffer that a call makes is not memory that the current stream's
pending work still reads, tensors of another device are refused, and what the
extension does not take it answers with None."""
import pytest
import torch

import test_attention_streams
from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_attention_device import _Nothing

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _linear():
    w = ops.q4_prepare(torch.full((4096, 32), 0x9a, dtype=torch.uint8, device="cuda"), torch.ones((4096, 1), device="cuda", dtype=BF))
    x, ws = torch.ones((64, 64), device="cuda", dtype=BF), ops.Workspace(ops.linear_q4_workspace_bytes(64, 4096, 64))
    return lambda stream, **kw: [ops.linear_q4(x, w, ws, stream=stream, **kw)]


def _few():
    w = ops.q4_prepare(torch.full((32768, 32), 0x9a, dtype=torch.uint8, device="cuda"), torch.ones((32768, 1), device="cuda", dtype=BF))
    x, ws = torch.ones((8, 64), device="cuda", dtype=BF), ops.Workspace(ops.linear_q4_workspace_bytes(8, 32768, 64))
    return lambda stream, **kw: [ops.linear_q4(x, w, ws, stream=stream, **kw)]


def _cache(pages, page, heads, D):
    cache, ws = torch.zeros(ops.kv4_shape(pages, page, heads, D), dtype=torch.uint8, device="cuda"), ops.Workspace(256)
    k = torch.linspace(-3, 3, pages * page * heads * D, device="cuda").to(BF).view(-1, heads, D)
    return ops.kv4_write(k, k, None, cache, ws)


def _read():
    cache, ws = _cache(8, 64, 8, 64), ops.Workspace(256)
    return lambda stream, **kw: list(ops.kv4_read(cache, 64, ws, stream=stream, **kw))


def _attention():
    cache, q = _cache(1, 64, 8, 64), torch.ones((64, 64, 64), device="cuda", dtype=BF)
    ws = ops.Workspace(ops.prefix_attention_kv4_workspace_bytes(64, 1, 64, 8, 64))
    start, pages, n = _i32(0, 64), _i32(0), _i32(64)
    return lambda stream, **kw: [ops.prefix_attention_kv4(q, cache, start, pages, n, None, None, ws, stream=stream, **kw)]


@pytest.mark.gpu
@pytest.mark.parametrize("make", [_linear, _few, _read, _attention])
def test_made_buffers(make):
    test_attention_streams.test_made_buffers(make)


def _write():
    cache, ws, k = _cache(1, 64, 8, 64), ops.Workspace(256), torch.ones((4, 8, 64), device="cuda", dtype=BF)
    return lambda stream, **kw: [ops.kv4_write(k, k, None, cache, ws, stream=stream, **kw)]


def _pages(name):
    refs, table, n = _i32(1, 0, 0, 0), _i32(0, -1, -1, -1).view(2, 2), _i32(5, 0)
    ws, cache = ops.Workspace(ops.pages_workspace_bytes(2, 4)), _cache(4, 16, 2, 64)
    state = (refs, table, n)
    calls = {"resize": lambda stream: ops.pages_resize(*state, _i32(9, 0), 16, ws, [cache], stream=stream),
             "fork": lambda stream: ops.pages_fork(*state, _i32(0), _i32(1), 16, ws, [cache], stream=stream),
             "compact": lambda stream: ops.pages_compact(table, _i32(0, 0), _i32(1, 2, -1, -1).view(2, 2), 16, ws, [cache],
                                                         new_len=_i32(0, 0), stream=stream)}
    return calls[name]


CALLS = {"linear_q4": _linear, "kv4_write": _write, "kv4_read": _read, "prefix_attention_kv4": _attention,
         "pages_resize": lambda: _pages("resize"), "pages_fork": lambda: _pages("fork"),
         "pages_compact": lambda: _pages("compact")}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_the_current_device(name, monkeypatch):
    """Takes the call on the tensors' own device; refuses it where that is another (one
    GPU stands in for two, as for the 16-bit calls)."""
    call, answers, real, stream = CALLS[name](), [], ops._binding(), torch.cuda.current_stream()
    given = {"linear_q4": lambda: dict(y=torch.empty((64, 4096), device="cuda", dtype=BF)),
             "kv4_read": lambda: {n: torch.empty((8, 64, 8, 64), device="cuda", dtype=BF) for n in "kv"},
             "prefix_attention_kv4": lambda: dict(out=torch.empty((64, 64, 64), device="cuda", dtype=BF))}.get(name, dict)()

    class Listen:
        def __getattr__(self, f):
            def g(*a):
                answers.append(getattr(real, f)(*a))
                return answers[-1]
            return g
    with monkeypatch.context() as m:
        m.setattr(ops, "_binding", Listen)
        call(stream, **given)
    torch.cuda.synchronize()
    assert answers == [0]
    with monkeypatch.context() as m:
        m.setattr(ops, "_binding", _Nothing)
        m.setattr(torch.cuda, "current_device", lambda: 1)
        with pytest.raises(ValueError, match="current CUDA device"):
            call(stream, **given)


def test_extension_answers_none_to_what_it_does_not_know():
    b = ops._binding()
    t = torch.zeros((2, 4, 64), dtype=BF)  # not on a GPU
    for f in (b.linear_q4, b.kv4_write, b.kv4_read, b.prefix_attention_kv4, b.pages_resize, b.pages_fork, b.pages_compact):
        assert f() is None
        for n in range(5, 18):
            for x in (None, "x", t, 1.5, (), (t,), [t]):
                assert f(*[x] * n) is None


@pytest.mark.gpu
def test_two_at_once():
    """Calls of all kinds on two streams at a time, each with a workspace of its own, give
    the bits that they give one after the other."""
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)
    w = ops.q4_prepare(torch.randint(0, 256, (1024, 512), generator=g, device="cuda", dtype=torch.uint8),
                       normal(1024, 8) * 0.02)
    cache = _cache(24, 64, 2, 64)
    starts = {n: torch.arange(5, dtype=torch.int32, device="cuda") * n for n in (1, 9)}
    prefix, prefix_len = torch.arange(12, dtype=torch.int32, device="cuda"), _i32(700)
    table, own = torch.arange(12, 24, dtype=torch.int32, device="cuda").view(4, 3), _i32(20, 64, 130, 9)
    x = {n: normal(4 * n, 1024) for n in (1, 9)}

    def lane():
        spaces = [ops.Workspace(n) for n in (ops.linear_q4_workspace_bytes(36, 1024, 1024),
                                             ops.prefix_attention_kv4_workspace_bytes(36, 4, 16, 2, 64), 256)]

        def call(n, stream=None):
            y = ops.linear_q4(x[n], w, spaces[0], activation="silu", stream=stream)
            o = ops.prefix_attention_kv4(y.view(4 * n, 16, 64), cache, starts[n], prefix, prefix_len, table, own, spaces[1],
                                         stream=stream)
            k, v = ops.kv4_read(cache, 64, spaces[2], pages=prefix, stream=stream)
            return y, o, k, v
        return call, spaces
    lanes, streams = [lane(), lane()], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = {n: lanes[0][0](n) for n in (1, 9)}
    torch.cuda.synchronize()
    got = []
    for turn in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                n = (1, 9)[(turn + i) % 2]
                got.append((n, lanes[i][0](n)))
    torch.cuda.synchronize()
    for n, outs in got:
        for a, b in zip(outs, want[n]):
            assert torch.equal(a, b)
    for _, spaces in lanes:
        for ws in spaces:
            assert ws.device_status() == (ops.MOE_OK, 0)
