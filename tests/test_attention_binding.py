"""The attention side's Python calls: what the extension does not take it answers
with None, and the call then says what is wrong, before anything runs."""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def test_extension_answers_none_to_what_it_does_not_know():
    b = ops._binding()
    t = torch.zeros((2, 4, 64), dtype=torch.bfloat16)  # not on a GPU
    for f, n in ((b.qk_norm_rope, 16), (b.prefix_attention, 15), (b.linear, 9)):
        assert f() is None
        assert f(*[None] * n) is None
        assert f(*["x"] * n) is None
        assert f(*[t] * n) is None
        assert f(*[1.5] * n) is None


def test_calls_say_what_is_wrong_without_a_gpu():
    t = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.linear(t, t, None)
    with pytest.raises(ValueError):
        ops.linear(t, t, None, activation="tanh")
    with pytest.raises(ValueError):
        ops.prefix_attention(t.view(2, 1, 64), None, None, None, None, None, None, None, None)


def _rope(**kw):
    a = dict(q=torch.zeros((3, 4, 64)), k=torch.zeros((3, 2, 64)), v=torch.zeros((3, 2, 64)),
             k_cache=torch.zeros((2, 8, 2, 64)), v_cache=torch.zeros((2, 8, 2, 64)))
    a = {n: t.to("cuda", torch.bfloat16) for n, t in a.items()}
    a.update(positions=torch.zeros(3, dtype=torch.int32, device="cuda"), rope=ops.rope_table(8, 64),
             ws=ops.Workspace(256), slots=torch.arange(3, dtype=torch.int32, device="cuda"))
    a.update(kw)
    return ops.qk_norm_rope(**a)


def _attn(**kw):
    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    cache = torch.zeros((4, 8, 2, 64), device="cuda", dtype=torch.bfloat16)
    a = dict(q=torch.zeros((3, 4, 64), device="cuda", dtype=torch.bfloat16), k_cache=cache, v_cache=cache.clone(),
             q_start=i32(0, 1, 3), prefix_pages=i32(0), prefix_len=i32(4), page_table=i32(1, 2).view(2, 1),
             own_len=i32(3, 2), ws=ops.Workspace(ops.prefix_attention_workspace_bytes(3, 2, 4, 2, 64)))
    a.update(kw)
    return ops.prefix_attention(**a)


def _linear(**kw):
    a = dict(x=torch.zeros((3, 64), device="cuda", dtype=torch.float16),
             w=torch.zeros((16, 64), device="cuda", dtype=torch.float16), ws=ops.Workspace(256))
    a.update(kw)
    return ops.linear(**a)


def _cuda(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, device="cuda", dtype=dtype)


@pytest.mark.gpu
def test_good_calls_pass():
    _rope()
    _attn()
    _linear()
    torch.cuda.synchronize()


BAD = [
    # call, what is changed, the exception
    (_rope, lambda: dict(q=_cuda(3, 4, 64, dtype=torch.float32)), TypeError),
    (_rope, lambda: dict(k=_cuda(3, 2, 64, dtype=torch.float16)), TypeError),
    (_rope, lambda: dict(k=_cuda(2, 2, 64)), ValueError),
    (_rope, lambda: dict(v=_cuda(3, 1, 64)), ValueError),
    (_rope, lambda: dict(q=_cuda(3, 64, 4).transpose(1, 2)), ValueError),
    (_rope, lambda: dict(positions=_cuda(3, dtype=torch.int64)), TypeError),
    (_rope, lambda: dict(positions=_cuda(2, dtype=torch.int32)), ValueError),
    (_rope, lambda: dict(slots=torch.zeros(3, dtype=torch.int32)), ValueError),
    (_rope, lambda: dict(k_cache=_cuda(2, 8, 64, 2)), ValueError),
    (_rope, lambda: dict(v_cache=_cuda(1, 8, 2, 64)), ValueError),
    (_rope, lambda: dict(q_out=_cuda(3, 4, 128)), ValueError),
    (_rope, lambda: dict(q_weight=_cuda(32)), ValueError),
    (_rope, lambda: dict(rope=_cuda(8, 64)), TypeError),
    (_rope, lambda: dict(positions=None), ops.MoeError),
    (_rope, lambda: dict(ws=ops.Workspace(0)), ops.MoeError),
    (_attn, lambda: dict(k_cache=_cuda(4, 8, 2, 64, dtype=torch.float16)), TypeError),
    (_attn, lambda: dict(v_cache=_cuda(3, 8, 2, 64)), ValueError),
    (_attn, lambda: dict(page_table=_cuda(3, 1, dtype=torch.int32)), ValueError),
    (_attn, lambda: dict(own_len=_cuda(2, dtype=torch.int64)), TypeError),
    (_attn, lambda: dict(prefix_len=None), ValueError),
    (_attn, lambda: dict(out=_cuda(3, 4, 128)), ValueError),
    (_attn, lambda: dict(lse=_cuda(3, 4)), TypeError),
    (_attn, lambda: dict(scale=0.0), ops.MoeError),
    (_attn, lambda: dict(ws=ops.Workspace(4096)), ops.MoeError),
    (_linear, lambda: dict(w=_cuda(16, 32, dtype=torch.float16)), ValueError),
    (_linear, lambda: dict(w=_cuda(16, 64)), TypeError),
    (_linear, lambda: dict(bias=_cuda(8, dtype=torch.float16)), ValueError),
    (_linear, lambda: dict(residual=_cuda(3, 8, dtype=torch.float16)), ValueError),
    (_linear, lambda: dict(y=_cuda(16, 3, dtype=torch.float16).t()), ValueError),
    (_linear, lambda: dict(activation="swish"), ValueError),
    (_linear, lambda: dict(w=_cuda(12, 64, dtype=torch.float16)), ops.MoeError),
]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    call, change, error = BAD[i]
    with pytest.raises(error):
        call(**change())
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_buffers_are_made_where_none_are_given():
    x = _cuda(3, 64, dtype=torch.float16) + 1
    w = _cuda(16, 64, dtype=torch.float16) + 0.5
    assert torch.equal(ops.linear(x, w, ops.Workspace(256)), torch.full((3, 16), 32.0, device="cuda").half())
    q_out, k_out, v_out = _rope(q=_cuda(3, 4, 64) + 1, k_cache=None, v_cache=None, slots=None, rope=None, positions=None)
    assert bool((q_out == 1).all()) and k_out.shape == v_out.shape == (3, 2, 64)
    with pytest.raises(ValueError):
        _rope(k_cache=None)
