"""The attention side's calls launch on the current device: tensors of another one
are refused.  (One GPU stands in for two: the checks that say what is wrong are
told that the current device is another, and the extension's answer to that, None,
is given for it.  On the device where they are, the extension takes the calls.)"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_attention_binding import _attn, _linear, _rope

NAMES = ("qk_norm_rope", "prefix_attention", "linear")


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


class _Nothing:
    """An extension that takes no call."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.mark.gpu
@pytest.mark.parametrize("call", [_rope, _attn, _linear])
def test_tensors_of_another_device(call, monkeypatch):
    out = _linear()  # (and buffers given, where a call would make them)
    given = {_rope: dict(q_out=torch.empty((3, 4, 64), device="cuda", dtype=torch.bfloat16)),
             _attn: dict(out=torch.empty((3, 4, 64), device="cuda", dtype=torch.bfloat16)), _linear: dict(y=out)}[call]
    for name in NAMES:
        def there(*a, fn=getattr(ops, name), **kw):
            with monkeypatch.context() as m:
                m.setattr(ops, "_binding", _Nothing)
                m.setattr(torch.cuda, "current_device", lambda: 1)
                return fn(*a, **kw)
        monkeypatch.setattr(ops, name, there)
    with pytest.raises(ValueError, match="current CUDA device"):
        call(stream=torch.cuda.current_stream(), **given)
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("call", [_rope, _attn, _linear])
def test_the_extension_takes_the_current_device(call, monkeypatch):
    answers = []
    real = ops._binding()

    class Listen:
        def __getattr__(self, name):
            def f(*a):
                answers.append(getattr(real, name)(*a))
                return answers[-1]
            return f
    monkeypatch.setattr(ops, "_binding", Listen)
    call()
    torch.cuda.synchronize()
    assert answers == [0]
