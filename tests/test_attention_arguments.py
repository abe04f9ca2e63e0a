"""Arguments of the attention side's calls that would be read under another
tensor's layout, or that lie in one another: refused before anything runs."""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _cuda(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, device="cuda", dtype=dtype)


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 16, 2, 64), (4, 8, 1, 128), (4, 8, 4, 32), (8, 4, 2, 64), (4096,)])
def test_value_cache_of_another_shape(shape):
    """As many elements as the key cache, laid out otherwise."""
    k = _cuda(4, 8, 2, 64)
    v = _cuda(*shape)
    assert v.numel() == k.numel()
    q = _cuda(3, 4, 64)
    with pytest.raises(ValueError, match="v_cache"):
        ops.prefix_attention(q, k, v, _i32(0, 3), _i32(0), _i32(4), None, None,
                             ops.Workspace(ops.prefix_attention_workspace_bytes(3, 1, 4, 2, 64)))
    kv = _cuda(3, 2, 64)
    before = v.clone()
    if v.dim() < 2 or v.shape[-2:] != (2, 64):
        with pytest.raises(ValueError, match="v_cache"):
            ops.qk_norm_rope(None, kv, kv + 1, None, None, ops.Workspace(256), k_cache=k, v_cache=v, slots=_i32(0, 5, 9))
        assert torch.equal(v, before)
