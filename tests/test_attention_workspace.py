"""The workspace of moe_prefix_attention: a size asked for T tokens of B requests
serves every smaller step of the same heads."""
import pytest
import torch

from moe_ffn_speculative_gb300 import decoder, ops
from moe_ffn_speculative_gb300 import synthetic as S
from moe_ffn_speculative_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _takes(T, B, Hq, Hkv, D, nbytes, buffers):
    """Whether a call of this shape accepts a workspace of nbytes.  Refused or
    not, nothing is read: a call that gets past the workspace's check attends
    over no keys at all."""
    q, out, start, ws = buffers
    return ops.lib().moe_prefix_attention(
        q.data_ptr(), Hq * D, T, B, start.data_ptr(), Hq, Hkv, D, ops.DTYPE_BF16, None, None, 0, 16, None, 0, None,
        None, 0, None, 1, 0.1, out.data_ptr(), None, ws.ptr(), nbytes, None) == ops.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (40, 8, 64), (28, 4, 128), (16, 16, 64), (64, 1, 128), (100, 1, 64),
                                      (129, 3, 64)])
def test_size_never_falls(Hq, Hkv, D):
    """Over all T and B: the size is not below any smaller call's."""
    size = ops.lib().moe_prefix_attention_workspace_bytes
    last = [0] * 17
    for T in range(1, 301):
        row = 0
        for B in range(17):
            n = size(T, B, Hq, Hkv, D)
            assert n >= row and n >= last[B], (T, B)
            row = last[B] = n


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,T,B", [(40, 8, 64, 72, 8), (32, 8, 128, 97, 1), (32, 8, 128, 96, 8), (28, 4, 128, 70, 5),
                                          (64, 1, 128, 9, 3)])
def test_smaller_steps_are_taken(Hq, Hkv, D, T, B):
    n = ops.prefix_attention_workspace_bytes(T, B, Hq, Hkv, D)
    ws = ops.Workspace(n)
    q = torch.zeros((T, Hq, D), device="cuda", dtype=torch.bfloat16)
    buffers = (q, torch.empty_like(q), torch.zeros(B + 1, device="cuda", dtype=torch.int32), ws)
    refused = [(t, b) for t in range(1, T + 1) for b in range(B + 1) if not _takes(t, b, Hq, Hkv, D, n, buffers)]
    torch.cuda.synchronize()
    assert refused == []
    assert ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_decoder_layer_takes_smaller_steps():
    """Sized for 72 tokens of 8 requests, then steps of fewer requests and fewer
    tokens: the same rows as a layer sized for that step."""
    a = decoder.AttentionConfig(q_heads=40, kv_heads=8, head_dim=64, max_positions=512)
    cfg = S.LayerConfig("dense", T=72, H=256, E=1, I=512, K=1, seed=3)
    d = S.make_inputs(cfg, "cuda")
    w = decoder.make_attention_weights(cfg.H, a, seed=3)
    layer = decoder.DecoderLayer(a, w, ops.MoELayer(d, ops.Recipe.from_config(cfg), 72), 8)
    g = torch.Generator(device="cuda").manual_seed(4)
    for requests, block in ((8, 9), (5, 14), (4, 18), (1, 72), (2, 33), (1, 1)):
        b = decoder.shared_prefix_batch(requests, block, 40, 7, 16)
        pages = 3 + b.page_table.numel()
        cache = decoder.KVCache(pages, 16, a)
        cache.k.normal_(generator=g)
        cache.v.normal_(generator=g)
        other = decoder.KVCache(pages, 16, a)
        other.k.copy_(cache.k)
        other.v.copy_(cache.v)
        x = torch.randn((requests * block, 256), generator=g, device="cuda").bfloat16()
        exact = decoder.DecoderLayer(a, w, layer.ffn, requests)
        exact.ws = ops.Workspace(ops.prefix_attention_workspace_bytes(requests * block, requests, 40, 8, 64))
        assert torch.equal(layer.attention(x, cache, b), exact.attention(x, other, b))
        assert layer.ws.device_status() == (ops.MOE_OK, 0)
