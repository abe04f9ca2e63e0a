"""The decoder layer that runs the attention side's operators and the FFN
together, against the same layer in 64 bits: a prompt into the shared prefix's
pages, then a block of every request over prefix and own pages.

The FFN is a dense one (one expert, top-1), so that no rounding moves a pick.
Tolerance: nine tensors are rounded to bf16 between x and y (two norms, qkv, the
rotated rows, the probabilities, the attention's output, its sum with x, the
FFN's and the last sum), each at most e/2 of its values off, uniform, e/sqrt(12)
in the 2-norm, and no step enlarges a relative error: 9 e/sqrt(12) = 2.6 e.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import decoder, ops
from moe_ffn_speculative_gb300 import synthetic as S
from moe_ffn_speculative_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _layer(a, T=64, H=256, seed=5):
    cfg = S.LayerConfig("dense", T=T, H=H, E=1, I=512, K=1, seed=seed)
    d = S.make_inputs(cfg, "cuda")
    w = decoder.make_attention_weights(H, a, seed=seed)
    return decoder.DecoderLayer(a, w, ops.MoELayer(d, ops.Recipe.from_config(cfg), T), 8), d, w


def _norm64(x, w, eps):
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()


def _exact(layer, d, w, x, past, positions, causal):
    """One request in 64 bits: x [n, H] after `past` (k, v) rows; -> y, (k, v)."""
    a = layer.a
    x = x.double()
    qkv = (_norm64(x, w["norm1"], a.eps) @ w["w_qkv"].double().t()).unflatten(1, (-1, a.head_dim))
    q, k, v = qkv.split([a.q_heads, a.kv_heads, a.kv_heads], dim=1)
    cs = layer.rope.double()[positions][:, None]
    c, s = cs.split(a.head_dim // 2, dim=-1)

    def turn(t, weight):
        p, r = _norm64(t, weight, a.eps).split(a.head_dim // 2, dim=-1)
        return torch.cat([p * c - r * s, r * c + p * s], dim=-1)
    q, k = turn(q, w["q_norm"]), turn(k, w["k_norm"])
    if past is not None:
        k, v = torch.cat([past[0], k]), torch.cat([past[1], v])
    G = a.q_heads // a.kv_heads
    z = torch.einsum("nhd,mhd->hnm", q, k.repeat_interleave(G, 1)) * a.head_dim ** -0.5
    if causal:
        n, m = z.shape[1:]
        z = z.masked_fill(torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None], float("-inf"))
    o = torch.einsum("hnm,mhd->nhd", z.softmax(-1), v.repeat_interleave(G, 1)).flatten(1)
    h = x + o @ w["w_out"].double().t()
    gu = _norm64(h, w["norm2"], a.eps) @ d["w_gate_up"][0].double().t()
    g, u = gu.chunk(2, dim=-1)
    return h + (torch.nn.functional.silu(g) * u) @ d["w_down"][0].double().t(), (k, v)


@pytest.mark.parametrize("causal", [True, False])
def test_prefix_then_blocks(causal):
    a = decoder.AttentionConfig(q_heads=8, kv_heads=2, head_dim=64, max_positions=512, causal=causal)
    layer, d, w = _layer(a)
    e = torch.finfo(torch.bfloat16).eps
    g = torch.Generator(device="cuda").manual_seed(1)
    page, P, n, B = 16, 40, 5, 3
    cache = decoder.KVCache(16, page, a)
    # the shared prompt: one request without a prefix, into pages 0, 1, 2
    x0 = torch.randn((P, 256), generator=g, device="cuda").bfloat16()
    b0 = decoder.shared_prefix_batch(1, P, 0, 0, page)
    y0 = layer.forward(x0, cache, b0)
    want, past = _exact(layer, d, w, x0, None, torch.arange(P, device="cuda"), causal)
    assert (y0.double() - want).norm() <= 2.6 * e * want.norm()
    # two rounds of blocks, each request's own
    own = [past] * B
    for step in range(2):
        x = torch.randn((B * n, 256), generator=g, device="cuda").bfloat16()
        b = decoder.shared_prefix_batch(B, n, P, step * n, page)
        if step == 0:
            y = layer.forward(x, cache, b)
        else:  # captured: the same bits as the direct call
            y = layer.forward(x, cache, b)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                again = layer.forward(x, cache, b)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(again, y)
        for r in range(B):
            pos = P + step * n + torch.arange(n, device="cuda")
            want, own[r] = _exact(layer, d, w, x[r * n:(r + 1) * n], own[r], pos, causal)
            assert (y[r * n:(r + 1) * n].double() - want).norm() <= 2.6 * e * want.norm()
    assert layer.ws.device_status() == (ops.MOE_OK, 0)


def test_example_runs():
    assert decoder.main(requests=2, block=3, prefix=100, own=20, steps=3) > 0
