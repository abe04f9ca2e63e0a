"""A decoder layer around the MoE-FFN layer, as a DFlash / DSpark draft (or its
target) runs it on a verify block: the attention side's operators and the FFN
in the order of use.

    x -> norm -> linear (q, k, v) -> qk_norm_rope (rotation, cache write)
      -> prefix_attention -> linear (+ x) -> norm -> MoE FFN (+)

Everything a step varies (positions, cache slots, block starts, lengths, page
tables) stays on the device, so one captured graph serves every later step of
the same token count.  ``DecoderLayer4`` is the layer with projections of 4 bits
over a cache of 4 bits, and ``PagedRequests`` the pages that requests hold of such
caches or of 16-bit ones.  ``python -m moe_ffn_speculative_gb300.decoder`` runs the
Qwen3-8B DSpark draft layer on 8 requests x 9 tokens over a shared prefix of
4096 tokens, in 16 and in 4 bits, and prints the time of a step.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import ops
from . import synthetic as S


@dataclass(frozen=True)
class AttentionConfig:
    """Heads of the layer (the defaults are Qwen3-8B's) and its rotation."""
    q_heads: int = 32
    kv_heads: int = 8
    head_dim: int = 128
    rope_base: float = 1e6
    max_positions: int = 40960
    eps: float = 1e-6
    causal: bool = True  # False: every token of a block sees the whole block


class KVCache:
    """Pages of keys and values, [pages, page_size, kv_heads, head_dim]."""

    def __init__(self, pages: int, page_size: int, a: AttentionConfig, device="cuda"):
        shape = (pages, page_size, a.kv_heads, a.head_dim)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros(shape, dtype=torch.bfloat16, device=device)


class KVCache4:
    """The same in 4 bits (e2m1 codes with a scale per 32 channels), a quarter of the bytes."""

    def __init__(self, pages: int, page_size: int, a: AttentionConfig, device="cuda"):
        self.data = torch.zeros(ops.kv4_shape(pages, page_size, a.kv_heads, a.head_dim), dtype=torch.uint8, device=device)


@dataclass
class Batch:
    """What a step brings: for T tokens of B requests, int32 on the device."""
    positions: torch.Tensor               # [T]
    slots: torch.Tensor                   # [T] cache rows that take the tokens (negative: padding)
    q_start: torch.Tensor                 # [B+1]
    own_len: torch.Tensor                 # [B] own keys, the block's among them
    page_table: torch.Tensor              # [B, width]
    prefix_pages: Optional[torch.Tensor]  # shared by all requests, with prefix_len [1]
    prefix_len: Optional[torch.Tensor]


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + eps) * weight.float()).to(x.dtype)


def make_attention_weights(H: int, a: AttentionConfig, device="cuda", seed: int = 0) -> dict:
    """Random weights of the layer's attention side: N(0, 0.02) projections,
    norm weights around 1."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=0.02, mean=0.0):
        return (torch.randn(shape, generator=g, device=device) * std + mean).bfloat16()
    heads = a.q_heads + 2 * a.kv_heads
    return {"norm1": normal(H, mean=1.0), "w_qkv": normal(heads * a.head_dim, H), "q_norm": normal(a.head_dim, mean=1.0),
            "k_norm": normal(a.head_dim, mean=1.0), "w_out": normal(H, a.q_heads * a.head_dim),
            "norm2": normal(H, mean=1.0)}


class DecoderLayer:
    """Weights, workspaces and buffers of one layer for up to max_tokens tokens
    of up to max_requests requests."""

    def __init__(self, a: AttentionConfig, weights: dict, ffn: ops.MoELayer, max_requests: int):
        self.a, self.w, self.ffn = a, weights, ffn
        self.rope = ops.rope_table(a.max_positions, a.head_dim, a.rope_base, device=weights["w_qkv"].device)
        T, H = ffn.max_tokens, weights["w_out"].shape[0]
        # one workspace for the whole attention side: its calls follow one another
        self.ws = ops.Workspace(max(
            ops.prefix_attention_workspace_bytes(T, max_requests, a.q_heads, a.kv_heads, a.head_dim),
            ops.linear_workspace_bytes(T, weights["w_qkv"].shape[0], H),
            ops.linear_workspace_bytes(T, H, a.q_heads * a.head_dim)), weights["w_qkv"].device)

    def attention(self, x: torch.Tensor, cache: KVCache, b: Batch) -> torch.Tensor:
        """x + the attention block's output; the tokens' keys and values are in
        the cache afterwards."""
        a, w = self.a, self.w
        qkv = ops.linear(rms_norm(x, w["norm1"], a.eps), w["w_qkv"], self.ws)
        q, k, v = (t.unflatten(1, (-1, a.head_dim))
                   for t in qkv.split([n * a.head_dim for n in (a.q_heads, a.kv_heads, a.kv_heads)], dim=1))
        q, _, _ = ops.qk_norm_rope(q, k, v, b.positions, self.rope, self.ws, q_weight=w["q_norm"], k_weight=w["k_norm"],
                                   eps=a.eps, k_cache=cache.k, v_cache=cache.v, slots=b.slots)
        o = ops.prefix_attention(q, cache.k, cache.v, b.q_start, b.prefix_pages, b.prefix_len, b.page_table, b.own_len,
                                 self.ws, causal=a.causal)
        return ops.linear(o.flatten(1), w["w_out"], self.ws, residual=x)

    def forward(self, x: torch.Tensor, cache: KVCache, b: Batch) -> torch.Tensor:
        h = self.attention(x, cache, b)
        return h + self.ffn.forward(rms_norm(h, self.w["norm2"], self.a.eps))


def quantize_q4(w: torch.Tensor, group: int = 128):
    """Weights [N, K] as ``ops.q4_prepare`` takes them, (codes, scales, zeros): the
    nearest of 16 evenly spaced values, 0 among them, from a group's least to its
    greatest weight."""
    f = w.float().unflatten(1, (-1, group))
    lo, hi = f.amin(-1).clamp(max=0), f.amax(-1).clamp(min=0)
    scales = ((hi - lo) / 15).clamp(min=2.0 ** -20).to(w.dtype)
    s = scales.float()
    zeros = (-lo / s).round().clamp(0, 15)
    code = (f / s[..., None] + zeros[..., None]).round().clamp(0, 15).to(torch.uint8).flatten(1)
    return code[:, 0::2] | code[:, 1::2] << 4, scales, zeros.to(torch.uint8)


class DecoderLayer4(DecoderLayer):
    """The layer with its projections in 4 bits, over a cache in 4 bits (KVCache4)."""

    def __init__(self, a: AttentionConfig, weights: dict, ffn: ops.MoELayer, max_requests: int, group: int = 128):
        super().__init__(a, weights, ffn, max_requests)
        self.w_qkv, self.w_out = (ops.q4_prepare(*quantize_q4(weights[n], group)) for n in ("w_qkv", "w_out"))
        T = ffn.max_tokens
        self.ws = ops.Workspace(max(
            ops.prefix_attention_kv4_workspace_bytes(T, max_requests, a.q_heads, a.kv_heads, a.head_dim),
            *(ops.linear_q4_workspace_bytes(T, w.N, w.K) for w in (self.w_qkv, self.w_out))), weights["w_qkv"].device)

    def attention(self, x: torch.Tensor, cache: KVCache4, b: Batch) -> torch.Tensor:
        a, w = self.a, self.w
        qkv = ops.linear_q4(rms_norm(x, w["norm1"], a.eps), self.w_qkv, self.ws)
        q, k, v = (t.unflatten(1, (-1, a.head_dim))
                   for t in qkv.split([n * a.head_dim for n in (a.q_heads, a.kv_heads, a.kv_heads)], dim=1))
        q, k, _ = ops.qk_norm_rope(q, k, None, b.positions, self.rope, self.ws, q_weight=w["q_norm"], k_weight=w["k_norm"],
                                   eps=a.eps)
        ops.kv4_write(k, v, b.slots, cache.data, self.ws)
        o = ops.prefix_attention_kv4(q, cache.data, b.q_start, b.prefix_pages, b.prefix_len, b.page_table, b.own_len,
                                     self.ws, causal=a.causal)
        return ops.linear_q4(o.flatten(1), self.w_out, self.ws, residual=x)


class PagedRequests:
    """The pages that requests hold of one layer's caches or of several layers': page
    counts, table and lengths on the device, so that a captured step (``block``, the
    layers, ``keep``) serves every later one.  The first `prefix_pages` pages are the
    shared prefix's and stay taken."""

    def __init__(self, requests: int, width: int, pages: int, page_size: int, caches, prefix_pages: int = 0, device="cuda"):
        def i32(*shape, value=0):
            return torch.full(shape, value, dtype=torch.int32, device=device)
        self.page, self.caches = page_size, tuple(caches)
        self.refs, self.table, self.own_len = i32(pages), i32(requests, width, value=-1), i32(requests)
        self.refs[:prefix_pages] = 1
        self.prefix_pages = torch.arange(prefix_pages, dtype=torch.int32, device=device) if prefix_pages else None
        self.ws = ops.Workspace(ops.pages_workspace_bytes(requests, pages), device)

    def resize(self, new_len: torch.Tensor) -> None:
        ops.pages_resize(self.refs, self.table, self.own_len, new_len, self.page, self.ws, self.caches)

    def fork(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """Requests dst become copies of requests src."""
        ops.pages_fork(self.refs, self.table, self.own_len, src, dst, self.page, self.ws, self.caches)

    def block(self, n: int, prefix_len: Optional[torch.Tensor] = None):
        """Pages for n more tokens of every request.  -> (Batch of them, the lengths before).
        Tokens of a request that there were no pages for (recorded in `ws`) go to no slot."""
        base = self.own_len.clone()
        self.resize(base + n)
        at = base[:, None] + torch.arange(n, dtype=torch.int32, device=base.device)
        pages = self.table.gather(1, (at // self.page).clamp(max=self.table.shape[1] - 1).long())
        positions = at if prefix_len is None else at + prefix_len
        slots = torch.where(at < self.own_len[:, None], pages * self.page + at % self.page, -1)
        return Batch(positions=positions.flatten(), slots=slots.flatten(),
                     q_start=torch.arange(len(base) + 1, dtype=torch.int32, device=base.device) * n, own_len=self.own_len,
                     page_table=self.table, prefix_pages=self.prefix_pages, prefix_len=prefix_len), base

    def keep(self, base: torch.Tensor, kept: torch.Tensor) -> None:
        """Of a block's tokens those at offsets kept [requests, n] stay (growing; the first
        negative one, or one past the block, ends a row), moved up behind the first `base`
        ones.  A request that `block` found no pages for has no block to keep of: it stays as
        it was."""
        # (its last page may still be another request's too, which a move would write into)
        granted = torch.where(base[:, None] + kept < self.own_len[:, None], kept, -1)
        self.resize(ops.pages_compact(self.table, base, granted, self.page, self.ws, self.caches))


def shared_prefix_batch(requests: int, block: int, prefix: int, own: int, page: int, device="cuda") -> Batch:
    """A step of `requests` requests: `block` tokens each after `own` cached
    ones of their own and a shared prefix, pages in order."""
    def i32(x):
        return torch.as_tensor(x, dtype=torch.int32, device=device).contiguous()
    width, shared = -(-(own + block) // page), -(-prefix // page)
    table = shared + torch.arange(requests * width).view(requests, width)
    at = own + torch.arange(block)
    slots = table[:, at // page] * page + at % page
    return Batch(positions=i32((prefix + at).repeat(requests)), slots=i32(slots.flatten()),
                 q_start=i32(torch.arange(requests + 1) * block), own_len=i32([own + block] * requests),
                 page_table=i32(table), prefix_pages=i32(torch.arange(shared)) if prefix else None,
                 prefix_len=i32([prefix]) if prefix else None)


def main(requests: int = 8, block: int = 9, prefix: int = 4096, own: int = 500, page: int = 64, steps: int = 200) -> float:
    cfg = S.CONFIGS["qwen3_8b_dspark"].with_(T=requests * block)
    a = AttentionConfig()
    d = S.make_inputs(cfg, "cuda")
    layer = DecoderLayer(a, make_attention_weights(cfg.H, a), ops.MoELayer(d, ops.Recipe.from_config(cfg), cfg.T), requests)
    b = shared_prefix_batch(requests, block, prefix, own, page)
    cache = KVCache(-(-prefix // page) + b.page_table.numel(), page, a)
    cache.k.normal_()
    cache.v.normal_()
    x = d["x"]
    layer.forward(x, cache, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, cache, b)
    for _ in range(20):
        graph.replay()
    t0, t1 = torch.cuda.Event(True), torch.cuda.Event(True)
    t0.record()
    for _ in range(steps):
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    for ws in (layer.ws, layer.ffn.ws):
        assert ws.device_status()[0] == ops.MOE_OK
    us = t0.elapsed_time(t1) * 1e3 / steps
    print(f"decoder layer, {requests} requests x {block} tokens over {prefix} shared + {own} own keys: {us:.1f} us a step")
    return us


def main4(requests: int = 8, block: int = 9, prefix: int = 4096, own: int = 500, page: int = 64, steps: int = 200) -> float:
    """Steps of the layer in 4 bits with their pages: a block of every request, of
    which a path of three tokens stays."""
    cfg = S.CONFIGS["qwen3_8b_dspark"].with_(T=requests * block)
    a = AttentionConfig()
    d = S.make_inputs(cfg, "cuda")
    layer = DecoderLayer4(a, make_attention_weights(cfg.H, a), ops.MoELayer(d, ops.Recipe.from_config(cfg), cfg.T), requests)
    path = [i for i in (0, 2, 3) if i < block]
    warm = 20
    shared, width = -(-prefix // page), -(-(own + len(path) * (steps + warm + 2) + block) // page)
    cache = KVCache4(shared + requests * width, page, a)
    r = PagedRequests(requests, width, cache.data.shape[0], page, [cache.data], shared)
    heads = torch.randn((2, r.refs.numel() * page, a.kv_heads, a.head_dim), device="cuda", dtype=torch.bfloat16)
    ops.kv4_write(heads[0], heads[1], None, cache.data, layer.ws)
    r.resize(torch.full_like(r.own_len, own))
    prefix_len = torch.tensor([prefix], dtype=torch.int32, device="cuda") if prefix else None
    kept = torch.tensor([path] * requests, dtype=torch.int32, device="cuda")
    x = d["x"]

    def step():
        b, base = r.block(block, prefix_len)
        y = layer.forward(x, cache, b)
        r.keep(base, kept)
        return y
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(warm):
        graph.replay()
    t0, t1 = torch.cuda.Event(True), torch.cuda.Event(True)
    t0.record()
    for _ in range(steps):
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    for ws in (layer.ws, layer.ffn.ws, r.ws):
        assert ws.device_status()[0] == ops.MOE_OK
    assert r.own_len.tolist() == [own + len(path) * (1 + warm + steps)] * requests
    us = t0.elapsed_time(t1) * 1e3 / steps
    print(f"the same in 4 bits, with its pages: {us:.1f} us a step")
    return us


if __name__ == "__main__":
    main()
    main4()
