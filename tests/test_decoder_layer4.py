"""The decoder layer in 4 bits with its pages, as a serving loop runs them: a prompt
into the shared prefix's pages, then for every request a block whose keys and values
are rounded into pages that it takes, a path of it kept, a request forked from
another; against the layer in 64 bits over the keys and values that the cache holds.

The FFN is a dense one.  Tolerance as for the 16-bit layer (nine tensors rounded to
bf16 between x and y, 9 e/sqrt(12) = 2.6 e in the 2-norm; the cache's values are the
64-bit layer's too).  The block's own keys and values in the cache: a group's scale
2^e is the least with max <= 6 * 2^e, so a code is at most 2^e < max/3 off, and
their own roundings (norm, projection, rotation) e of a row's norm each.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import decoder, ops
from test_decoder_layer import _layer, _norm64
from moe_ffn_speculative_gb300.build import build

E = torch.finfo(torch.bfloat16).eps


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _weights64(w, group):
    """What quantize_q4's codes stand for."""
    codes, scales, zeros = decoder.quantize_q4(w, group)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(1).double()
    return ((c.unflatten(1, (-1, group)) - zeros.double()[..., None]) * scales.double()[..., None]).flatten(1)


def test_quantized_weights():
    g = torch.Generator().manual_seed(3)
    w = torch.randn((24, 256), generator=g).bfloat16()
    w[3] = 0
    w[4] = w[4].abs()
    for group in (32, 64, 128):
        v, f = _weights64(w, group), w.double().unflatten(1, (-1, group))
        step = ((f.amax(-1).clamp(min=0) - f.amin(-1).clamp(max=0)) / 15)[..., None]
        # half a step, and at the ends what the zero point's rounding (half a step) and the scale's (e/2 of 15 steps) move
        assert bool(((v.unflatten(1, (-1, group)) - f).abs() <= (1 + 8 * E) * step + 2.0 ** -19).all())
        assert bool((v[3] == 0).all())


def _exact(layer, d, x, k, v, positions):
    """One request in 64 bits over the cache's rows k, v [len, heads, D], the block's
    the last ones (causal).  -> y, the block's own (k, v)."""
    a, w = layer.a, layer.w
    x, n = x.double(), x.shape[0]
    qkv = (_norm64(x, w["norm1"], a.eps) @ _weights64(w["w_qkv"], 128).t()).unflatten(1, (-1, a.head_dim))
    q, mine, value = qkv.split([a.q_heads, a.kv_heads, a.kv_heads], dim=1)
    c, s = layer.rope.double()[positions][:, None].split(a.head_dim // 2, dim=-1)

    def turn(t, weight):
        p, r = _norm64(t, weight, a.eps).split(a.head_dim // 2, dim=-1)
        return torch.cat([p * c - r * s, r * c + p * s], dim=-1)
    q, mine = turn(q, w["q_norm"]), turn(mine, w["k_norm"])
    G, m = a.q_heads // a.kv_heads, k.shape[0]
    z = torch.einsum("nhd,mhd->hnm", q, k.double().repeat_interleave(G, 1)) * a.head_dim ** -0.5
    z = z.masked_fill(torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None], float("-inf"))
    o = torch.einsum("hnm,mhd->nhd", z.softmax(-1), v.double().repeat_interleave(G, 1)).flatten(1)
    h = x + o @ _weights64(w["w_out"], 128).t()
    g, u = (_norm64(h, w["norm2"], a.eps) @ d["w_gate_up"][0].double().t()).chunk(2, dim=-1)
    return h + (torch.nn.functional.silu(g) * u) @ d["w_down"][0].double().t(), (mine, value)


def _rounded(cache, want):
    """Whether cache rows are `want` to within a code."""
    c, f = cache.double().unflatten(-1, (-1, 32)), want.unflatten(-1, (-1, 32))
    top = f.abs().amax(-1, keepdim=True)
    noise = 4 * E * want.norm(dim=-1)[..., None, None] / want.shape[-1] ** 0.5 * 6  # (a Gaussian row's 6 sigma)
    return bool(((c - f).abs() <= top / 3 + noise).all())


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_steps(captured):
    a = decoder.AttentionConfig(q_heads=8, kv_heads=2, head_dim=64, max_positions=512)
    plain, d, w = _layer(a)
    layer = decoder.DecoderLayer4(a, w, plain.ffn, 8)
    page, P, n, B, width = 16, 40, 6, 3, 4
    prefix_pages = 3
    cache = decoder.KVCache4(prefix_pages + 9, page, a)
    r = decoder.PagedRequests(B, width, cache.data.shape[0], page, [cache.data], prefix_pages)
    g = torch.Generator(device="cuda").manual_seed(1)

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def rows(pages, count):
        k, v = ops.kv4_read(cache.data, a.head_dim, layer.ws, pages=pages)
        return k.flatten(0, 1)[:count].clone(), v.flatten(0, 1)[:count].clone()

    # the shared prompt
    x0 = torch.randn((P, 256), generator=g, device="cuda").bfloat16()
    y0 = layer.forward(x0, cache, decoder.shared_prefix_batch(1, P, 0, 0, page))
    k, v = rows(r.prefix_pages, P)
    want, (mine, value) = _exact(layer, d, x0, k, v, torch.arange(P, device="cuda"))
    assert (y0.double() - want).norm() <= 2.6 * E * want.norm()
    assert _rounded(k, mine) and _rounded(v, value)
    prefix, prefix_len = (k, v), i32(P)

    x, kept = torch.empty((B * n, 256), device="cuda", dtype=torch.bfloat16), i32(*[[-1] * n] * B)
    base = torch.empty_like(r.own_len)
    batch = None

    def run():
        nonlocal batch
        batch, before = r.block(n, prefix_len)
        base.copy_(before)
        return layer.forward(x, cache, batch)
    forward, keep = run, lambda: r.keep(base, kept)
    if captured:  # one graph of the block and one of what is kept serve every step
        state = [t.clone() for t in (r.refs, r.table, r.own_len)]
        graphs = []
        for f in (run, keep):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = f()
            graphs.append((graph, y))
        for t, s in zip((r.refs, r.table, r.own_len), state):
            assert torch.equal(t, s)  # (a capture runs nothing)

        def forward():
            graphs[0][0].replay()
            return graphs[0][1]

        def keep():
            graphs[1][0].replay()
    held = [(prefix[0][:0], prefix[1][:0]) for _ in range(B)]  # each request's rows behind the prefix
    paths = [[[0, 2, 5], [0, 1, 2, 3, 4, 5], []], [[1, 2, 4], [3], [0, 1, 2, 3, 4]],
             [[5], [0, 1, 2, 3, 4, 5], [0, 3]], [[0, 1], [0, 4], [2, 4, 5]]]
    for step, path in enumerate(paths):
        if step == 2:  # request 0 goes on as a copy of request 1
            r.resize(i32(0, *r.own_len.tolist()[1:]))
            r.fork(i32(1), i32(0))
            held[0] = held[1]
        assert r.own_len.tolist() == [len(h[0]) for h in held]
        x.copy_(torch.randn((B * n, 256), generator=g, device="cuda"))
        for b in range(B):
            kept[b] = i32(*(path[b] + [-1] * (n - len(path[b]))))
        y = forward().clone()
        for b in range(B):
            old, at = held[b], len(held[b][0])
            assert int(r.own_len[b]) == at + n
            k, v = rows(r.table[b, :-(-(at + n) // page)].contiguous(), at + n)
            assert torch.equal(k[:at], old[0]) and torch.equal(v[:at], old[1])
            want, (mine, value) = _exact(layer, d, x[b * n:(b + 1) * n], torch.cat([prefix[0], k]),
                                         torch.cat([prefix[1], v]), P + at + torch.arange(n, device="cuda"))
            assert (y[b * n:(b + 1) * n].double() - want).norm() <= 2.6 * E * want.norm(), (step, b)
            assert _rounded(k[at:], mine) and _rounded(v[at:], value)
            take = torch.tensor(list(range(at)) + [at + j for j in path[b]], dtype=torch.long, device="cuda")
            held[b] = k[take], v[take]
        keep()
    for b in range(B):
        count = len(held[b][0])
        assert int(r.own_len[b]) == count
        k, v = rows(r.table[b, :-(-count // page)].contiguous(), count)
        assert torch.equal(k, held[b][0]) and torch.equal(v, held[b][1])
    r.resize(torch.zeros_like(r.own_len))
    assert r.refs.tolist() == [1] * prefix_pages + [0] * 9 and bool((r.table == -1).all())
    for ws in (layer.ws, r.ws):
        assert ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_requests_without_pages():
    """What finds no page is recorded and written nowhere: not into the page that a fork
    shares, nor past the table."""
    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    a = decoder.AttentionConfig(q_heads=4, kv_heads=1, head_dim=64)
    cache = decoder.KVCache4(3, 8, a)
    r = decoder.PagedRequests(3, 2, 3, 8, [cache.data])
    r.resize(i32(5, 8, 0))
    r.fork(i32(0), i32(2))          # takes the last page
    assert r.own_len.tolist() == [5, 8, 5] and sorted(r.refs.tolist()) == [1, 1, 1]
    b, base = r.block(2)            # 5 + 2 fit their pages; 8 + 2 need one that there is not
    assert base.tolist() == [5, 8, 5] and r.own_len.tolist() == [7, 8, 7]
    first = r.table[:, 0].tolist()
    assert b.slots.tolist() == [first[0] * 8 + 5, first[0] * 8 + 6, -1, -1, first[2] * 8 + 5, first[2] * 8 + 6]
    assert r.ws.device_status()[0] == ops.MOE_ERR_DEVICE_POOL
    # past the table's end: left alone
    r = decoder.PagedRequests(1, 2, 3, 8, [cache.data])
    r.resize(i32(15))
    b, _ = r.block(2)
    assert r.own_len.tolist() == [15] and b.slots.tolist() == [-1, -1]
    assert r.ws.device_status()[0] != ops.MOE_OK


@pytest.mark.gpu
def test_example_runs():
    assert decoder.main4(requests=2, block=3, prefix=100, own=20, steps=3) > 0
