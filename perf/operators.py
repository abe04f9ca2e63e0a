"""Cases of the attention side of a draft decoder layer, in two forms.

Three operators stand next to the MoE-FFN layer in every decoder layer of a
draft or target model that serves verify blocks:

* ``qk_norm_rope``: RMS norms of the query and key heads and the position
  rotation in one pass, with the rotated keys and the values written to their
  slots of a paged cache;
* ``prefix_attention``: attention of a batch of requests whose cached context
  begins with one prefix that all of them share, followed by pages of their
  own;
* ``linear``: matrix product with bias, activation and residual in its
  epilogue (the projections before and after the attention).

Where ``own`` is false, ``run`` computes them from elementary torch operations
in 32 bits, rounded once at the end; where it is true, through
``moe_ffn_speculative_gb300.ops``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"


# ----------------------------------------------------------------- the cases

def _rope_case(name, T, Hq, Hkv, D, dtype="bf16", rot=None, interleaved=False, page=64, far=40960, pad=0):
    return {"name": name, "op": "qk_norm_rope", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            "rot": D if rot is None else rot, "interleaved": interleaved, "page": page, "far": far, "pad": pad}


def _attn_case(name, B, n, P, lo, hi, Hq, Hkv, D, dtype="bf16", causal=True, page=64, ragged=False):
    return {"name": name, "op": "prefix_attention", "B": B, "n": n, "P": P, "own_lo": lo, "own_hi": hi, "Hq": Hq,
            "Hkv": Hkv, "D": D, "dtype": dtype, "causal": causal, "page": page, "ragged": ragged}


def _linear_case(name, M, K, N, dtype="bf16", bias=False, act="none", residual=False):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "dtype": dtype, "bias": bias, "act": act,
            "residual": residual}


def listed():
    return [
        # one request's verify block of 9 positions, heads of the Qwen3-8B target and its draft: pure latency
        _rope_case("rope_verify_block", 9, 32, 8, 128),
        # 8 concurrent requests x verify block 9, the batch of every decode benchmark here, two rows padding
        _rope_case("rope_batch_72", 72, 32, 8, 128, pad=2),
        # a ragged batch of prompts in fp16 with 64-wide heads, half of each rotated in neighbouring pairs
        _rope_case("rope_fp16_pairs", 1003, 40, 8, 64, dtype="fp16", rot=32, interleaved=True, page=16, pad=5),
        # prefill of long prompts: bandwidth
        _rope_case("rope_prefill", 16384, 32, 8, 128),
        # four chats one token at a time after a short system prompt: the smallest attention call
        _attn_case("attn_single_tokens", 4, 1, 640, 5, 100, 32, 8, 128),
        # the 72-token verify step over a system prompt of 4096 tokens
        _attn_case("attn_verify_72", 8, 9, 4096, 100, 900, 32, 8, 128),
        # block-diffusion drafting (every position of a block sees the whole block), 64-wide heads in groups of
        # five, pages of 16, ragged blocks, one request with nothing of its own, a long odd prefix
        _attn_case("attn_draft_blocks", 13, 8, 30011, 0, 1500, 40, 8, 64, dtype="fp16", causal=False, page=16,
                   ragged=True),
        # 64 requests verifying over one document of 16384 tokens: the arithmetic of a full batch
        _attn_case("attn_batch_64", 64, 9, 16384, 10, 2000, 32, 8, 128),
        # output projection of one verify block with the residual: latency and 34 MB of weights
        _linear_case("linear_out_9", 9, 4096, 4096, residual=True),
        # fused query/key/value projection of the 72-token batch, with bias
        _linear_case("linear_qkv_72", 72, 4096, 6144, bias=True),
        # odd sizes in fp16, all of the epilogue
        _linear_case("linear_odd_fp16", 1001, 2056, 5000, dtype="fp16", bias=True, act="silu", residual=True),
        # prefill of a dense MLP's up projection (the dense draft layer's width): tensor-core rate
        _linear_case("linear_prefill", 4096, 4096, 12288, bias=True, act="gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "prefix_attention", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "qk_norm_rope":
        D = rng.choice([64, 128, 128])
        Hq, Hkv = rng.choice([(32, 8), (40, 8), (28, 4), (16, 16), (24, 3), (64, 8)])
        T = _log(rng, 1, 8192)
        c = _rope_case("", T, Hq, Hkv, D, dtype, rng.choice([D, D, D // 2]), rng.random() < 0.3,
                       rng.choice([16, 32, 64, 128]), _log(rng, 64, 131072), rng.randint(0, min(5, T - 1)))
    elif op == "prefix_attention":
        D = rng.choice([64, 128, 128])
        Hq, Hkv = rng.choice([(32, 8), (40, 8), (28, 4), (16, 16), (24, 3), (64, 8)])
        while True:
            B, n, P = _log(rng, 1, 64), rng.randint(1, 16), rng.choice([0, _log(rng, 1, 32768), _log(rng, 256, 32768)])
            hi = _log(rng, 1, 2048)
            if B * n * Hq * (P + hi) <= 576 * 32 * 17000:  # the largest listed case
                break
        c = _attn_case("", B, n, P, rng.randint(0, hi), hi, Hq, Hkv, D, dtype, rng.random() < 0.6,
                       rng.choice([16, 32, 64, 128]), rng.random() < 0.5)
    else:
        while True:
            M, K, N = _log(rng, 1, 4096), 8 * _log(rng, 8, 1536), 8 * _log(rng, 8, 1536)
            if M * K * N <= 4096 * 4096 * 12288:
                break
        c = _linear_case("", M, K, N, dtype, rng.random() < 0.5, rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]),
                         rng.random() < 0.5)
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly apart."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _block_lengths(c):
    return _spread(1, c["n"], c["B"]) if c["ragged"] else [c["n"]] * c["B"]


def _pair_lengths(c):
    """(tokens of the block, own cached tokens) of every request.  The block's
    own keys are in the cache before the attention runs."""
    return list(zip(_block_lengths(c), _spread(c["own_lo"], c["own_hi"], c["B"])))


def work(c):
    if c["op"] == "qk_norm_rope":
        row = (c["Hq"] + 2 * c["Hkv"]) * c["D"] * 2
        return {"bytes": c["T"] * (2 * row + 4 * c["rot"] + 8), "flops": c["T"] * (c["Hq"] + c["Hkv"]) * c["D"] * 8}
    if c["op"] == "prefix_attention":
        pairs = _pair_lengths(c)
        T = sum(n for n, _ in pairs)
        keys = T * c["P"]
        for n, own_len in pairs:
            keys += sum(max(0, own_len - n + i + 1) for i in range(n)) if c["causal"] else n * own_len
        kv = (c["P"] + sum(o for _, o in pairs)) * c["Hkv"] * c["D"] * 2 * 2
        return {"bytes": kv + T * c["Hq"] * (c["D"] * 2 * 2 + 4), "flops": 4 * c["D"] * c["Hq"] * keys}
    M, K, N = c["M"], c["K"], c["N"]
    return {"bytes": 2 * (M * K + N * K + M * N * (2 if c["residual"] else 1) + (N if c["bias"] else 0)),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _prepare_rope(c, g):
    T, Hq, Hkv, D, dt = c["T"], c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
    # the rows of one fused projection: query heads, key heads, value heads
    qkv = _normal(g, (T, (Hq + 2 * Hkv) * D), dt)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    inv = 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEVICE, dtype=torch.float64) / c["rot"])
    angle = torch.arange(c["far"], device=DEVICE, dtype=torch.float64)[:, None] * inv
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    positions = torch.randint(0, c["far"], (T,), generator=g, device=DEVICE, dtype=torch.int32)
    pages = -(-2 * T // c["page"]) + 1
    rows = pages * c["page"]
    slots = torch.randperm(rows, generator=g, device=DEVICE)[:T].to(torch.int32)
    if c["pad"]:
        slots[T - c["pad"]:] = -1
    # the pool's rows, and one more that the plain form writes padding to
    k_rows, v_rows = _normal(g, (rows + 1, Hkv, D), dt), _normal(g, (rows + 1, Hkv, D), dt)
    return {"q": q, "k": k, "v": v, "table": table, "positions": positions, "slots": slots,
            "q_weight": _normal(g, (D,), dt, 0.2) + 1, "k_weight": _normal(g, (D,), dt, 0.2) + 1, "eps": 1e-6,
            "k_rows": k_rows, "v_rows": v_rows,
            "k_cache": k_rows[:rows].view(pages, c["page"], Hkv, D),
            "v_cache": v_rows[:rows].view(pages, c["page"], Hkv, D),
            "q_out": torch.empty((T, Hq, D), dtype=dt, device=DEVICE)}


def _prepare_attn(c, g):
    Hq, Hkv, D, dt, page = c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]], c["page"]
    pairs = _pair_lengths(c)
    order = torch.randperm(c["B"], generator=g, device=DEVICE).tolist()
    pairs = [pairs[i] for i in order]
    lens = [n for n, _ in pairs]
    T = sum(lens)
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    prefix_pages = -(-c["P"] // page)
    width = max(1, max(-(-o // page) for _, o in pairs))
    pages = prefix_pages + c["B"] * width + 3
    table = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    return {"q": _normal(g, (T, Hq, D), dt), "k_cache": _normal(g, (pages, page, Hkv, D), dt),
            "v_cache": _normal(g, (pages, page, Hkv, D), dt),
            "q_start": torch.tensor(start, dtype=torch.int32, device=DEVICE),
            "prefix_pages": table[:max(1, prefix_pages)].contiguous(),
            "prefix_len": torch.tensor([c["P"]], dtype=torch.int32, device=DEVICE),
            "page_table": table[max(1, prefix_pages):][:c["B"] * width].view(c["B"], width).contiguous(),
            "own_len": torch.tensor([o for _, o in pairs], dtype=torch.int32, device=DEVICE),
            "scale": D ** -0.5, "causal": c["causal"], "P": c["P"], "n": max(lens), "own_max": max(o for _, o in pairs),
            "out": torch.empty((T, Hq, D), dtype=dt, device=DEVICE),
            "lse": torch.empty((T, Hq), dtype=torch.float32, device=DEVICE)}


def _prepare_linear(c, g):
    M, K, N, dt = c["M"], c["K"], c["N"], DTYPES[c["dtype"]]
    return {"x": _normal(g, (M, K), dt), "w": _normal(g, (N, K), dt, 0.02),
            "bias": _normal(g, (N,), dt) if c["bias"] else None, "act": c["act"],
            "residual": _normal(g, (M, N), dt) if c["residual"] else None,
            "y": torch.empty((M, N), dtype=dt, device=DEVICE)}


def _inputs(case, seed):
    g = _gen(seed)
    return {"qk_norm_rope": _prepare_rope, "prefix_attention": _prepare_attn, "linear": _prepare_linear}[case["op"]](case, g)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"], s["case"] = case["op"], case
    if own:
        # the workspace that a user's program keeps next to its buffers
        from moe_ffn_speculative_gb300 import ops
        s["ops"] = ops
        if case["op"] == "qk_norm_rope":
            s["ws"] = ops.Workspace(ops.STATUS_BYTES)
        elif case["op"] == "prefix_attention":
            s["ws"] = ops.Workspace(ops.prefix_attention_workspace_bytes(s["q"].shape[0], case["B"], case["Hq"],
                                                                         case["Hkv"], case["D"]))
        else:
            s["ws"] = ops.Workspace(ops.linear_workspace_bytes(case["M"], case["N"], case["K"]))
    return s


# ------------------------------------------------------------ the two forms

def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    cs = s["table"][s["positions"].long()][:, None]
    cos, sin = cs[..., :half], cs[..., half:]

    def norm_rotate(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        r, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([r, rest], dim=-1)

    s["q_out"].copy_(norm_rotate(s["q"], s["q_weight"]))
    spare = s["k_rows"].shape[0] - 1
    at = torch.where(s["slots"] < 0, spare, s["slots"]).long()
    s["k_rows"].index_copy_(0, at, norm_rotate(s["k"], s["k_weight"]).to(s["k_rows"].dtype))
    s["v_rows"].index_copy_(0, at, s["v"].contiguous())
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attn(s):
    c = s["case"]
    T, Hq, D = s["q"].shape
    Hkv, page, P, L, B = c["Hkv"], c["page"], s["P"], s["own_max"], c["B"]
    G = Hq // Hkv
    q = s["q"].float().view(T, Hkv, G, D) * s["scale"]
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    token = torch.arange(T, device=q.device)
    req = torch.searchsorted(start, token, right=True) - 1
    place = token - start[req]
    at = torch.arange(P, device=q.device)
    pages = s["prefix_pages"].long()
    kp, vp = (x[pages[at // page], at % page].float() for x in (s["k_cache"], s["v_cache"]))
    score = torch.einsum("thgd,phd->thgp", q, kp)
    # the requests' own keys, padded to the longest, against their blocks, padded to the longest
    at = torch.arange(L, device=q.device)
    own_pages = s["page_table"].long()[:, at // page]
    ko, vo = (x[own_pages, at % page].float() for x in (s["k_cache"], s["v_cache"]))
    blocks = q.new_zeros((B, s["n"], Hkv, G, D))
    blocks[req, place] = q
    own_len = s["own_len"].long()[req]
    seen = (own_len - n[req] + place + 1).clamp(min=0) if s["causal"] else own_len
    own_score = torch.einsum("bnhgd,blhd->bnhgl", blocks, ko)[req, place]
    own_score = own_score.masked_fill((at >= seen[:, None])[:, None, None], float("-inf"))
    score = torch.cat([score, own_score], dim=-1)
    top = score.amax(-1, keepdim=True) if P + L else score.new_full((T, Hkv, G, 1), float("-inf"))
    p = torch.exp(score - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("thgp,phd->thgd", p[..., :P], vp)
    po = p.new_zeros((B, s["n"], Hkv, G, L))
    po[req, place] = p[..., P:]
    out = out + torch.einsum("bnhgl,blhd->bnhgd", po, vo)[req, place]
    s["out"].copy_((out / torch.where(total > 0, total, torch.ones_like(total))).reshape(T, Hq, D))
    s["lse"].copy_((top + total.log()).reshape(T, Hq))
    return s["out"], s["lse"]


def _activate(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    if act == "relu":
        return torch.clamp(v, min=0)
    return v


def _plain_linear(s):
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _activate(v, s["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    s["y"].copy_(v)
    return s["y"]


def run(s):
    if not own:
        return {"qk_norm_rope": _plain_rope, "prefix_attention": _plain_attn, "linear": _plain_linear}[s["op"]](s)
    ops = s["ops"]
    if s["op"] == "qk_norm_rope":
        return ops.qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["table"], s["ws"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=s["eps"], interleaved=s["case"]["interleaved"],
                                q_out=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"])
    if s["op"] == "prefix_attention":
        out = ops.prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["q_start"], s["prefix_pages"],
                                   s["prefix_len"], s["page_table"], s["own_len"], s["ws"], causal=s["causal"],
                                   scale=s["scale"], out=s["out"], lse=s["lse"])
        return out, s["lse"]
    return ops.linear(s["x"], s["w"], s["ws"], bias=s["bias"], activation=s["act"], residual=s["residual"], y=s["y"])


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    if case["op"] == "linear":
        y = torch.nn.functional.linear(s["x"].to(f), s["w"].to(f), None if s["bias"] is None else s["bias"].to(f))
        if case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * 0.5 * torch.erfc(-y / math.sqrt(2))
        elif case["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif case["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        return y if s["residual"] is None else y + s["residual"].to(f)
    if case["op"] == "qk_norm_rope":
        rot, half, D = case["rot"], case["rot"] // 2, case["D"]
        # first[i], second[i]: the places of the i-th rotated pair
        first = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        turn = torch.complex(*(t.to(f) for t in s["table"][s["positions"].long()].split(half, dim=1)))
        done = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.to(f)
            y = x / ((x.norm(dim=-1, keepdim=True) ** 2) / D + s["eps"]).sqrt() * w.to(f)
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            done.append(y)
        k_cache, v_cache = s["k_cache"].to(f), s["v_cache"].to(f)
        keep = s["slots"] >= 0
        k_cache.view(-1, case["Hkv"], D)[s["slots"][keep].long()] = done[1][keep]
        v_cache.view(-1, case["Hkv"], D)[s["slots"][keep].long()] = s["v"][keep].to(f)
        return done[0], k_cache, v_cache
    # attention: one request and one key head at a time over the keys it sees
    T, Hq, D = s["q"].shape
    G, page = Hq // case["Hkv"], case["page"]
    out = torch.zeros((T, Hq, D), dtype=f, device=DEVICE)
    lse = torch.full((T, Hq), float("-inf"), dtype=f, device=DEVICE)
    starts, lens = s["q_start"].tolist(), s["own_len"].tolist()
    hkv = case["Hkv"]

    def rows(pages, count):
        n = -(-count // page)
        ids = pages[:n].long()
        return (x[ids].reshape(n * page, hkv, D)[:count].transpose(0, 1).to(f) for x in (s["k_cache"], s["v_cache"]))

    kp, vp = rows(s["prefix_pages"], case["P"])
    for b, own_len in enumerate(lens):
        t0, t1 = starts[b], starts[b + 1]
        n = t1 - t0
        ko, vo = rows(s["page_table"][b], own_len)
        k, v = torch.cat([kp, ko], dim=1), torch.cat([vp, vo], dim=1)
        if k.shape[1] == 0:
            continue
        q = s["q"][t0:t1].to(f).view(n, hkv, G, D).permute(1, 2, 0, 3)  # head, group, token
        logit = q.reshape(hkv, G * n, D) @ k.transpose(1, 2) * s["scale"]
        logit = logit.view(hkv, G, n, -1)
        if s["causal"]:
            last = case["P"] + own_len - n + torch.arange(n, device=DEVICE)
            logit = torch.where(torch.arange(k.shape[1], device=DEVICE) <= last[:, None], logit, float("-inf"))
        z = torch.logsumexp(logit, dim=-1, keepdim=True)
        w = torch.where(z == float("-inf"), torch.zeros_like(logit), torch.exp(logit - z))
        o = (w.view(hkv, G * n, -1) @ v).view(hkv, G, n, D)
        out[t0:t1] = o.permute(2, 0, 1, 3).reshape(n, Hq, D)
        lse[t0:t1] = z[..., 0].permute(2, 0, 1).reshape(n, Hq)
    return out, lse
