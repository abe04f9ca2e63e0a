"""Cases of serving in 4 bits around the MoE-FFN layer, in two forms.

The experts of a draft layer are served in 4 bits already; these operators do
the same for the attention side of its decoder layer, whose projections and
cache are otherwise read in 16 bits, and keep the pages of that cache:

* ``linear_q4``: matrix product with weights of 4 bits (whole numbers 0 .. 15,
  a scale and a zero point for every group of inputs) and the epilogue of the
  16-bit ``linear``;
* ``kv4_write`` with ``kv4_read``: keys and values rounded to e2m1 codes with
  one e8m0 scale per 32 channels as they go to their slots of a paged cache,
  and pages of that cache expanded to 16 bits again;
* ``prefix_attention_kv4``: attention over such a cache: a prefix that all
  requests share, followed by pages of their own;
* ``pages_resize``, ``pages_fork``, ``pages_compact``: pages given out, shared,
  taken back and moved up as requests grow, fork, keep part of a draft and end.

A kv4 cache is uint8 [pages, key heads, page_size * (D + D / 16)].  The block of
a page and a head holds the codes of its keys, then those of its values, each as
[D / 32][page_size][16 bytes] (the even channel in the low nibble), then the
scales of its keys and those of its values, each as [page_size][D / 32].

Where ``own`` is false, ``run`` computes from elementary torch operations in
32 bits, rounded once at the end; where it is true, through
``moe_ffn_speculative_gb300.ops``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"
GROUP = 32                    # channels that share a scale in the cache
E8M0_LOW, E8M0_HIGH = 104, 140  # scales 2^-23 .. 2^13, whose products with a code are exact in f16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- the cases

def _linear_case(name, M, K, N, group, dtype="bf16", zeros=True, bias=False, act="none", residual=False):
    return {"name": name, "op": "linear_q4", "M": M, "K": K, "N": N, "group": group, "dtype": dtype, "zeros": zeros,
            "bias": bias, "act": act, "residual": residual}


def _write_case(name, T, Hkv, D, dtype="bf16", page=64, pad=0):
    return {"name": name, "op": "kv4_write", "T": T, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "pad": pad}


def _attn_case(name, B, n, P, lo, hi, Hq, Hkv, D, dtype="bf16", causal=True, page=64, ragged=False):
    return {"name": name, "op": "prefix_attention_kv4", "B": B, "n": n, "P": P, "own_lo": lo, "own_hi": hi, "Hq": Hq,
            "Hkv": Hkv, "D": D, "dtype": dtype, "causal": causal, "page": page, "ragged": ragged}


def _fork_case(name, parents, children, lo, hi, page, pools, Hkv, D, spare):
    return {"name": name, "op": "pages_fork", "parents": parents, "children": children, "lo": lo, "hi": hi,
            "page": page, "pools": pools, "Hkv": Hkv, "D": D, "spare": spare}


def _step_case(name, B, n, lo, hi, page, pools, Hkv, D, spare):
    return {"name": name, "op": "pages_step", "B": B, "n": n, "lo": lo, "hi": hi, "page": page, "pools": pools,
            "Hkv": Hkv, "D": D, "spare": spare}


def listed():
    return [
        # output projection of the Qwen3-8B target for one token of one request: latency and 8 MB of weights
        _linear_case("q4_out_single", 1, 4096, 4096, 128, residual=True),
        # fused query/key/value projection of the 72-token verify batch (8 requests x 9), with bias
        _linear_case("q4_qkv_72", 72, 4096, 6144, 128, bias=True),
        # odd sizes in fp16, small groups, all of the epilogue
        _linear_case("q4_odd_fp16", 37, 2080, 5000, 32, dtype="fp16", bias=True, act="silu", residual=True),
        # prefill of a dense MLP's up projection: symmetric codes, tensor-core rate
        _linear_case("q4_prefill", 2048, 4096, 12288, 64, zeros=False, act="gelu"),
        # the verify batch's keys and values, two rows padding: pure latency
        _write_case("kv4_write_72", 72, 8, 128, pad=2),
        # prefill of long prompts into small pages, and the pages read back for a prompt's 16-bit attention
        _write_case("kv4_write_prefill", 16384, 8, 128, page=16, pad=5),
        # four chats one token at a time after a short system prompt: the smallest attention call
        _attn_case("kv4_single_tokens", 4, 1, 640, 5, 100, 32, 8, 128),
        # the 72-token verify step over a system prompt of 4096 tokens
        _attn_case("kv4_verify_72", 8, 9, 4096, 100, 900, 32, 8, 128),
        # block-diffusion drafting in fp16 (a block sees itself whole), 64-wide heads in groups of five, pages of 16,
        # ragged blocks, one request with nothing of its own, a long odd prefix
        _attn_case("kv4_draft_blocks", 13, 8, 30011, 0, 1500, 40, 8, 64, dtype="fp16", causal=False, page=16,
                   ragged=True),
        # single tokens of 16 long conversations, what a cache in 4 bits is for: bandwidth
        _attn_case("kv4_long", 16, 1, 0, 20011, 60000, 32, 8, 128),
        # every one of 64 conversations forked twice, over the caches of a five-layer draft: the last pages are copied
        _fork_case("fork_128", 64, 128, 100, 2000, 64, 10, 8, 128, 500),
        # a verify step of 8 requests: pages for the block, the accepted tokens moved up, the rest given back
        _step_case("step_8x9", 8, 9, 100, 900, 64, 5, 8, 128, 100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_q4", "linear_q4", "kv4_write", "prefix_attention_kv4", "prefix_attention_kv4", "pages"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    heads = rng.choice([(32, 8), (40, 8), (28, 4), (16, 16), (24, 3), (64, 8)])
    D, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "linear_q4":
        group = rng.choice([32, 64, 128, 128])
        while True:
            M, K, N = _log(rng, 1, 2048), group * _log(rng, 2, 12288 // group), 8 * _log(rng, 8, 1536)
            if M * K * N <= 2048 * 4096 * 12288:
                break
        c = _linear_case("", M, K, N, group, dtype, rng.random() < 0.6, rng.random() < 0.5,
                         rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]), rng.random() < 0.5)
    elif op == "kv4_write":
        T = _log(rng, 1, 16384)
        c = _write_case("", T, heads[1], D, dtype, page, rng.randint(0, min(5, T - 1)))
    elif op == "prefix_attention_kv4":
        while True:
            B, n, P = _log(rng, 1, 64), rng.randint(1, 16), rng.choice([0, _log(rng, 1, 32768), _log(rng, 256, 32768)])
            hi = _log(rng, 1, 60000)
            lo = rng.randint(0, hi)
            # no more cached bytes and no more products than the listed cases
            if ((P + B * (lo + hi) // 2) * heads[1] * D <= 16 * 40000 * 8 * 128
                    and B * n * heads[0] * (P + hi) * D <= 72 * 40 * 31511 * 128):
                break
        c = _attn_case("", B, n, P, lo, hi, *heads, D, dtype, rng.random() < 0.6, page, rng.random() < 0.5)
    elif rng.random() < 0.5:
        parents, pools = _log(rng, 1, 64), rng.randint(1, 10)
        c = _fork_case("", parents, _log(rng, 1, 2 * parents), 0, _log(rng, 1, 2000), page, pools, rng.choice([2, 4, 8]),
                       D, 2 * parents + rng.randint(0, 500))
    else:
        B, n = _log(rng, 1, 64), rng.randint(1, 16)
        c = _step_case("", B, n, 0, _log(rng, 1, 2000), page, rng.randint(1, 5), rng.choice([2, 4, 8]), D,
                       2 * B + rng.randint(0, 500))
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly apart."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _pair_lengths(c):
    """(tokens of the block, own cached tokens) of every request.  The block's
    own keys are in the cache before the attention runs."""
    blocks = _spread(1, c["n"], c["B"]) if c["ragged"] else [c["n"]] * c["B"]
    return list(zip(blocks, _spread(c["own_lo"], c["own_hi"], c["B"])))


def _kept(i, n):
    """Tokens of its block of n that the i-th request keeps."""
    return (i * 5 + 2) % n + 1


def work(c):
    op = c["op"]
    if op == "linear_q4":
        M, K, N = c["M"], c["K"], c["N"]
        groups = N * (K // c["group"])
        weights = N * K // 2 + groups * 2 + (groups if c["zeros"] else 0)
        return {"bytes": weights + 2 * (M * K + M * N * (2 if c["residual"] else 1) + (N if c["bias"] else 0)),
                "flops": 2 * M * N * K}
    if op == "kv4_write":
        row, rows = c["Hkv"] * c["D"], (-(-c["T"] // c["page"]) + 1) * c["page"]
        # keys and values in, codes and scales out; then every page in, keys and values out
        return {"bytes": c["T"] * (4 * row + row + row // 16 + 4) + rows * (row + row // 16 + 4 * row),
                "flops": 4 * row * (c["T"] + rows)}
    if op == "prefix_attention_kv4":
        pairs = _pair_lengths(c)
        T = sum(n for n, _ in pairs)
        keys = T * c["P"]
        for n, own_len in pairs:
            keys += sum(max(0, own_len - n + i + 1) for i in range(n)) if c["causal"] else n * own_len
        kv = (c["P"] + sum(o for _, o in pairs)) * c["Hkv"] * (c["D"] + c["D"] // 16)
        return {"bytes": kv + T * c["Hq"] * (c["D"] * 2 * 2 + 4), "flops": 4 * c["D"] * c["Hq"] * keys}
    pages = _page_count(c)
    if op == "pages_fork":
        lens = _spread(c["lo"], c["hi"], c["parents"])
        tails = sum(1 for i in range(c["children"]) if lens[i % c["parents"]] % c["page"])
        shared = sum(lens[i % c["parents"]] // c["page"] for i in range(c["children"]))
        return {"bytes": 2 * tails * c["pools"] * c["page"] * c["Hkv"] * c["D"] * 2 + 4 * pages + 8 * shared,
                "flops": pages}
    moved = sum(sum(1 for j, s in enumerate(_keep(i, c["n"])) if s >= 0 and s != j) for i in range(c["B"]))
    return {"bytes": 2 * moved * c["pools"] * c["Hkv"] * (c["D"] + c["D"] // 16) + 4 * pages + 8 * c["B"] * c["n"],
            "flops": pages}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _encode(x):
    """x [..., D] as e2m1 codes (uint8, one a byte) and e8m0 scales [..., D / 32]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    _, e = torch.frexp(top / 6)
    # the least e with top <= 6 * 2^e; the quotient was rounded, so exact products settle it
    e = torch.where(top > 6 * torch.ldexp(torch.ones_like(top), e), e + 1, e)
    e = torch.where(top <= 6 * torch.ldexp(torch.ones_like(top), e - 1), e - 1, e)
    e = e.clamp(E8M0_LOW - 127, E8M0_HIGH - 127)
    e = torch.where(top == 0, torch.full_like(e, E8M0_LOW - 127), e)
    v = torch.ldexp(g, -e[..., None]).abs()
    # nearest value; a tie goes to the even code
    code = ((v > 0.25).int() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5)).to(torch.uint8)
    code = code | (torch.signbit(g).to(torch.uint8) << 3)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _values(code, scale):
    """The numbers that codes [..., D] with scales [..., D / 32] stand for, fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    v = table[code.int()].unflatten(-1, (-1, GROUP))
    return torch.ldexp(v, (scale.int() - 127)[..., None]).flatten(-2)


def _block(k, v):
    """k, v [pages, page, Hkv, D] as a kv4 cache."""
    parts = []
    for codes, _ in (_encode(k), _encode(v)):
        pairs = codes[..., 0::2] | (codes[..., 1::2] << 4)                       # pages, page, head, D / 2
        parts.append(pairs.unflatten(-1, (-1, 16)).permute(0, 2, 3, 1, 4).flatten(2))
    for _, scales in (_encode(k), _encode(v)):
        parts.append(scales.permute(0, 2, 1, 3).flatten(2))
    return torch.cat(parts, dim=2).contiguous()


def _cache(g, pages, page, Hkv, D):
    """A kv4 cache of normally distributed keys and values."""
    cache = torch.empty((pages, Hkv, page * (D + D // 16)), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (page * Hkv * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        cache[a:a + n] = _block(_normal(g, (n, page, Hkv, D), torch.float32), _normal(g, (n, page, Hkv, D), torch.float32))
    return cache


def _split(cache, D):
    """The codes (two a byte, [pages, Hkv, D / 32, page, 16]) and scales
    ([pages, Hkv, page, D / 32]) of keys and values."""
    pages, Hkv, size = cache.shape
    page = size // (D + D // 16)
    half, sc = page * D // 2, page * D // 32
    codes = [cache[..., i * half:(i + 1) * half].view(pages, Hkv, D // 32, page, 16) for i in (0, 1)]
    scales = [cache[..., 2 * half + i * sc:2 * half + (i + 1) * sc].view(pages, Hkv, page, D // 32) for i in (0, 1)]
    return codes, scales


def _expand(pairs, scales):
    """[n, Hkv, D / 32, page, 16] bytes with [n, Hkv, page, D / 32] scales -> fp32 [n, page, Hkv, D]."""
    code = torch.stack([pairs & 15, pairs >> 4], dim=-1).flatten(-2)              # n, head, group, page, 32
    return _values(code.permute(0, 3, 1, 2, 4).flatten(-2), scales.permute(0, 2, 1, 3))


def _prepare_linear(c, g):
    M, K, N, dt = c["M"], c["K"], c["N"], DTYPES[c["dtype"]]
    groups = K // c["group"]
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    # weights of about N(0, 0.02): a code's deviation is 4.6
    scales = (0.02 / 4.6 * (0.5 + torch.rand((N, groups), generator=g, device=DEVICE))).to(dt)
    zeros = torch.randint(5, 11, (N, groups), generator=g, device=DEVICE, dtype=torch.uint8) if c["zeros"] else None
    return {"x": _normal(g, (M, K), dt), "codes": codes, "scales": scales, "zeros": zeros, "group": c["group"],
            "bias": _normal(g, (N,), dt) if c["bias"] else None, "act": c["act"],
            "residual": _normal(g, (M, N), dt) if c["residual"] else None,
            "y": torch.empty((M, N), dtype=dt, device=DEVICE)}


def _prepare_write(c, g):
    T, Hkv, D, dt, page = c["T"], c["Hkv"], c["D"], DTYPES[c["dtype"]], c["page"]
    pages = -(-T // page) + 1
    rows = pages * page
    kv = _normal(g, (T, 2 * Hkv * D), dt)  # the rows of one fused projection
    k, v = (x.unflatten(1, (-1, D)) for x in kv.split([Hkv * D, Hkv * D], dim=1))
    slots = torch.randperm(rows, generator=g, device=DEVICE)[:T].to(torch.int32)
    if c["pad"]:
        slots[T - c["pad"]:] = -1
    return {"k": k, "v": v, "slots": slots, "rows": rows, "cache": _cache(g, pages, page, Hkv, D),
            "k_out": torch.empty((pages, page, Hkv, D), dtype=dt, device=DEVICE),
            "v_out": torch.empty((pages, page, Hkv, D), dtype=dt, device=DEVICE)}


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
    counts = [-(-o // page) for _, o in pairs]
    width = max(1, max(counts))
    pages = prefix_pages + sum(counts) + 3
    table = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    # each request's pages, its row filled up with a page of no one
    own_pages = table[-1].repeat(c["B"], width)
    at = max(1, prefix_pages)
    for b, n in enumerate(counts):
        own_pages[b, :n] = table[at:at + n]
        at += n
    return {"q": _normal(g, (T, Hq, D), dt), "cache": _cache(g, pages, page, Hkv, D), "q_start": _i32(start),
            "prefix_pages": table[:max(1, prefix_pages)].contiguous(), "prefix_len": _i32([c["P"]]),
            "page_table": own_pages, "own_len": _i32([o for _, o in pairs]), "scale": D ** -0.5, "causal": c["causal"],
            "P": c["P"], "n": max(lens), "own_max": max(o for _, o in pairs),
            "out": torch.empty((T, Hq, D), dtype=dt, device=DEVICE),
            "lse": torch.empty((T, Hq), dtype=torch.float32, device=DEVICE)}


def _page_count(c):
    if c["op"] == "pages_fork":
        lens = _spread(c["lo"], c["hi"], c["parents"])
    else:
        lens = [x + c["n"] for x in _spread(c["lo"], c["hi"], c["B"])]
    return sum(-(-x // c["page"]) for x in lens) + c["spare"] + (c["children"] if c["op"] == "pages_fork" else 0)


def _owned(g, lens, rows, page, n_pages):
    """Reference counts, a page table of `rows` requests and their lengths:
    request i holds pages for lens[i] tokens, drawn from all of the pool."""
    counts = [-(-x // page) for x in lens]
    width = max(1, max(counts) + 2)
    ids = torch.randperm(n_pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = ids[at:at + n]
        at += n
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEVICE)
    refs[ids[:at].long()] = 1
    return refs, table, _i32(lens + [0] * (rows - len(lens)))


def _keep(i, n):
    """The offsets in its block that the i-th request keeps: a path through a
    tree of drafts, of which most nodes were refused."""
    k = _kept(i, n)
    return [j * (n - 1) // max(1, k - 1) if k > 1 else i % n for j in range(k)] + [-1] * (n - k)


def _prepare_fork(c, g):
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    n_pages, rows = _page_count(c), c["parents"] + c["children"]
    refs, table, own_len = _owned(g, _spread(c["lo"], c["hi"], c["parents"]), rows, page, n_pages)
    # one page more than the pool has: where the plain form sends what is not copied
    pools = [_normal(g, (n_pages + 1, page, Hkv, D), torch.bfloat16) for _ in range(c["pools"])]
    new_len = own_len.clone()  # the last fork's children, which end before the next
    new_len[c["parents"]:] = 0
    return {"refs": refs, "page_table": table, "own_len": own_len, "new_len": new_len, "page": page,
            "src": _i32([i % c["parents"] for i in range(c["children"])]),
            "dst": _i32([c["parents"] + i for i in range(c["children"])]), "wide": pools,
            "pools": [p[:n_pages] for p in pools]}


def _prepare_step(c, g):
    page, Hkv, D, n, B = c["page"], c["Hkv"], c["D"], c["n"], c["B"]
    n_pages = _page_count(c)
    lens = _spread(c["lo"], c["hi"], B)
    refs, table, own_len = _owned(g, lens, B, page, n_pages)
    pools = [torch.randint(0, 256, (n_pages + 1, Hkv, page * (D + D // 16)), generator=g, device=DEVICE,
                           dtype=torch.uint8) for _ in range(c["pools"])]
    return {"refs": refs, "page_table": table, "own_len": own_len, "page": page, "base": own_len.clone(),
            "grown": own_len + n, "keep": _i32([_keep(i, n) for i in range(B)]),
            "kept_len": torch.empty(B, dtype=torch.int32, device=DEVICE), "wide": pools,
            "pools": [p[:n_pages] for p in pools]}


_PREPARE = {"linear_q4": _prepare_linear, "kv4_write": _prepare_write, "prefix_attention_kv4": _prepare_attn,
            "pages_fork": _prepare_fork, "pages_step": _prepare_step}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["op"], s["case"] = case["op"], case
    if own:
        # the weights as laid out once, and the workspace that a user's program keeps next to its buffers
        from moe_ffn_speculative_gb300 import ops
        s["ops"] = ops
        if case["op"] == "linear_q4":
            s["w"] = ops.q4_prepare(s["codes"], s["scales"], s["zeros"])
            n = ops.linear_q4_workspace_bytes(case["M"], case["N"], case["K"])
        elif case["op"] == "kv4_write":
            n = ops.STATUS_BYTES
        elif case["op"] == "prefix_attention_kv4":
            n = ops.prefix_attention_kv4_workspace_bytes(s["q"].shape[0], case["B"], case["Hq"], case["Hkv"], case["D"])
        else:
            n = ops.pages_workspace_bytes(s["page_table"].shape[0], s["refs"].numel())
        s["ws"] = ops.Workspace(n)
    elif case["op"] == "kv4_write":
        # the plain form's cache: the values themselves, and one row more that padding goes to
        D = case["D"]
        codes, scales = _split(s["cache"], D)
        for name, i in (("k_rows", 0), ("v_rows", 1)):
            rows = _expand(codes[i], scales[i]).to(s["k"].dtype).flatten(0, 1)
            s[name] = torch.cat([rows, torch.zeros_like(rows[:1])])
    elif case["op"] == "pages_step":
        # places in a block of one token's bytes: its codes of both kinds, its scales of both
        page, D = case["page"], case["D"]
        half, sc = page * D // 2, page * D // 32
        at = torch.arange(page, device=DEVICE)[:, None]
        code = (torch.arange(D // 32, device=DEVICE)[:, None] * page * 16 + torch.arange(16, device=DEVICE)).flatten()
        scale = torch.arange(D // 32, device=DEVICE)
        s["bytes_of"] = torch.cat([code + at * 16, half + code + at * 16, 2 * half + scale + at * (D // 32),
                                   2 * half + sc + scale + at * (D // 32)], dim=1)
    return s


# ------------------------------------------------------------ the plain forms

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
    codes, scales = s["codes"], s["scales"].float()
    w = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(1).float().unflatten(1, (-1, s["group"]))
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((w - zero) * scales[..., None]).flatten(1)
    v = s["x"].float() @ w.t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _activate(v, s["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    s["y"].copy_(v)
    return s["y"]


def _plain_write(s):
    at = torch.where(s["slots"] < 0, s["rows"], s["slots"]).long()
    for rows, x in ((s["k_rows"], s["k"]), (s["v_rows"], s["v"])):
        rows.index_copy_(0, at, _values(*_encode(x)).to(rows.dtype))
    c = s["case"]
    return tuple(r[:s["rows"]].view(-1, c["page"], c["Hkv"], c["D"]) for r in (s["k_rows"], s["v_rows"]))


def _plain_attn(s):
    c = s["case"]
    T, Hq, D = s["q"].shape
    Hkv, page, P, L, B = c["Hkv"], c["page"], s["P"], s["own_max"], c["B"]
    G = Hq // Hkv
    codes, scales = _split(s["cache"], D)

    def rows(pages, count, i):
        """The first `count` keys (i = 0) or values (1) on lists of pages [..., n]."""
        at = pages[..., :-(-count // page)].long()
        x = _expand(codes[i][at.flatten()], scales[i][at.flatten()])
        return x.view(*at.shape, page, Hkv, D).flatten(-4, -3)[..., :count, :, :]

    q = s["q"].float().view(T, Hkv, G, D) * s["scale"]
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    token = torch.arange(T, device=q.device)
    req = torch.searchsorted(start, token, right=True) - 1
    place = token - start[req]
    score = torch.einsum("thgd,phd->thgp", q, rows(s["prefix_pages"], P, 0))
    # the requests' own keys, padded to the longest, against their blocks, padded to the longest
    blocks = q.new_zeros((B, s["n"], Hkv, G, D))
    blocks[req, place] = q
    own_len = s["own_len"].long()[req]
    seen = (own_len - n[req] + place + 1).clamp(min=0) if s["causal"] else own_len
    own_score = torch.einsum("bnhgd,blhd->bnhgl", blocks, rows(s["page_table"], L, 0))[req, place]
    at = torch.arange(L, device=q.device)
    own_score = own_score.masked_fill((at >= seen[:, None])[:, None, None], float("-inf"))
    score = torch.cat([score, own_score], dim=-1)
    top = score.amax(-1, keepdim=True) if P + L else score.new_full((T, Hkv, G, 1), float("-inf"))
    p = torch.exp(score - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("thgp,phd->thgd", p[..., :P], rows(s["prefix_pages"], P, 1))
    po = p.new_zeros((B, s["n"], Hkv, G, L))
    po[req, place] = p[..., P:]
    out = out + torch.einsum("bnhgl,blhd->bnhgd", po, rows(s["page_table"], L, 1))[req, place]
    s["out"].copy_((out / torch.where(total > 0, total, torch.ones_like(total))).reshape(T, Hq, D))
    s["lse"].copy_((top + total.log()).reshape(T, Hq))
    return s["out"], s["lse"]


def _free_pages(refs):
    """The numbers of the free pages in order (the rest of the list is of no use)."""
    free = refs == 0
    at = torch.where(free, free.cumsum(0) - 1, refs.numel())
    out = torch.zeros(refs.numel() + 1, dtype=torch.int64, device=refs.device)
    out.scatter_(0, at, torch.arange(refs.numel(), device=refs.device))
    return out, free.sum()


def _copy_pages(wide, src, dst, do):
    """Page dst = page src in every pool, where `do` holds."""
    spare = wide[0].shape[0] - 1
    src, dst = torch.where(do, src, spare), torch.where(do, dst, spare)
    for p in wide:
        p[dst] = p[src]


def _plain_resize(s, new_len):
    refs, table, own_len, page = s["refs"], s["page_table"], s["own_len"], s["page"]
    B, width = table.shape
    col = torch.arange(width, device=refs.device)
    old, new = own_len.long(), new_len.long()
    has, want, stay = -(-old // page), -(-new // page), torch.minimum(old, new)
    drop = (col >= want[:, None]) & (col < has[:, None])
    refs.index_add_(0, torch.where(drop, table, 0).flatten(), -drop.flatten().int())
    table.masked_fill_(drop, -1)
    # the page that goes on being written, when another request holds it too, is exchanged for a copy
    tail = stay // page
    last = table.gather(1, tail.clamp(max=width - 1)[:, None])[:, 0].long()
    split = (stay % page != 0) & (refs[last.clamp(min=0)] > 1)
    need = (want - has).clamp(min=0) + split
    pages, free = _free_pages(refs)
    end = need.cumsum(0)
    ok = (end <= free) & (need > 0)
    first = end - need
    split = split & ok
    own = pages[first.clamp(max=refs.numel())]
    refs.index_add_(0, torch.where(split, last, 0), -split.int())
    refs.index_add_(0, torch.where(split, own, 0), split.int())
    table.scatter_(1, tail.clamp(max=width - 1)[:, None],
                   torch.where(split, own, table.gather(1, tail.clamp(max=width - 1)[:, None])[:, 0])[:, None].int())
    take = (col >= has[:, None]) & (col < want[:, None]) & ok[:, None]
    ids = pages[((first + split)[:, None] + col - has[:, None]).clamp(0, refs.numel())]
    refs.index_add_(0, torch.where(take, ids, 0).flatten(), take.flatten().int())
    table.copy_(torch.where(take, ids.int(), table))
    own_len.copy_(torch.where(ok | (need == 0), new, stay))
    _copy_pages(s["wide"], last, own, split)


def _plain_fork(s):
    refs, table, own_len, page = s["refs"], s["page_table"], s["own_len"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device=refs.device)
    length = own_len[src].long()
    whole, tail = length // page, length % page != 0
    pages, free = _free_pages(refs)
    end = tail.long().cumsum(0)
    ok = (end <= free) | ~tail
    tail = tail & ok
    own = pages[(end - 1).clamp(min=0)]
    shared = (col < whole[:, None]) & ok[:, None]
    rows = table[src]
    last = rows.gather(1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    refs.index_add_(0, torch.where(shared, rows, 0).flatten(), shared.flatten().int())
    refs.index_add_(0, torch.where(tail, own, 0), tail.int())
    child = torch.where(shared, rows, table[dst])
    child = torch.where((col == whole[:, None]) & tail[:, None], own[:, None].int(), child)
    table[dst] = child
    own_len[dst] = torch.where(ok, length.int(), own_len[dst])
    _copy_pages(s["wide"], last, own, tail)


def _plain_compact(s):
    table, page, keep = s["page_table"].long(), s["page"], s["keep"].long()
    B, n = keep.shape
    real = keep >= 0
    spare = s["wide"][0].shape[0] - 1

    def place(offset):
        at = s["base"].long()[:, None] + offset
        return torch.where(real, table.gather(1, at // page), spare), at % page

    (sp, so), (dp, do) = place(keep.clamp(min=0)), place(torch.arange(n, device=keep.device).expand(B, n))
    which, heads = s["bytes_of"], torch.arange(s["wide"][0].shape[1], device=keep.device)[:, None]
    for p in s["wide"]:
        moved = p[sp[..., None, None], heads, which[so][:, :, None]]
        p[dp[..., None, None], heads, which[do][:, :, None]] = moved
    s["kept_len"].copy_(s["base"] + real.sum(1))


def _plain_pages(s):
    if s["op"] == "pages_fork":
        _plain_resize(s, s["new_len"])
        _plain_fork(s)
    else:
        _plain_resize(s, s["grown"])
        _plain_compact(s)
        _plain_resize(s, s["kept_len"])


# --------------------------------------------------------- one pass, both forms

def run(s):
    op = s["op"]
    if op in ("pages_fork", "pages_step"):
        if not own:
            _plain_pages(s)
        else:
            ops, args = s["ops"], (s["refs"], s["page_table"], s["own_len"])
            if op == "pages_fork":
                ops.pages_resize(*args, s["new_len"], s["page"], s["ws"], caches=s["pools"])
                ops.pages_fork(*args, s["src"], s["dst"], s["page"], s["ws"], caches=s["pools"])
            else:
                ops.pages_resize(*args, s["grown"], s["page"], s["ws"], caches=s["pools"])
                ops.pages_compact(s["page_table"], s["base"], s["keep"], s["page"], s["ws"], caches=s["pools"],
                                  new_len=s["kept_len"])
                ops.pages_resize(*args, s["kept_len"], s["page"], s["ws"], caches=s["pools"])
        return {"refs": s["refs"], "page_table": s["page_table"], "own_len": s["own_len"], "pools": s["pools"]}
    if not own:
        return {"linear_q4": _plain_linear, "kv4_write": _plain_write, "prefix_attention_kv4": _plain_attn}[op](s)
    ops = s["ops"]
    if op == "linear_q4":
        return ops.linear_q4(s["x"], s["w"], s["ws"], bias=s["bias"], activation=s["act"], residual=s["residual"],
                             y=s["y"])
    if op == "kv4_write":
        ops.kv4_write(s["k"], s["v"], s["slots"], s["cache"], s["ws"])
        return ops.kv4_read(s["cache"], s["k"].shape[2], s["ws"], k=s["k_out"], v=s["v_out"])
    out = ops.prefix_attention_kv4(s["q"], s["cache"], s["q_start"], s["prefix_pages"], s["prefix_len"],
                                   s["page_table"], s["own_len"], s["ws"], causal=s["causal"], scale=s["scale"],
                                   out=s["out"], lse=s["lse"])
    return out, s["lse"]


# ------------------------------------------- the definitions, in 64 bits

def _exact_round(x):
    """x [..., D] in 64 bits as a kv4 cache gives it back."""
    f = x.double().unflatten(-1, (-1, GROUP))
    top = f.abs().amax(-1, keepdim=True)
    power = torch.full_like(top, 2.0 ** (E8M0_LOW - 127))
    for _ in range(E8M0_HIGH - E8M0_LOW):
        power = torch.where(top > 6 * power, 2 * power, power)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    at = (f / power).abs().clamp(max=6)
    up = torch.searchsorted(grid, at).clamp(max=7)         # first code at or above
    down = (up - 1).clamp(min=0)
    a, b = at - grid[down], grid[up] - at
    code = torch.where((a < b) | ((a == b) & (down % 2 == 0)), down, up)
    return (torch.where(f < 0, -grid[code], grid[code]) * power).flatten(-2)


def _exact_cached(cache, D, page, ids, head, which):
    """One head's keys (which = 0) or values (1) on the pages `ids`, in order, in 64 bits."""
    block = cache[ids, head]                               # pages, bytes
    half, sc = page * D // 2, page * D // 32
    raw = block[:, which * half:(which + 1) * half].view(-1, D // 32, page, 16).transpose(1, 2).reshape(-1, D // 2)
    e = block[:, 2 * half + which * sc:2 * half + (which + 1) * sc].reshape(-1, D // 32).double() - 127
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64,
                        device=cache.device) / 2
    out = torch.empty((raw.shape[0], D), dtype=torch.float64, device=cache.device)
    out[:, 0::2], out[:, 1::2] = grid[(raw % 16).long()], grid[(raw // 16).long()]
    return out * torch.repeat_interleave(2.0 ** e, 32, dim=1)


def _exact_attn(case, s):
    f = torch.float64
    T, Hq, D = s["q"].shape
    hkv, page = case["Hkv"], case["page"]
    G = Hq // hkv
    out = torch.zeros((T, Hq, D), dtype=f, device=DEVICE)
    lse = torch.full((T, Hq), float("-inf"), dtype=f, device=DEVICE)
    starts, lens = s["q_start"].tolist(), s["own_len"].tolist()
    for h in range(hkv):

        def rows(pages, count, which):
            ids = pages[:-(-count // page)].long()
            return _exact_cached(s["cache"], D, page, ids, h, which)[:count]

        kp, vp = (rows(s["prefix_pages"], case["P"], i) for i in (0, 1))
        for b, own_len in enumerate(lens):
            t0, t1 = starts[b], starts[b + 1]
            n = t1 - t0
            ko, vo = (rows(s["page_table"][b], own_len, i) for i in (0, 1))
            k, v = torch.cat([kp, ko]), torch.cat([vp, vo])
            if k.shape[0] == 0:
                continue
            q = s["q"][t0:t1, h * G:(h + 1) * G].to(f)     # n, G, D
            logit = (q.reshape(n * G, D) @ k.t() * s["scale"]).view(n, G, -1)
            if s["causal"]:
                last = case["P"] + own_len - n + torch.arange(n, device=DEVICE)
                hidden = torch.arange(k.shape[0], device=DEVICE) > last[:, None]
                logit = logit.masked_fill(hidden[:, None], float("-inf"))
            z = torch.logsumexp(logit, dim=-1, keepdim=True)
            w = torch.where(z == float("-inf"), torch.zeros_like(logit), torch.exp(logit - z))
            out[t0:t1, h * G:(h + 1) * G] = (w.view(n * G, -1) @ v).view(n, G, D)
            lse[t0:t1, h * G:(h + 1) * G] = z[..., 0]
    return out, lse


def exact(case, seed):
    op = case["op"]
    if op.startswith("pages"):
        return None  # whole numbers, and bytes that are only moved
    s = _PREPARE[op](case, _gen(seed))
    f = torch.float64
    if op == "prefix_attention_kv4":
        return _exact_attn(case, s)
    if op == "kv4_write":
        keep = s["slots"] >= 0
        done = []
        for which, x in ((0, s["k"]), (1, s["v"])):
            ids = torch.arange(s["cache"].shape[0], device=DEVICE)
            rows = torch.stack([_exact_cached(s["cache"], case["D"], case["page"], ids, h, which)
                                for h in range(case["Hkv"])], dim=1)
            rows[s["slots"][keep].long()] = _exact_round(x)[keep]
            done.append(rows.view(-1, case["page"], case["Hkv"], case["D"]))
        return tuple(done)
    group = case["group"]
    w = torch.empty((case["N"], case["K"]), dtype=f, device=DEVICE)
    w[:, 0::2], w[:, 1::2] = s["codes"] % 16, s["codes"] // 16
    w -= 8 if s["zeros"] is None else torch.repeat_interleave(s["zeros"].to(f), group, dim=1)
    w *= torch.repeat_interleave(s["scales"].to(f), group, dim=1)
    y = torch.nn.functional.linear(s["x"].to(f), w, None if s["bias"] is None else s["bias"].to(f))
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2))
    elif case["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif case["act"] == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    return y if s["residual"] is None else y + s["residual"].to(f)
