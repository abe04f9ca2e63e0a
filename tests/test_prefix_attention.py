"""moe_prefix_attention: refusals on the host (no GPU), and on the GPU out and
lse of every row against the definition in 64 bits.

Tolerances, derived from the formats.  With w the exact probabilities, N keys
and e = eps of the 16-bit type:
* a logit: a sum of D exact products in fp32, at most
  ds = (D + 4) 2^-24 scale sum|q k| off;
* a probability enters the second product rounded, e/2 of itself off (f16 also
  2^-25 of the row's largest), on top of e^ds and the exponential (2^-21);
* sums over the keys in fp32 (2^-23 a step, tensor cores may truncate);
* the output is rounded once, e/2.
An output may be off by
  e/2 |o| + (e/2 + 2 ds + N 2^-22 + 2^-20) sum w|v| (+ N 2^-25 max|v| + 2^-25 in f16),
and lse by ds + N 2^-23 + 2^-20 + 2^-22 |lse|.  Rounding errors of the many
probabilities are independent, so besides the worst case the 2-norm of the
error is held: two roundings of at most e/2, uniform, are e/sqrt(12) each,
together 0.41 e of the output's norm for values of mean zero; 0.5 e is the bar.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ refusals (no GPU)

def _call(**kw):
    a = dict(q=1 << 20, qs=512, T=4, B=2, start=2 << 20, Hq=4, Hkv=1, D=128, dtype=0, k=3 << 20, v=4 << 20, pages=8,
             page=16, pp=5 << 20, cap=2, pl=6 << 20, table=7 << 20, width=2, own=8 << 20, causal=1, scale=0.1,
             out=9 << 20, lse=None, ws=10 << 20, wb=1 << 40)
    a.update(kw)
    return ops.lib().moe_prefix_attention(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), ops.MOE_ERR_INVALID_ARG), (dict(B=-1), ops.MOE_ERR_INVALID_ARG),
    (dict(Hkv=0), ops.MOE_ERR_INVALID_ARG), (dict(Hkv=3), ops.MOE_ERR_INVALID_ARG),
    (dict(dtype=2), ops.MOE_ERR_INVALID_ARG), (dict(causal=2), ops.MOE_ERR_INVALID_ARG),
    (dict(scale=0.0), ops.MOE_ERR_INVALID_ARG), (dict(scale=NAN), ops.MOE_ERR_INVALID_ARG),
    (dict(scale=float("inf")), ops.MOE_ERR_INVALID_ARG), (dict(pages=-1), ops.MOE_ERR_INVALID_ARG),
    (dict(pages=0), ops.MOE_ERR_INVALID_ARG), (dict(q=None), ops.MOE_ERR_INVALID_ARG),
    (dict(out=None), ops.MOE_ERR_INVALID_ARG), (dict(out=1 << 20), ops.MOE_ERR_INVALID_ARG),
    (dict(start=None), ops.MOE_ERR_INVALID_ARG), (dict(pp=None), ops.MOE_ERR_INVALID_ARG),
    (dict(pl=None), ops.MOE_ERR_INVALID_ARG), (dict(table=None), ops.MOE_ERR_INVALID_ARG),
    (dict(own=None), ops.MOE_ERR_INVALID_ARG), (dict(k=None), ops.MOE_ERR_INVALID_ARG),
    (dict(v=(4 << 20) + 8), ops.MOE_ERR_INVALID_ARG),
    (dict(D=96), ops.MOE_ERR_UNSUPPORTED), (dict(page=24), ops.MOE_ERR_UNSUPPORTED),
    (dict(page=4), ops.MOE_ERR_UNSUPPORTED), (dict(page=2048), ops.MOE_ERR_UNSUPPORTED),
    (dict(Hq=129, Hkv=1), ops.MOE_ERR_UNSUPPORTED), (dict(qs=516), ops.MOE_ERR_UNSUPPORTED),
    (dict(cap=1 << 25), ops.MOE_ERR_UNSUPPORTED), (dict(width=1 << 25), ops.MOE_ERR_UNSUPPORTED),
    (dict(B=65537), ops.MOE_ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), ops.MOE_ERR_UNSUPPORTED),
    (dict(ws=None), ops.MOE_ERR_WORKSPACE), (dict(ws=(10 << 20) + 128), ops.MOE_ERR_WORKSPACE),
    (dict(wb=4096), ops.MOE_ERR_WORKSPACE),
    (dict(T=0, q=None, out=None, ws=None), ops.MOE_OK),
])
def test_refusals(change, status):
    assert _call(**change) == status


def test_workspace_query_refuses_bad_shapes():
    assert ops.lib().moe_prefix_attention_workspace_bytes(4, 1, 5, 2, 128) == 0
    assert ops.lib().moe_prefix_attention_workspace_bytes(4, 1, 4, 2, 80) == 0
    assert ops.lib().moe_prefix_attention_workspace_bytes(-1, 1, 4, 2, 64) == 0


# ------------------------------------------------------------------ values (GPU)

class Batch:
    """Inputs of one call: `blocks` lists (tokens, own keys) of each request."""

    def __init__(self, Hq, Hkv, D, dtype, page, P, blocks, seed=0, pad=(0, 0), amplify=1.0, fill=NAN, strided=False):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(dtype)
        self.page, self.P, self.blocks, self.Hkv = page, P, blocks, Hkv
        start = [pad[0]]
        for n, _ in blocks:
            start.append(start[-1] + n)
        self.start = start
        T = start[-1] + pad[1]
        self.q = normal(T, Hq + 3, D)[:, :Hq] if strided else normal(T, Hq, D)
        self.q *= amplify
        need = [-(-P // page)] + [-(-own // page) for _, own in blocks]
        width = max(need[1:], default=0) + 1  # one page more than the longest needs
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        # every slot that no length covers holds `fill`
        self.k = torch.full((pages, page, Hkv, D), fill, device="cuda", dtype=dtype)
        self.v = torch.full((pages, page, Hkv, D), fill, device="cuda", dtype=dtype)
        spare = int(order[-1])
        at = 0
        self.keys = []
        lists = []
        for cnt, length in zip(need, [P] + [own for _, own in blocks]):
            ids = order[at:at + cnt].long()
            at += cnt
            k, v = normal(length, Hkv, D), normal(length, Hkv, D)
            idx = torch.arange(length, device="cuda")
            self.k[ids[idx // page], idx % page] = k
            self.v[ids[idx // page], idx % page] = v
            self.keys.append((k, v))
            lists.append(ids.to(torch.int32))
        self.prefix_pages = lists[0] if P else torch.full((1,), spare, device="cuda", dtype=torch.int32)
        self.table = torch.full((len(blocks), width), spare, device="cuda", dtype=torch.int32)
        for b, ids in enumerate(lists[1:]):
            self.table[b, :ids.numel()] = ids

        def i32(x):
            return torch.tensor(x, device="cuda", dtype=torch.int32)
        self.prefix_len, self.own = i32([P]), i32([own for _, own in blocks])
        self.q_start = i32(start)
        self.ws = ops.Workspace(ops.prefix_attention_workspace_bytes(T, len(blocks), Hq, Hkv, D))

    def run(self, causal, lse=True, scale=None, **kw):
        T, Hq, _ = self.q.shape
        z = torch.full((T, Hq), 5.0, device="cuda") if lse else None
        out = torch.full(self.q.shape, 3.0, device="cuda", dtype=self.q.dtype)
        o = ops.prefix_attention(self.q, self.k, self.v, self.q_start, self.prefix_pages, self.prefix_len, self.table,
                                 self.own, self.ws, causal=causal, scale=scale, out=out, lse=z, **kw)
        assert o is out
        return out, z

    def exact(self, causal, scale):
        """(out, lse, tolerance of out, of lse) in 64 bits."""
        T, Hq, D = self.q.shape
        G = Hq // self.Hkv
        eps = torch.finfo(self.q.dtype).eps
        half = 2.0 ** -25 if self.q.dtype == torch.float16 else 0.0
        out = torch.zeros((T, Hq, D), device="cuda", dtype=torch.float64)
        lse = torch.full((T, Hq), float("-inf"), device="cuda", dtype=torch.float64)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        kp, vp = self.keys[0]
        for b, (n, own) in enumerate(self.blocks):
            ko, vo = self.keys[b + 1]
            for i in range(n):
                t = self.start[b] + i
                seen = max(0, own - n + i + 1) if causal else own
                N = self.P + seen
                if N == 0:
                    continue
                k, v = (torch.cat(x).double().repeat_interleave(G, dim=1)
                        for x in ((kp, ko[:seen]), (vp, vo[:seen])))
                q = self.q[t].double()
                prod = q * k
                s = prod.sum(-1) * scale                                      # [N, Hq]
                ds = (D + 4) * 2.0 ** -24 * scale * prod.abs().sum(-1).amax(0)  # [Hq]
                lse[t] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[t])
                out[t] = torch.einsum("nh,nhd->hd", w, v)
                mass = torch.einsum("nh,nhd->hd", w, v.abs())
                tol[t] = (eps / 2 * out[t].abs() + (eps / 2 + 2 * ds[:, None] + N * 2.0 ** -22 + 2.0 ** -20) * mass
                          + (N * half * v.abs().amax(0) + half))
                tol_lse[t] = ds + N * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * lse[t].abs()
        return out, lse, tol, tol_lse

    def check(self, causal, scale=None, norm=True):
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        got, z = self.run(causal, scale=scale)
        assert self.ws.device_status() == (ops.MOE_OK, 0)
        out, lse, tol, tol_lse = self.exact(causal, scale)
        assert bool(torch.isfinite(got).all())
        off = (got.double() - out).abs()
        assert bool((off <= tol).all()), f"{(off > tol).sum().item()} of {off.numel()} outputs, worst {off.max().item()}"
        empty = torch.isinf(lse)
        assert torch.equal(empty, torch.isinf(z)) and bool((z[empty] < 0).all())
        assert bool(((z.double() - lse).abs() <= tol_lse)[~empty].all())
        if norm and out.norm() > 0:
            assert (got.double() - out).norm() <= 0.5 * torch.finfo(got.dtype).eps * out.norm()
        return got


BF, HF = torch.bfloat16, torch.float16
CASES = {
    # name: (Hq, Hkv, D, dtype, page, causal, P, [(tokens, own keys)])
    "one_key": (1, 1, 64, BF, 8, True, 0, [(1, 1)]),
    "nothing": (4, 2, 128, BF, 16, True, 0, [(1, 0), (3, 0)]),
    "prefix_of_one": (4, 2, 128, HF, 16, False, 1, [(1, 0)]),
    "single_tokens": (32, 8, 128, BF, 64, True, 640, [(1, 5), (1, 37), (1, 100), (1, 1)]),
    "verify_blocks": (32, 8, 128, BF, 64, True, 1000, [(9, 9), (9, 100), (9, 129), (9, 300)]),
    "verify_fp16": (32, 8, 128, HF, 16, True, 257, [(9, 128), (9, 127), (9, 12)]),
    "draft_blocks": (40, 8, 64, HF, 16, False, 515, [(8, 8), (1, 0), (5, 77), (8, 256)]),
    "d64_causal": (8, 2, 64, BF, 32, True, 130, [(4, 60), (16, 16), (2, 200)]),
    "no_groups": (16, 16, 64, BF, 128, True, 200, [(3, 140), (7, 9)]),
    "groups_of_seven": (28, 4, 128, BF, 32, True, 384, [(9, 40), (4, 64)]),
    "one_key_head": (64, 1, 128, BF, 16, True, 100, [(3, 33), (2, 2)]),
    "widest_group": (128, 1, 64, HF, 16, True, 140, [(2, 10), (1, 3)]),
    "no_prefix": (8, 2, 128, BF, 16, True, 0, [(5, 5), (1, 300), (9, 128)]),
    "prompts": (8, 2, 128, BF, 64, True, 100, [(200, 200), (77, 400)]),
    "prompts_bidirectional": (4, 2, 64, HF, 16, False, 0, [(150, 150), (33, 33)]),
    "fewer_own_than_tokens": (8, 2, 128, BF, 16, True, 0, [(9, 3), (4, 1)]),
    "fewer_own_with_prefix": (8, 2, 64, BF, 16, True, 33, [(9, 3), (4, 0)]),
    "empty_blocks": (8, 2, 128, BF, 16, True, 150, [(0, 50), (2, 20), (0, 0), (3, 300), (0, 10)]),
    "big_pages": (8, 2, 128, BF, 1024, True, 1500, [(2, 1030), (1, 5)]),
    "small_pages": (8, 2, 128, HF, 8, True, 133, [(2, 77), (1, 5)]),
    "many_requests": (8, 2, 64, BF, 16, True, 300, [(1 + i % 3, 1 + 7 * i % 90) for i in range(70)]),
    "rows_past_two_tiles": (32, 4, 128, BF, 64, True, 700, [(9, 30 + i) for i in range(8)]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_against_definition(name):
    Hq, Hkv, D, dtype, page, causal, P, blocks = CASES[name]
    Batch(Hq, Hkv, D, dtype, page, P, blocks, seed=len(name)).check(causal)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 400, 1100])
def test_many_blocks(B):
    """More requests than a block of threads looks at in one step."""
    Batch(2, 1, 64, BF, 8, 40, [(i % 2, (5 * i) % 40) for i in range(B)], seed=B).check(True)


@pytest.mark.gpu
def test_many_tiles_per_row_tile():
    """A long context for few rows: split over every SM and joined."""
    Batch(8, 2, 128, BF, 64, 20000, [(4, 5000), (2, 7)], seed=2).check(True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sharp_rows_and_scale(dtype):
    """Logits of tens: the running maximum moves far between tiles.  The
    probabilities gather on few keys, so only the worst case is held."""
    b = Batch(8, 2, 64, dtype, 16, 700, [(5, 300), (1, 40)], seed=9, amplify=6.0)
    b.check(True, norm=False)
    b.check(False, scale=0.5, norm=False)


@pytest.mark.gpu
def test_descending_and_ascending_logits():
    """Keys sorted by their logit, both ways, over many tiles."""
    for sign in (1, -1):
        b = Batch(2, 1, 64, BF, 16, 2000, [(1, 200)], seed=4)
        k, v = b.keys[0]
        ramp = torch.linspace(-40 * sign, 40 * sign, 2000, device="cuda").to(BF)
        k.zero_()
        k[:, 0, 0] = ramp
        b.q.zero_()
        b.q[..., 0] = 8.0
        idx = torch.arange(2000, device="cuda")
        b.k[b.prefix_pages.long()[idx // 16], idx % 16] = k
        b.check(True, norm=False)


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [NAN, float("inf"), float("-inf")])
def test_uncovered_slots_hold_anything(fill):
    Batch(8, 2, 128, BF, 64, 130, [(3, 65), (2, 1)], seed=5, fill=fill).check(True)
    Batch(8, 2, 64, HF, 128, 1, [(3, 3), (2, 127)], seed=6, fill=fill).check(False)


@pytest.mark.gpu
def test_padding_tokens_strided_rows_no_lse():
    b = Batch(8, 2, 128, BF, 16, 90, [(4, 20), (3, 44)], seed=7, pad=(3, 5), strided=True)
    b.q[:3] = NAN  # padding rows may hold anything
    b.q[-5:] = NAN
    got = b.check(True)
    assert bool((got[:3] == 0).all()) and bool((got[-5:] == 0).all())
    assert torch.equal(b.run(True, lse=False)[0], got)


@pytest.mark.gpu
def test_same_bits_again_other_stream_and_graph():
    """The split does not depend on timing; lengths may change between replays
    of a captured call."""
    b = Batch(32, 8, 128, BF, 64, 3000, [(9, 100), (9, 500), (9, 77)], seed=8)
    want, z = b.run(True)
    for _ in range(3):
        again, z2 = b.run(True)
        assert torch.equal(again, want) and torch.equal(z, z2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other, _ = b.run(True)
    s.synchronize()
    assert torch.equal(other, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.prefix_attention(b.q, b.k, b.v, b.q_start, b.prefix_pages, b.prefix_len, b.table, b.own, b.ws, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    b.own.copy_(torch.tensor([90, 17, 60], dtype=torch.int32))
    b.prefix_len.fill_(1234)
    direct, _ = b.run(True)
    assert not torch.equal(direct, want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, direct)


@pytest.mark.gpu
def test_workspace_shared_with_the_layer():
    """The workspace header that the FFN's counters live in is left alone, and
    nothing is written outside the workspace or the outputs."""
    b = Batch(8, 2, 128, BF, 64, 500, [(4, 100), (4, 30)], seed=10)
    margin = 1 << 16
    full = torch.full((b.ws.nbytes + 2 * margin,), 0xA5, device="cuda", dtype=torch.uint8)
    b.ws.buf = full[margin:margin + b.ws.nbytes]
    b.ws.buf.zero_()
    b.check(True)
    assert bool((full[:margin] == 0xA5).all()) and bool((full[-margin:] == 0xA5).all())
    assert bool((b.ws.buf[:64 * 1024] == 0).all())


@pytest.mark.gpu
def test_indexes_outside_their_tables():
    """Bad pages read as zeros, bad lengths are held within their tables, blocks
    out of order leave the other requests as they are; each is recorded."""
    b = Batch(8, 2, 64, BF, 16, 64, [(2, 20), (3, 33)], seed=11)
    want, _ = b.run(True)
    for bad in (-1, b.k.shape[0], 2 ** 31 - 1):
        page = b.table[1, 0].item()
        b.table[1, 0] = bad
        got, _ = b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_PAGE)
        assert torch.equal(got[:2], want[:2]) and not torch.equal(got[2:], want[2:])
        b.table[1, 0] = page
        kept = b.keys[2]
        k, v = kept[0].clone(), kept[1].clone()
        k[:16], v[:16] = 0, 0
        b.keys[2] = (k, v)
        out, _, tol, _ = b.exact(True, 64 ** -0.5)
        assert bool(((got.double() - out).abs() <= tol).all())
        b.keys[2] = kept
    keep = b.own.clone()
    for bad in (-1, b.table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        b.own[0] = bad
        got, _ = b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_LENGTH)
        assert torch.equal(got[2:], want[2:])
    b.own.copy_(keep)
    for bad in (65, -5):
        b.prefix_len.fill_(bad)
        b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_LENGTH)
    b.prefix_len.fill_(64)
    for bad in (-1, 4, 100):  # request 0: negative, past its end (request 1's start), past T
        b.q_start[0] = bad
        b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_STARTS)
    b.q_start[0] = 0
    assert torch.equal(b.run(True)[0], want)
    assert b.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_no_requests_and_no_pages():
    """A batch without requests, without a prefix or without own pages."""
    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.randn((5, 4, 64), device="cuda").to(BF)
    k = torch.randn((3, 8, 2, 64), device="cuda").to(BF)
    ws = ops.Workspace(ops.prefix_attention_workspace_bytes(5, 2, 4, 2, 64))
    lse = torch.zeros((5, 4), device="cuda")
    out = ops.prefix_attention(q, k, k, i32(0), i32(1), i32(8), None, None, ws, lse=lse)  # B = 0: all padding
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    out = ops.prefix_attention(q, k, k, i32(0, 2, 5), None, None, None, None, ws, lse=lse)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    only_prefix = ops.prefix_attention(q, k, k, i32(0, 2, 5), i32(1, 2), i32(11), None, None, ws)
    keys = k[1:3].flatten(0, 1)[:11].double().repeat_interleave(2, 1)
    z = torch.einsum("nhd,mhd->hnm", q.double(), keys) * 64 ** -0.5
    want = torch.einsum("hnm,mhd->nhd", z.softmax(-1), keys)
    assert (only_prefix.double() - want).norm() <= 0.5 * torch.finfo(BF).eps * want.norm()
    assert ws.device_status() == (ops.MOE_OK, 0)
    empty = ops.prefix_attention(q[:0], k, k, i32(0, 0, 0), i32(1), i32(8), None, None, ws)
    assert empty.shape == (0, 4, 64)


@pytest.mark.gpu
def test_pages_past_32_bit_offsets():
    """The pool holds more than 2^31 elements and the batch's pages lie at its
    end."""
    page, Hkv, D = 64, 8, 128
    pages = 2 ** 31 // (page * Hkv * D) + 40
    b = Batch(32, Hkv, D, BF, page, 300, [(9, 100), (4, 20)], seed=21)
    far = torch.arange(b.k.shape[0], device="cuda") + pages - b.k.shape[0]
    for name in ("k", "v"):
        pool = torch.zeros((pages, page, Hkv, D), device="cuda", dtype=BF)
        pool[far] = getattr(b, name)
        setattr(b, name, pool)
    shift = pages - far.numel()
    b.prefix_pages = b.prefix_pages + shift
    b.table = b.table + shift
    b.check(True)


@pytest.mark.gpu
@pytest.mark.parametrize("D,causal", [(128, True), (64, False)])
def test_long_prompts(D, causal):
    """Thousands of tokens against a thousand keys each: every row tile and
    every tile of keys, by norms (the exact rows head by head)."""
    b = Batch(8, 2, D, BF, 64, 200, [(1500, 1700), (3, 90), (700, 700)], seed=31)
    got, lse = b.run(causal)
    kp, vp = b.keys[0]
    for r, (n, own) in enumerate(b.blocks):
        t0 = b.start[r]
        k, v = (torch.cat(x).double() for x in ((kp, b.keys[r + 1][0]), (vp, b.keys[r + 1][1])))
        seen = 200 + (own - n + torch.arange(n, device="cuda") + 1 if causal else torch.full((n,), own, device="cuda"))
        for h in range(8):
            z = b.q[t0:t0 + n, h].double() @ k[:, h // 4].t() * D ** -0.5
            z = z.masked_fill(torch.arange(k.shape[0], device="cuda") >= seen[:, None], float("-inf"))
            want = z.softmax(-1) @ v[:, h // 4]
            off = (got[t0:t0 + n, h].double() - want).norm(dim=-1) / want.norm(dim=-1)
            # a row's error is a mean over D elements of two roundings of at most e/2
            assert off.max() <= torch.finfo(BF).eps
            assert (lse[t0:t0 + n, h].double() - torch.logsumexp(z, -1)).abs().max() <= 1e-4
