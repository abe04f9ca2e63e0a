"""moe_prefix_attention_kv4: refusals on the host (no GPU), and on the GPU out and lse
of every row against the definition in 64 bits on the numbers that the codes stand for.

Tolerances: those of the 16-bit attention (test_prefix_attention), but that the
probabilities are f16 whatever the inputs' type: each is 2^-11 of itself off, and 2^-32
of the row's largest.  An output may be off by
  e/2 |o| + (2^-11 + 2 ds + N 2^-22 + 2^-20) sum w|v| + N 2^-32 max|v| (+ 2^-25 in f16).
The 2-norm: the output's rounding is e/sqrt(12) of it and the probabilities' at most
2^-10/sqrt(12), together 0.41 e in f16 and 0.31 e in bf16; 0.5 e is the bar.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_prefix_attention import BF, CASES, HF, NAN, Batch


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ refusals (no GPU)

def _call(**kw):
    a = dict(q=1 << 30, qs=512, T=4, B=2, start=2 << 30, Hq=4, Hkv=1, D=128, dtype=0, cache=3 << 30, pages=8, page=16,
             pp=5 << 30, cap=2, pl=6 << 30, table=7 << 30, width=2, own=8 << 30, causal=1, scale=0.1, out=9 << 30,
             lse=None, ws=10 << 30, wb=1 << 40)
    a.update(kw)
    return ops.lib().moe_prefix_attention_kv4(*a.values(), None)


INVALID, UNSUPPORTED, WORKSPACE = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID),
    (dict(dtype=2), INVALID), (dict(causal=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(pages=-1), INVALID), (dict(pages=0), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(out=1 << 30), INVALID), (dict(start=None), INVALID), (dict(pp=None), INVALID),
    (dict(pl=None), INVALID), (dict(table=None), INVALID), (dict(own=None), INVALID), (dict(cache=None), INVALID),
    (dict(cache=(3 << 30) + 8), INVALID), (dict(out=3 << 30), INVALID), (dict(lse=3 << 30), INVALID),
    (dict(lse=9 << 30), INVALID), (dict(qs=504), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=4), UNSUPPORTED),
    (dict(page=2048), UNSUPPORTED), (dict(Hq=65, Hkv=1), UNSUPPORTED), (dict(qs=516), UNSUPPORTED),
    (dict(cap=1 << 25), UNSUPPORTED), (dict(width=1 << 25), UNSUPPORTED), (dict(B=65537), UNSUPPORTED),
    (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(pages=1 << 27), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=(10 << 30) + 128), WORKSPACE), (dict(wb=4096), WORKSPACE),
    (dict(T=0, q=None, out=None, ws=None), ops.MOE_OK),
])
def test_refusals(change, status):
    assert _call(**change) == status


def test_workspace_query_refuses_bad_shapes():
    for bad in ((4, 1, 5, 2, 128), (4, 1, 4, 2, 80), (-1, 1, 4, 2, 64), (4, 1, 130, 2, 64)):
        assert ops.lib().moe_prefix_attention_kv4_workspace_bytes(*bad) == 0


def test_tensors_that_are_not_on_a_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        ops.prefix_attention_kv4(torch.zeros((1, 1, 64)), None, None, None, None, None, None, None)


# ------------------------------------------------------------------ values (GPU)

class Batch4(Batch):
    """A batch whose keys and values lie in a kv4 cache; bytes that no length covers
    are `fill`."""

    def __init__(self, Hq, Hkv, D, dtype, page, P, blocks, fill4=0xff, spread=0, **kw):
        super().__init__(Hq, Hkv, D, dtype, page, P, blocks, fill=0.0, **kw)
        T = self.q.shape[0]
        if spread:  # keys and values of every magnitude, a factor a group of 32 channels
            g = torch.Generator(device="cuda").manual_seed(99)
            for x in (self.k, self.v):
                f = torch.randint(-spread, spread + 1, (*x.shape[:-1], D // 32, 1), generator=g, device="cuda")
                x.copy_((x.unflatten(-1, (-1, 32)).float() * 2.0 ** f).flatten(-2))
        pages = self.k.shape[0]
        ws = ops.Workspace(ops.STATUS_BYTES)
        self.cache = torch.full(ops.kv4_shape(pages, page, Hkv, D), fill4, device="cuda", dtype=torch.uint8)
        lists = [(self.prefix_pages, P)] + [(self.table[b], own) for b, (_, own) in enumerate(blocks)]
        for i, (ids, n) in enumerate(lists):
            at = torch.arange(n, device="cuda")
            slots = (ids.long()[at // page] * page + at % page).to(torch.int32)
            k, v = (x[ids.long()[at // page], at % page] for x in (self.k, self.v))
            if n:
                ops.kv4_write(k, v, slots, self.cache, ws)
            kk, vv = ops.kv4_read(self.cache, D, ws, dtype=BF)  # (exactly what the codes stand for)
            self.keys[i] = tuple(x.flatten(0, 1)[slots.long()].double() for x in (kk, vv))
        assert ws.device_status() == (ops.MOE_OK, 0)
        del self.k, self.v
        self.ws = ops.Workspace(ops.prefix_attention_kv4_workspace_bytes(T, len(blocks), Hq, Hkv, D))

    def run(self, causal, lse=True, scale=None, **kw):
        T, Hq, _ = self.q.shape
        z = torch.full((T, Hq), 5.0, device="cuda") if lse else None
        out = torch.full(self.q.shape, 3.0, device="cuda", dtype=self.q.dtype)
        o = ops.prefix_attention_kv4(self.q, self.cache, self.q_start, self.prefix_pages, self.prefix_len, self.table,
                                     self.own, self.ws, causal=causal, scale=scale, out=out, lse=z, **kw)
        assert o is out
        return out, z

    def exact(self, causal, scale):
        T, Hq, D = self.q.shape
        G = Hq // self.Hkv
        eps = torch.finfo(self.q.dtype).eps
        half = 2.0 ** -25 if self.q.dtype == HF else 0.0
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
                k, v = (torch.cat(x).repeat_interleave(G, dim=1) for x in ((kp, ko[:seen]), (vp, vo[:seen])))
                q = self.q[t].double()
                prod = q * k
                s = prod.sum(-1) * scale                                      # [N, Hq]
                ds = (D + 4) * 2.0 ** -24 * scale * prod.abs().sum(-1).amax(0)  # [Hq]
                lse[t] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[t])
                out[t] = torch.einsum("nh,nhd->hd", w, v)
                mass = torch.einsum("nh,nhd->hd", w, v.abs())
                tol[t] = (eps / 2 * out[t].abs() + (2.0 ** -11 + 2 * ds[:, None] + N * 2.0 ** -22 + 2.0 ** -20) * mass
                          + (N * 2.0 ** -32 * v.abs().amax(0) + half))
                tol_lse[t] = ds + N * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * lse[t].abs()
        return out, lse, tol, tol_lse


CASES4 = {n: c for n, c in CASES.items() if c[0] // c[1] <= 64}
CASES4["sixty_four_of_a_head"] = (64, 1, 64, HF, 16, True, 140, [(2, 10), (1, 3)])
CASES4["three_of_a_tile"] = (42, 2, 128, BF, 16, True, 300, [(7, 200), (4, 129)])


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES4))
def test_against_definition(name):
    Hq, Hkv, D, dtype, page, causal, P, blocks = CASES4[name]
    Batch4(Hq, Hkv, D, dtype, page, P, blocks, seed=len(name)).check(causal)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 31, 32, 33, 500, 1100])
def test_many_blocks(B):
    """More requests than a block of threads looks at in one step."""
    Batch4(2, 1, 64, BF, 8, 40, [(i % 2, (5 * i) % 40) for i in range(B)], seed=B).check(True)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 12, 13, 16])
def test_every_width_over_a_shared_prefix(n):
    """Row tiles of 4 to 64 rows over own keys of none to four tiles, behind a prefix that
    keeps them with the kernel for many rows."""
    Batch4(8, 2, 64, HF, 32, 1500, [(n, max(n, own)) for own in (0, 10, 127, 128, 129, 256, 300, 400)], seed=n).check(True)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [64, 16, 512])
def test_many_tiles_per_row_tile(page):
    """A long context for few rows: split over every SM and joined."""
    Batch4(8, 2, 128, BF, page, 20000, [(4, 5000), (2, 7)], seed=2).check(True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sharp_rows_and_scale(dtype):
    """Logits of tens: the reference moves often.  The probabilities gather on few
    keys, so only the worst case is held."""
    b = Batch4(8, 2, 64, dtype, 16, 700, [(5, 300), (1, 40)], seed=9, amplify=6.0)
    b.check(True, norm=False)
    b.check(False, scale=0.5, norm=False)
    b.check(False, scale=3.0, norm=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
def test_magnitudes(dtype, D):
    """Scales of neighbouring groups that differ by up to 2^16, and query rows from
    very small to very large."""
    b = Batch4(8, 2, D, dtype, 16, 300, [(5, 200), (3, 40)], seed=19, spread=8)
    b.q *= 2.0 ** torch.randint(-12, 3, (b.q.shape[0], 8, 1), device="cuda")
    b.check(True, scale=2.0 ** -8, norm=False)
    if dtype == BF:
        b.q[0] *= 2.0 ** 100
        b.q[1] = 0
        b.q[2] *= 2.0 ** -110
        b.q[3, :, 7] = 2.0 ** 90
        b.check(False, scale=2.0 ** -120, norm=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_descending_and_ascending_logits(dtype):
    """Keys sorted by their logit, both ways, over many tiles."""
    for sign in (1, -1):
        b = Batch4(2, 1, 64, dtype, 16, 2000, [(1, 200)], seed=4)
        ramp = torch.linspace(-40 * sign, 40 * sign, 2000, device="cuda").to(BF)
        k = torch.zeros((2000, 1, 64), device="cuda", dtype=BF)
        k[:, 0, 0] = ramp
        v = torch.randn((2000, 1, 64), device="cuda").to(BF)
        idx = torch.arange(2000, device="cuda")
        slots = (b.prefix_pages.long()[idx // 16] * 16 + idx % 16).to(torch.int32)
        ops.kv4_write(k, v, slots, b.cache, b.ws)
        kk, vv = ops.kv4_read(b.cache, 64, b.ws)
        b.keys[0] = tuple(x.flatten(0, 1)[slots.long()].double() for x in (kk, vv))
        b.q.zero_()
        b.q[..., 0] = 8.0
        b.check(True, norm=False)


@pytest.mark.gpu
def test_a_mass_of_small_probabilities():
    """One key far above very many others that weigh as much together."""
    N = 60000
    b = Batch4(1, 1, 64, HF, 64, N, [(1, 1)], seed=3)
    k = torch.zeros((N, 1, 64), device="cuda", dtype=HF)
    k[777, 0, 0] = 11.0  # e^11 = 59874
    v = torch.where(torch.arange(N, device="cuda") == 777, -1.0, 1.0).to(HF)[:, None, None].expand(N, 1, 64).contiguous()
    idx = torch.arange(N, device="cuda")
    slots = (b.prefix_pages.long()[idx // 64] * 64 + idx % 64).to(torch.int32)
    ops.kv4_write(k, v, slots, b.cache, b.ws)
    kk, vv = ops.kv4_read(b.cache, 64, b.ws)
    b.keys[0] = tuple(x.flatten(0, 1)[slots.long()].double() for x in (kk, vv))
    b.q.zero_()
    b.q[..., 0] = 1.0
    b.check(True, scale=1.0, norm=False)


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [0xff, 0x7f, 0x00])
def test_uncovered_slots_hold_anything(fill):
    """Codes of any value with scales of NaN (0xff), 1 and below the range."""
    Batch4(8, 2, 128, BF, 64, 130, [(3, 65), (2, 1)], seed=5, fill4=fill).check(True)
    Batch4(8, 2, 64, HF, 128, 1, [(3, 3), (2, 127)], seed=6, fill4=fill).check(False)
    Batch4(8, 2, 128, HF, 512, 300, [(3, 3), (2, 127)], seed=6, fill4=fill).check(False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_what_is_not_finite(dtype):
    """A NaN group, and infinities and NaN in queries, reach their rows only."""
    b = Batch4(8, 2, 64, dtype, 16, 200, [(3, 50), (2, 60)], seed=12)
    want, _ = b.run(True)
    b.q[0, 1, 3], b.q[1, 2, 5], b.q[2, 7, 0] = float("inf"), NAN, float("-inf")
    got, _ = b.run(True)
    clean = torch.ones_like(want, dtype=torch.bool)
    clean[0, 1], clean[1, 2], clean[2, 7] = False, False, False
    assert torch.equal(got[clean], want[clean]) and got[1, 2].isnan().all()
    k = torch.full((1, 2, 64), 1.0, device="cuda", dtype=dtype)
    bad = k.clone()
    bad[:, 1] = NAN
    slot = b.table[1, 0] * 16 + 5
    ops.kv4_write(bad, k, slot[None], b.cache, b.ws)
    assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_RANGE, ops.INFO_KV_RANGE)
    again, lse = b.run(True)
    assert torch.equal(again[:3], got[:3], ) or torch.equal(again[:3].nan_to_num(), got[:3].nan_to_num())
    assert again[3:, 4:].isnan().all() and lse[3:, 4:].isnan().all() and torch.isfinite(again[3:, :4]).all()
    assert b.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_padding_tokens_strided_rows_no_lse():
    b = Batch4(8, 2, 128, BF, 16, 90, [(4, 20), (3, 44)], seed=7, pad=(3, 5), strided=True)
    b.q[:3] = NAN  # padding rows may hold anything
    b.q[-5:] = NAN
    got = b.check(True)
    assert bool((got[:3] == 0).all()) and bool((got[-5:] == 0).all())
    assert torch.equal(b.run(True, lse=False)[0], got)


@pytest.mark.gpu
def test_same_bits_again_other_stream_and_graph():
    """The split does not depend on timing; lengths may change between replays of a
    captured call."""
    b = Batch4(32, 8, 128, BF, 64, 3000 + 1, [(9, 100), (9, 500), (9, 77)], seed=8)
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
        ops.prefix_attention_kv4(b.q, b.cache, b.q_start, b.prefix_pages, b.prefix_len, b.table, b.own, b.ws, out=out)
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
def test_workspace_and_its_neighbours():
    """Nothing is written outside the workspace, its header apart from the status is
    left alone, and a size serves every smaller call."""
    b = Batch4(8, 2, 128, BF, 64, 500, [(4, 100), (4, 30)], seed=10)
    margin = 1 << 16
    n = ops.prefix_attention_kv4_workspace_bytes(9, 5, 8, 2, 128)
    assert n >= b.ws.nbytes
    full = torch.full((b.ws.nbytes + 2 * margin,), 0xA5, device="cuda", dtype=torch.uint8)
    b.ws.buf = full[margin:margin + b.ws.nbytes]
    b.ws.buf.zero_()
    b.check(True)
    assert bool((full[:margin] == 0xA5).all()) and bool((full[-margin:] == 0xA5).all())
    assert bool((b.ws.buf[:64 * 1024] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 256])
def test_indexes_outside_their_tables(page):
    """Bad pages read as zeros, bad lengths are held within their tables, blocks out of
    order leave the other requests as they are; each is recorded."""
    b = Batch4(8, 2, 64, BF, page, 4 * page, [(2, 20), (3, page + 17)], seed=11)
    want, _ = b.run(True)
    for bad in (-1, b.cache.shape[0], 2 ** 31 - 1):
        page_id = b.table[1, 0].item()
        b.table[1, 0] = bad
        got, _ = b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_PAGE)
        assert torch.equal(got[:2], want[:2]) and not torch.equal(got[2:], want[2:])
        b.table[1, 0] = page_id
        kept = b.keys[2]
        k, v = kept[0].clone(), kept[1].clone()
        k[:page], v[:page] = 0, 0
        b.keys[2] = (k, v)
        out, _, tol, _ = b.exact(True, 64 ** -0.5)
        assert bool(((got.double() - out).abs() <= tol).all())
        b.keys[2] = kept
    keep = b.own.clone()
    for bad in (-1, b.table.shape[1] * page + 1, 2 ** 31 - 1, -2 ** 31):
        b.own[0] = bad
        got, _ = b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_LENGTH)
        assert torch.equal(got[2:], want[2:])
    b.own.copy_(keep)
    for bad in (4 * page + 1, -5):
        b.prefix_len.fill_(bad)
        b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_LENGTH)
    b.prefix_len.fill_(4 * page)
    for bad in (-1, 4, 100):  # request 0: negative, past its end (request 1's start), past T
        b.q_start[0] = bad
        b.run(True)
        assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_STARTS)
    b.q_start[0] = 0
    assert torch.equal(b.run(True)[0], want)
    assert b.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_blocks_that_overlap():
    """Starts out of order whose blocks claim more tokens than there are: no request is
    served."""
    b = Batch4(4, 2, 64, BF, 16, 40, [(5, 20), (5, 30), (5, 40)], seed=14)
    b.q_start.copy_(torch.tensor([0, 15, 0, 15], dtype=torch.int32))
    got, lse = b.run(True)
    assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_STARTS)
    assert not got.any() and (lse == float("-inf")).all()


@pytest.mark.gpu
def test_no_requests_and_no_pages():
    """A batch without requests, without a prefix or without own pages."""
    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.randn((5, 4, 64), device="cuda").to(BF)
    cache = torch.full(ops.kv4_shape(3, 8, 2, 64), 0x79, dtype=torch.uint8, device="cuda")
    ws = ops.Workspace(ops.prefix_attention_kv4_workspace_bytes(5, 2, 4, 2, 64))
    k = torch.randn((24, 2, 64), device="cuda").to(BF)
    ops.kv4_write(k, k, None, cache, ws)
    lse = torch.zeros((5, 4), device="cuda")
    out = ops.prefix_attention_kv4(q, cache, i32(0), i32(1), i32(8), None, None, ws, lse=lse)  # B = 0: all padding
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    out = ops.prefix_attention_kv4(q, cache, i32(0, 2, 5), None, None, None, None, ws, lse=lse)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    only_prefix = ops.prefix_attention_kv4(q, cache, i32(0, 2, 5), i32(1, 2), i32(11), None, None, ws)
    keys = ops.kv4_read(cache, 64, ws)[0][1:3].flatten(0, 1)[:11].double().repeat_interleave(2, 1)
    z = torch.einsum("nhd,mhd->hnm", q.double(), keys) * 64 ** -0.5
    want = torch.einsum("hnm,mhd->nhd", z.softmax(-1), keys)
    assert (only_prefix.double() - want).norm() <= 0.5 * torch.finfo(BF).eps * want.norm()
    assert ws.device_status() == (ops.MOE_OK, 0)
    empty = ops.prefix_attention_kv4(q[:0], cache, i32(0, 0, 0), i32(1), i32(8), None, None, ws)
    assert empty.shape == (0, 4, 64)


@pytest.mark.gpu
def test_pages_past_32_bit_offsets():
    """The pool holds more than 2^32 bytes and the batch's pages lie at its end."""
    page, Hkv, D = 64, 8, 128
    b = Batch4(32, Hkv, D, BF, page, 300, [(9, 100), (4, 20)], seed=21)
    pages = 2 ** 32 // (page * Hkv * (D + D // 16)) + 40
    pool = torch.zeros(ops.kv4_shape(pages, page, Hkv, D), device="cuda", dtype=torch.uint8)
    shift = pages - b.cache.shape[0]
    pool[shift:] = b.cache
    b.cache = pool
    b.prefix_pages = b.prefix_pages + shift
    b.table = b.table + shift
    b.check(True)


@pytest.mark.gpu
@pytest.mark.parametrize("D,causal", [(128, True), (64, False)])
def test_long_prompts(D, causal):
    """Thousands of tokens against a thousand keys each: every row tile and every tile
    of keys, by norms (the exact rows head by head)."""
    b = Batch4(8, 2, D, BF, 64, 200, [(1500, 1700), (3, 90), (700, 700)], seed=31)
    got, lse = b.run(causal)
    kp, vp = b.keys[0]
    for r, (n, own) in enumerate(b.blocks):
        t0 = b.start[r]
        k, v = (torch.cat(x) for x in ((kp, b.keys[r + 1][0]), (vp, b.keys[r + 1][1])))
        seen = 200 + (own - n + torch.arange(n, device="cuda") + 1 if causal else torch.full((n,), own, device="cuda"))
        for h in range(8):
            z = b.q[t0:t0 + n, h].double() @ k[:, h // 4].t() * D ** -0.5
            z = z.masked_fill(torch.arange(k.shape[0], device="cuda") >= seen[:, None], float("-inf"))
            want = z.softmax(-1) @ v[:, h // 4]
            off = (got[t0:t0 + n, h].double() - want).norm(dim=-1) / want.norm(dim=-1)
            # a row's error is a mean over D elements of two roundings of at most e/2
            assert off.max() <= torch.finfo(BF).eps
            assert (lse[t0:t0 + n, h].double() - torch.logsumexp(z, -1)).abs().max() <= 1e-4
    assert b.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,page", [(1, 16), (4, 64)])
def test_same_bits_from_cold_memory(n, page):
    """Copies that land late and in any order: long requests on scattered pages, call behind
    call, with what lies in L2 replaced between some of them."""
    batch = Batch4(8, 2, 128, BF, page, 0, [(n, 9000 + 700 * b) for b in range(12)], seed=n)
    batch.check(True)
    want = [t.clone() for t in batch.run(True)]
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for turn in range(60):
        if turn % 3 == 0:
            other.fill_(turn)
        for got, w in zip(batch.run(True), want):
            differ += (got != w).sum()
    assert differ.item() == 0
    assert batch.ws.device_status() == (ops.MOE_OK, 0)
