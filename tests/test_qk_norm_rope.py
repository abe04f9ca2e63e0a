"""moe_qk_norm_rope: refusals on the host (no GPU), and on the GPU every output
against the formula in 64 bits.

Tolerance of an element, derived: one rounding to the output type, half a
step, eps/2 relative to the value (2^-25 for f16 subnormals), on top of fp32
arithmetic: the norm factor (a sum of up to 256 squares over at most 8 + 5
additions, a square root and a division) and two products and a sum per
rotated pair, together below 24 steps of 2^-24 relative to |a c| + |b s|.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ refusals (no GPU)

def _call(**kw):
    """The C entry point on plain addresses that no refused call dereferences."""
    a = dict(q=1 << 20, qs=512, k=2 << 20, ks=128, v=3 << 20, vs=128, T=4, Hq=4, Hkv=1, D=128, dtype=0, qw=None, kw=None,
             eps=1e-6, rope=4 << 20, rot=128, maxp=64, inter=0, pos=5 << 20, qo=6 << 20, qos=512, kc=7 << 20,
             vc=8 << 20, slots=9 << 20, n=16, ws=10 << 20, wb=256)
    a.update(kw)
    return ops.lib().moe_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), ops.MOE_ERR_INVALID_ARG), (dict(dtype=2), ops.MOE_ERR_INVALID_ARG),
    (dict(rot=256), ops.MOE_ERR_INVALID_ARG), (dict(inter=2), ops.MOE_ERR_INVALID_ARG),
    (dict(eps=-1.0), ops.MOE_ERR_INVALID_ARG), (dict(eps=float("nan")), ops.MOE_ERR_INVALID_ARG),
    (dict(q=None), ops.MOE_ERR_INVALID_ARG), (dict(qo=None), ops.MOE_ERR_INVALID_ARG),
    (dict(k=None), ops.MOE_ERR_INVALID_ARG), (dict(kc=None), ops.MOE_ERR_INVALID_ARG),
    (dict(v=None), ops.MOE_ERR_INVALID_ARG), (dict(vc=None), ops.MOE_ERR_INVALID_ARG),
    (dict(rope=None), ops.MOE_ERR_INVALID_ARG), (dict(pos=None), ops.MOE_ERR_INVALID_ARG),
    (dict(slots=None, n=3), ops.MOE_ERR_INVALID_ARG), (dict(q=(1 << 20) + 2), ops.MOE_ERR_INVALID_ARG),
    (dict(qos=256), ops.MOE_ERR_INVALID_ARG), (dict(n=-1), ops.MOE_ERR_INVALID_ARG),
    (dict(D=96, rot=96), ops.MOE_ERR_UNSUPPORTED), (dict(rot=24), ops.MOE_ERR_UNSUPPORTED),
    (dict(qs=514), ops.MOE_ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), ops.MOE_ERR_UNSUPPORTED),
    (dict(ws=None), ops.MOE_ERR_WORKSPACE), (dict(ws=(10 << 20) + 64), ops.MOE_ERR_WORKSPACE),
    (dict(wb=128), ops.MOE_ERR_WORKSPACE),
    (dict(T=0, q=None, ws=None), ops.MOE_OK), (dict(Hq=0, Hkv=0, ws=None), ops.MOE_OK),
])
def test_refusals(change, status):
    assert _call(**change) == status


def test_python_refusals():
    """The binding's own checks, before any library call."""
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, None, None, None, None, None)  # not on a CUDA device
    with pytest.raises(TypeError):
        ops.qk_norm_rope(q.float(), None, None, None, None, None)
    with pytest.raises(TypeError):
        ops.qk_norm_rope(q, q.half(), None, None, None, None)


# ------------------------------------------------------------------ values (GPU)

def _formula(x, w, eps, table, pos, rot, interleaved):
    """(y, bound on the fp32 arithmetic's magnitude) in 64 bits, on the CPU."""
    x = x.cpu().double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.cpu().double()
    y, mag = x.clone(), x.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = (table.cpu().double()[pos.cpu().long(), j][:, None] for j in (i, i + rot // 2))
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def _near(got, y, mag, dtype):
    tol = torch.finfo(dtype).eps / 2 * y.abs() + 24 * 2.0 ** -24 * mag + (2.0 ** -25 if dtype == torch.float16 else 0)
    off = (got.cpu().double() - y).abs()
    assert bool((off <= tol).all()), f"off by up to {(off / tol).max().item():.3f} of the tolerance"


CASES = [
    # T, Hq, Hkv, D, rot, interleaved, dtype, weights, page
    (1, 1, 1, 64, 64, False, torch.bfloat16, True, 16),
    (1, 32, 8, 128, 128, False, torch.bfloat16, True, 64),
    (9, 32, 8, 128, 128, True, torch.float16, True, 16),
    (72, 32, 8, 128, 128, False, torch.bfloat16, True, 64),
    (33, 5, 1, 256, 256, False, torch.float16, True, 32),
    (17, 40, 8, 64, 32, True, torch.bfloat16, False, 16),
    (17, 28, 4, 128, 64, False, torch.bfloat16, True, 128),
    (7, 24, 3, 256, 96, False, torch.bfloat16, True, 16),
    (5, 16, 16, 64, 48, False, torch.float16, False, 16),
    (5, 3, 2, 128, 0, False, torch.float16, True, 16),
    (1001, 64, 8, 64, 64, False, torch.float16, True, 64),
    (4, 0, 8, 128, 128, False, torch.bfloat16, True, 16),   # keys and values alone
    (4, 8, 0, 128, 128, False, torch.bfloat16, True, 16),   # queries alone
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,dtype,weights,page", CASES)
def test_against_formula(T, Hq, Hkv, D, rot, interleaved, dtype, weights, page):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + D + rot)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    qkv = normal(T, (Hq + 2 * Hkv) * D)
    if T > 1:
        qkv[T // 2] *= 0.001  # a row whose mean square is near eps
        qkv[T // 3] = 0
    q, k, v = (x.unflatten(1, (n, D)) if n else None
               for x, n in zip(qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1), (Hq, Hkv, Hkv)))
    table = ops.rope_table(5000, rot, base=1e6) if rot else None
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32) if rot else None
    if rot:
        pos[0], pos[-1] = 4999, 0
    qw, kw = (normal(D), normal(D)) if weights else (None, None)
    pages = -(-T // page) + 2
    kc = vc = slots = None
    if Hkv:
        kc, vc = normal(pages, page, Hkv, D), normal(pages, page, Hkv, D)
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
        if T > 2:
            slots[1] = -1
    kc0, vc0 = (None if c is None else c.clone() for c in (kc, vc))
    ws = ops.Workspace(ops.STATUS_BYTES)
    q_out, _, _ = ops.qk_norm_rope(q, k, v, pos, table, ws, q_weight=qw, k_weight=kw, eps=1e-6,
                                   interleaved=interleaved, k_cache=kc, v_cache=vc, slots=slots)
    assert ws.device_status() == (ops.MOE_OK, 0)
    if Hq:
        _near(q_out, *_formula(q, qw, 1e-6, table, pos, rot, interleaved), dtype)
    if Hkv:
        y, mag = _formula(k, kw, 1e-6, table, pos, rot, interleaved)
        at = slots.cpu().long()
        keep = at >= 0
        _near(kc.view(-1, Hkv, D).cpu()[at[keep]], y[keep], mag[keep], dtype)
        rows = vc.view(-1, Hkv, D).cpu()
        assert torch.equal(rows[at[keep]], v.cpu()[keep])
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at[keep]] = False
        for new, old in ((kc, kc0), (vc, vc0)):  # every other row of the cache is as it was
            assert torch.equal(new.view(-1, Hkv, D).cpu()[rest], old.view(-1, Hkv, D).cpu()[rest])


@pytest.mark.gpu
def test_in_place_dense_rows_and_stream():
    """q rotated in place; no slots: row t; on a stream of its own, and
    captured into a graph, the same bits."""
    T, Hq, Hkv, D = 19, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((T, Hq, D), generator=g, device="cuda").bfloat16()
    k = torch.randn((T, Hkv, D), generator=g, device="cuda").bfloat16()
    table = ops.rope_table(64, D)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    ws = ops.Workspace(ops.STATUS_BYTES)
    want, kc, _ = ops.qk_norm_rope(q, k, None, pos, table, ws)
    assert kc.shape == (T, Hkv, D)
    _near(kc, *_formula(k, None, 0, table, pos, D, False), torch.bfloat16)
    inplace = q.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.qk_norm_rope(inplace, None, None, pos, table, ws, q_out=inplace, stream=s)
    s.synchronize()
    assert torch.equal(inplace, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.qk_norm_rope(q, None, None, pos, table, ws, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_indexes_outside_their_tables():
    """A position past the table or negative: the token is skipped; a slot past
    the cache: not cached; both recorded, everything else is written."""
    T, H, D = 6, 2, 64
    q = torch.ones((T, H, D), device="cuda").bfloat16()
    table = ops.rope_table(10, D)
    ws = ops.Workspace(ops.STATUS_BYTES)
    for bad in (10, -1, 2 ** 31 - 1):
        pos = torch.zeros(T, device="cuda", dtype=torch.int32)
        pos[3] = bad
        out = torch.full_like(q, 7)
        ops.qk_norm_rope(q, None, None, pos, table, ws, q_out=out)
        assert ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_POSITION)
        assert bool((out[3] == 7).all()) and bool((out[[0, 1, 2, 4, 5]] == 1).all())
    for bad in (8, 2 ** 31 - 1):
        slots = torch.arange(T, device="cuda", dtype=torch.int32)
        slots[2] = bad
        kc, vc = torch.zeros((8, H, D), device="cuda").bfloat16(), torch.zeros((8, H, D), device="cuda").bfloat16()
        pos = torch.zeros(T, device="cuda", dtype=torch.int32)
        ops.qk_norm_rope(None, q, q, pos, table, ws, k_cache=kc, v_cache=vc, slots=slots)
        assert ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_SLOT)
        want = torch.tensor([1, 1, 0, 1, 1, 1, 0, 0], device="cuda").bfloat16()
        assert torch.equal(kc[:, 0, 0], want) and torch.equal(vc[:, 1, 5], want)
    assert ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
def test_slots_past_32_bit_offsets():
    """Rows of a cache of more than 2^31 elements, and a projection row stride
    that takes the last token past 2^31 elements of its tensor."""
    Hkv, D = 8, 128
    rows = 2 ** 31 // (Hkv * D) + 64
    g = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.zeros((3, 2 ** 30 + 64), device="cuda", dtype=torch.bfloat16)
    k = wide[:, :Hkv * D].unflatten(1, (Hkv, D))
    k.copy_(torch.randn((3, Hkv, D), generator=g, device="cuda"))
    table, pos = ops.rope_table(16, D), torch.tensor([3, 0, 15], device="cuda", dtype=torch.int32)
    cache = torch.zeros((rows, Hkv, D), device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([rows - 1, rows - 64, 5], device="cuda", dtype=torch.int32)
    ws = ops.Workspace(ops.STATUS_BYTES)
    ops.qk_norm_rope(None, k, None, pos, table, ws, k_cache=cache, slots=slots)
    assert ws.device_status() == (ops.MOE_OK, 0)
    _near(cache[slots.long()], *_formula(k, None, 0, table, pos, D, False), torch.bfloat16)
