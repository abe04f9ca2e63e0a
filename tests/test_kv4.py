"""moe_kv4_write and moe_kv4_read: refusals on the host (no GPU), and on the GPU
every byte of the cache and every element read back against the rounding's
definition in 64 bits.

Tolerance: none.  A scale is a power of two and a product by it exact, so a code
and what it stands for do not depend on how they are computed.
"""
import numpy as np
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

BF, HF = torch.bfloat16, torch.float16
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ the definition

def encode(x):
    """x [..., 32] float64 -> (codes, scale byte)."""
    top = np.abs(x).max(-1)
    if not np.isfinite(x).all():
        return np.zeros(32, dtype=np.uint8), 255
    b = 104
    while b < 140 and top > 6 * 2.0 ** (b - 127):
        b += 1
    v = np.minimum(np.abs(x) / 2.0 ** (b - 127), 6)
    codes = np.empty(32, dtype=np.uint8)
    for i, a in enumerate(v):
        d = np.abs(GRID - a)
        near = np.flatnonzero(d == d.min())
        codes[i] = near[near % 2 == 0][0] if len(near) > 1 else near[0]
    return codes | (np.signbit(x).astype(np.uint8) << 3), b


def decode(codes, b):
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * (np.nan if b == 255 else 2.0 ** (int(b) - 127))


def put(cache, page, slot, h, which, D, x):
    """Stores one head's row of D channels in a numpy cache [pages, Hkv, bytes]."""
    block = cache[slot // page, h]
    at = slot % page
    for g in range(D // 32):
        codes, b = encode(x[32 * g:32 * g + 32])
        o = which * page * D // 2 + (g * page + at) * 16
        block[o:o + 16] = codes[0::2] | (codes[1::2] << 4)
        block[page * D + which * page * D // 32 + at * (D // 32) + g] = b


def get(cache, page, slot, h, which, D):
    block, at = cache[slot // page, h], slot % page
    out = []
    for g in range(D // 32):
        o = which * page * D // 2 + (g * page + at) * 16
        raw = block[o:o + 16]
        codes = np.stack([raw & 15, raw >> 4], axis=1).reshape(-1)
        out.append(decode(codes, block[page * D + which * page * D // 32 + at * (D // 32) + g]))
    return np.concatenate(out)


def whole(cache, page, which, D):
    """[pages, page, Hkv, D] in 64 bits."""
    return np.stack([np.stack([np.stack([get(cache, page, p * page + s, h, which, D) for h in range(cache.shape[1])])
                               for s in range(page)]) for p in range(cache.shape[0])])


# ------------------------------------------------------------------ refusals (no GPU)

def _write(**kw):
    a = dict(k=1 << 30, ks=1024, v=2 << 30, vs=1024, T=4, Hkv=8, D=128, dtype=0, slots=3 << 30, cache=4 << 30, pages=4,
             page=64, ws=5 << 30, wb=256)
    a.update(kw)
    return ops.lib().moe_kv4_write(*a.values(), None)


def _read(**kw):
    a = dict(cache=4 << 30, pages=4, page=64, Hkv=8, D=128, ids=3 << 30, n=2, k=1 << 30, v=2 << 30, dtype=0, ws=5 << 30,
             wb=256)
    a.update(kw)
    return ops.lib().moe_kv4_read(*a.values(), None)


INVALID, UNSUPPORTED, WORKSPACE = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(dtype=2), INVALID), (dict(pages=-1), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cache=None), INVALID), (dict(ks=-8), INVALID),
    (dict(k=(1 << 30) + 8), INVALID), (dict(cache=(4 << 30) + 8), INVALID), (dict(slots=None, T=257), INVALID),
    (dict(cache=1 << 30), INVALID), (dict(cache=3 << 30), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=4), UNSUPPORTED),
    (dict(page=2048), UNSUPPORTED), (dict(ks=1028), UNSUPPORTED), (dict(Hkv=1025), UNSUPPORTED),
    (dict(pages=1 << 25), UNSUPPORTED), (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(wb=128), WORKSPACE), (dict(ws=(5 << 30) + 16), WORKSPACE), (dict(T=0, k=None, ws=None), ops.MOE_OK),
])
def test_write_refusals(change, status):
    assert _write(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(k=None), INVALID), (dict(cache=None), INVALID), (dict(ids=None, n=5), INVALID),
    (dict(v=1 << 30), INVALID), (dict(k=4 << 30), INVALID), (dict(v=3 << 30), INVALID), (dict(dtype=-1), INVALID),
    (dict(k=(1 << 30) + 2), INVALID), (dict(D=32), UNSUPPORTED), (dict(page=12), UNSUPPORTED),
    (dict(n=1 << 23), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(wb=255), WORKSPACE),
    (dict(n=0, k=None, ws=None), ops.MOE_OK),
])
def test_read_refusals(change, status):
    assert _read(**change) == status


def test_tensors_that_are_not_on_a_gpu():
    k, cache = torch.zeros((2, 1, 64), dtype=BF), torch.zeros(ops.kv4_shape(2, 8, 1, 64), dtype=torch.uint8)
    ws = type("W", (), {"ptr": lambda s: 256, "nbytes": 256})()
    stream = type("S", (), {"cuda_stream": 0})()
    with pytest.raises(ValueError, match="CUDA"):
        ops.kv4_write(k, k, None, cache, ws, stream=stream)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kv4_read(cache, 64, ws, stream=stream)
    with pytest.raises(TypeError):
        ops.kv4_write(None, k, None, cache, ws, stream=stream)


# ------------------------------------------------------------------ against the definition

def _rows(T, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, 2 * Hkv * D), generator=g)
    # groups of every magnitude, values next to and on the codes' borders, zeros of both signs, type's extremes
    x.view(T, -1, 32).mul_(2.0 ** torch.randint(-26, 15, (T, 2 * Hkv * D // 32, 1), generator=g).float())
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, -0.25, -2.5, -5.0, 0.125, 4.5, 3.0])
    x[0, :32] = border.repeat(2) * 4
    x[0, 32:64] = 0
    if T > 1:
        x[1, :16] = torch.nextafter(border * 2, torch.tensor(100.0))
        x[1, 32:64] = 1e-7
        x[1, -32:] = torch.finfo(dtype).tiny
    return x.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hkv,D,page,dtype", [
    (1, 1, 64, 8, BF), (1, 8, 128, 64, HF), (2, 3, 64, 16, HF), (9, 2, 128, 8, BF), (37, 8, 64, 128, BF),
    (72, 5, 128, 16, HF), (8, 1, 128, 1024, BF)])
def test_write_and_read(T, Hkv, D, page, dtype):
    kv = _rows(T, Hkv, D, dtype, seed=T)
    k, v = (x.unflatten(1, (Hkv, D)) for x in kv.cuda().split(Hkv * D, dim=1))
    pages = -(-2 * T // page) + 1
    g = np.random.default_rng(T)
    slots = g.permutation(pages * page)[:T].astype(np.int32)
    if T > 2:
        slots[T // 2] = -1
    cache = torch.full(ops.kv4_shape(pages, page, Hkv, D), 0x7f, dtype=torch.uint8, device="cuda")
    want = cache.cpu().numpy()
    ws = ops.Workspace(ops.STATUS_BYTES)
    assert ops.kv4_write(k, v, torch.from_numpy(slots).cuda(), cache, ws) is cache
    over = False
    for t, s in enumerate(slots):
        for h in range(Hkv if s >= 0 else 0):
            for which, x in ((0, k), (1, v)):
                row = x[t, h].double().cpu().numpy()
                over |= bool((np.abs(row) > 49152).any())
                put(want, page, s, h, which, D, row)
    assert ws.device_status() == ((ops.MOE_ERR_DEVICE_RANGE, ops.INFO_KV_RANGE) if over else (0, 0))
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    for out in (BF, HF):
        got = ops.kv4_read(cache, D, ws, dtype=out)
        for which in (0, 1):
            assert got[which].shape == (pages, page, Hkv, D) and got[which].dtype == out
            ref = torch.from_numpy(whole(want, page, which, D)).to(out)
            assert torch.equal(got[which].cpu(), ref)
    ids = torch.tensor([pages - 1, 0, pages - 1], dtype=torch.int32, device="cuda")
    some = ops.kv4_read(cache, D, ws, pages=ids, dtype=dtype)
    every = ops.kv4_read(cache, D, ws, dtype=dtype)
    for a, b in zip(some, every):
        assert torch.equal(a, b[ids.long()])
    assert ws.device_status() == (0, 0)


@pytest.mark.gpu
def test_without_slots_and_with_bad_ones():
    T, Hkv, D, page = 11, 2, 64, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((T, Hkv, D), generator=g, device="cuda").to(BF) for _ in range(2))
    ws = ops.Workspace(ops.STATUS_BYTES)
    a = torch.zeros(ops.kv4_shape(2, page, Hkv, D), dtype=torch.uint8, device="cuda")
    b = a.clone()
    ops.kv4_write(k, v, None, a, ws)
    ops.kv4_write(k, v, torch.arange(T, dtype=torch.int32, device="cuda"), b, ws)
    assert torch.equal(a, b)
    slots = torch.tensor([16, 3, -5, 2 ** 31 - 1, -2 ** 31] + [-1] * (T - 5), dtype=torch.int32, device="cuda")
    c = torch.zeros_like(a)
    ops.kv4_write(k, v, slots, c, ws)
    assert ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_SLOT)
    d = torch.zeros_like(a)
    ops.kv4_write(k[1:2], v[1:2], slots[1:2], d, ws)
    assert torch.equal(c, d) and c.any()
    k2, v2 = ops.kv4_read(c, D, ws, pages=torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda"))
    assert ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_PAGE)
    assert not k2[1:].any() and not v2[1:].any() and k2[0, 3].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_groups_that_no_scale_holds(dtype):
    """Infinities and NaN make their group NaN; what is past 49152 becomes that."""
    D, ws = 64, ops.Workspace(ops.STATUS_BYTES)
    for bad in (float("inf"), float("-inf"), float("nan"), 60000.0):
        k = torch.ones((1, 1, D), dtype=dtype, device="cuda")
        k[0, 0, 5] = bad
        cache = torch.zeros(ops.kv4_shape(1, 8, 1, D), dtype=torch.uint8, device="cuda")
        ops.kv4_write(k, torch.ones_like(k), None, cache, ws)
        assert ws.device_status() == (ops.MOE_ERR_DEVICE_RANGE, ops.INFO_KV_RANGE)
        a, b = ops.kv4_read(cache, D, ws, dtype=dtype)
        assert (b[0, 0] == 1).all() and (a[0, 0, 0, 32:] == 1).all()
        if bad == 60000.0:
            assert a[0, 0, 0, 5] == 49152 and not a[0, 0, 0, :5].any()
        else:
            assert a[0, 0, 0, :32].isnan().all()


@pytest.mark.gpu
def test_captured():
    """A captured write serves later steps' slots."""
    T, Hkv, D, page = 5, 2, 128, 16
    k = torch.randn((T, Hkv, D), device="cuda").to(BF)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    cache = torch.zeros(ops.kv4_shape(3, page, Hkv, D), dtype=torch.uint8, device="cuda")
    ws = ops.Workspace(ops.STATUS_BYTES)
    ko, vo = (torch.empty((3, page, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
    ops.kv4_write(k, k, slots, cache, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.kv4_write(k, k, slots, cache, ws)
        ops.kv4_read(cache, D, ws, k=ko, v=vo)
    for first in (0, 20, 43):
        slots.copy_(torch.arange(first, first + T, dtype=torch.int32))
        cache.zero_()
        graph.replay()
        fresh = torch.zeros_like(cache)
        ops.kv4_write(k, k, slots, fresh, ws)
        assert torch.equal(fresh, cache)
        assert torch.equal(ko, ops.kv4_read(fresh, D, ws)[0])
    assert ws.device_status() == (0, 0)


@pytest.mark.gpu
def test_a_cache_past_2_31_bytes():
    """Pages whose bytes begin past what 32 bits count."""
    page, Hkv, D = 64, 8, 128
    pages = 2 ** 31 // (page * Hkv * (D + D // 16)) + 3
    cache = torch.empty(ops.kv4_shape(pages, page, Hkv, D), dtype=torch.uint8, device="cuda")
    cache[-1].zero_()
    cache[0].zero_()
    k = torch.randn((2, Hkv, D), device="cuda").to(BF)
    ws = ops.Workspace(ops.STATUS_BYTES)
    slots = torch.tensor([pages * page - 1, 1], dtype=torch.int32, device="cuda")
    ops.kv4_write(k, -k, slots, cache, ws)
    a, b = ops.kv4_read(cache, D, ws, pages=torch.tensor([pages - 1, 0], dtype=torch.int32, device="cuda"))
    assert ws.device_status() == (0, 0)
    small = torch.zeros(ops.kv4_shape(1, page, Hkv, D), dtype=torch.uint8, device="cuda")
    ops.kv4_write(k, -k, None, small, ws)
    ref, _ = ops.kv4_read(small, D, ws)
    assert torch.equal(a[0, -1], ref[0, 0]) and torch.equal(a[1, 1], ref[0, 1]) and torch.equal(a, -b)
    assert not a[0, :-1].any() and not a[1, 2:].any()
