"""moe_pages_resize, moe_pages_fork and moe_pages_compact: refusals on the host
(no GPU), and on the GPU random walks against a model of the pages on the host:
reference counts, tables, lengths and every byte of every pool.
"""
import random

import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build

INVALID, UNSUPPORTED, WORKSPACE = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


# ------------------------------------------------------------------ refusals (no GPU)

class Pool(ops.ctypes.Structure):
    """Mirror of moe_page_pool."""
    _fields_ = [("data", ops.ctypes.c_void_p), ("format", ops.ctypes.c_int32), ("heads", ops.ctypes.c_int32),
                ("head_dim", ops.ctypes.c_int32), ("row_bytes", ops.ctypes.c_int64)]


def _pools(*p):
    return ops.ctypes.cast((Pool * max(1, len(p)))(*[Pool(*x) for x in p]), ops.ctypes.c_void_p), len(p)


ROWS, KV4 = (8 << 30, 0, 0, 0, 2048), (9 << 30, 1, 8, 128, 0)


def _resize(pools=(ROWS, KV4), **kw):
    p, n = _pools(*pools)
    a = dict(refs=1 << 30, n_pages=16, table=2 << 30, B=4, width=8, page=16, own=3 << 30, new=4 << 30, pools=p, n=n,
             ws=7 << 30, wb=1 << 30)
    a.update(kw)
    return ops.lib().moe_pages_resize(*a.values(), None)


def _fork(pools=(ROWS, KV4), **kw):
    p, n = _pools(*pools)
    a = dict(refs=1 << 30, n_pages=16, table=2 << 30, B=4, width=8, page=16, own=3 << 30, src=4 << 30, dst=5 << 30, n=2,
             pools=p, np=n, ws=7 << 30, wb=1 << 30)
    a.update(kw)
    return ops.lib().moe_pages_fork(*a.values(), None)


def _compact(pools=(ROWS, KV4), **kw):
    p, n = _pools(*pools)
    a = dict(table=2 << 30, n_pages=16, B=4, width=8, page=16, base=3 << 30, keep=4 << 30, n=5, pools=p, np=n,
             new=5 << 30, ws=7 << 30, wb=256)
    a.update(kw)
    return ops.lib().moe_pages_compact(*a.values(), None)


SIZES = [(dict(n_pages=-1), INVALID), (dict(B=-1), INVALID), (dict(width=-1), INVALID), (dict(page=0), INVALID),
         (dict(table=None), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=4), UNSUPPORTED),
         (dict(page=2048), UNSUPPORTED), (dict(width=1 << 25), UNSUPPORTED), (dict(n_pages=1 << 28), UNSUPPORTED),
         (dict(B=65537), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=(7 << 30) + 8), WORKSPACE),
         (dict(wb=128), WORKSPACE), (dict(pools=[ROWS] * 2), INVALID), (dict(pools=[(2 << 30, 0, 0, 0, 64)]), INVALID),
         (dict(pools=[(None, 0, 0, 0, 64)]), INVALID), (dict(pools=[(8 << 30, 2, 0, 0, 64)]), INVALID),
         (dict(pools=[(8 << 30, 0, 0, 0, 0)]), INVALID), (dict(pools=[((8 << 30) + 4, 0, 0, 0, 64)]), INVALID),
         (dict(pools=[(8 << 30, 0, 0, 0, 24)]), UNSUPPORTED), (dict(pools=[(8 << 30, 1, 8, 96, 0)]), UNSUPPORTED),
         (dict(pools=[(8 << 30, 1, 0, 64, 0)]), INVALID),
         (dict(pools=[((8 << 30) + (i << 20), 0, 0, 0, 16) for i in range(65)]), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(refs=None), INVALID), (dict(own=None), INVALID), (dict(new=None), INVALID), (dict(new=3 << 30), INVALID),
    (dict(own=2 << 30), INVALID), (dict(refs=2 << 30), INVALID), (dict(B=0, ws=None), ops.MOE_OK)])
def test_resize_refusals(change, status):
    assert _resize(**change) == status


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(n=-1), INVALID), (dict(n=5), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID),
    (dict(src=2 << 30), INVALID), (dict(n=0, ws=None, src=None), ops.MOE_OK)])
def test_fork_refusals(change, status):
    assert _fork(**change) == status


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(n=-1), INVALID), (dict(n=1025), UNSUPPORTED), (dict(base=None), INVALID), (dict(keep=None), INVALID),
    (dict(new=3 << 30), INVALID), (dict(B=0, ws=None), ops.MOE_OK)])
def test_compact_refusals(change, status):
    assert _compact(**change) == status


def test_workspace_query():
    assert ops.pages_workspace_bytes(8, 1000) >= 4 * 1000
    for bad in ((-1, 5), (5, -1), (1 << 20, 5)):
        assert ops.lib().moe_pages_workspace_bytes(*bad) == 0


def test_tensors_that_are_not_on_a_gpu():
    i = torch.zeros((2, 3), dtype=torch.int32)
    ws = type("W", (), {"ptr": lambda s: 256, "nbytes": 256})()
    stream = type("S", (), {"cuda_stream": 0})()
    with pytest.raises(ValueError, match="CUDA"):
        ops.pages_resize(i[0], i, i[0, :2], i[1, :2], 16, ws, stream=stream)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pages_fork(i[0], i, i[0, :2], i[0, :1], i[1, :1], 16, ws, stream=stream)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pages_compact(i, i[0, :2], i, 16, ws, new_len=i[0, :2], stream=stream)


# ------------------------------------------------------------------ a model of the pages

class Model:
    """The calls' meaning, one request after the other."""

    def __init__(self, B, width, page, n_pages):
        self.B, self.width, self.page, self.n_pages = B, width, page, n_pages
        self.refs, self.table, self.len = [0] * n_pages, [[-1] * width for _ in range(B)], [0] * B
        self.rows = [[("start", p, o) for o in range(page)] for p in range(n_pages)]  # what each slot holds

    def pages(self, n):
        return -(-n // self.page)

    def resize(self, new):
        failed = False
        for b in range(self.B):
            for c in range(self.pages(new[b]), self.pages(self.len[b])):
                self.refs[self.table[b][c]] -= 1
                self.table[b][c] = -1
        free = [p for p in range(self.n_pages) if self.refs[p] == 0]
        shared = list(self.refs)
        before = [list(r) for r in self.rows]
        wanted = 0
        for b in range(self.B):
            stay = min(new[b], self.len[b])
            at = stay // self.page
            split = bool(stay % self.page) and shared[self.table[b][at]] > 1
            more = max(0, self.pages(new[b]) - self.pages(self.len[b]))
            wanted += more + split
            if more + split and wanted > len(free):
                failed = True
                self.len[b] = stay
                continue
            take = free[wanted - more - split:wanted]
            for p in take:
                self.refs[p] = 1
            if split:
                old, p = self.table[b][at], take.pop(0)
                self.refs[old] -= 1
                self.table[b][at] = p
                self.rows[p] = list(before[old])
            for i, p in enumerate(take):
                self.table[b][self.pages(self.len[b]) + i] = p
            self.len[b] = new[b]
        return failed

    def fork(self, pairs):
        failed, free, wanted = False, [p for p in range(self.n_pages) if self.refs[p] == 0], 0
        before = [list(r) for r in self.rows]
        for s, d in pairs:
            n = self.len[s]
            whole, tail = n // self.page, n % self.page != 0
            wanted += tail
            if tail and wanted > len(free):
                failed = True
                continue
            for c in range(whole):
                self.table[d][c] = self.table[s][c]
                self.refs[self.table[s][c]] += 1
            if tail:
                p = free[wanted - 1]
                self.refs[p] = 1
                self.table[d][whole] = p
                self.rows[p] = list(before[self.table[s][whole]])
            self.len[d] = n
        return failed

    def write(self, b, token, what):
        self.rows[self.table[b][token // self.page]][token % self.page] = what

    def read(self, b, token):
        return self.rows[self.table[b][token // self.page]][token % self.page]

    def compact(self, b, base, keep):
        for j, o in enumerate(keep):
            self.write(b, base + j, self.read(b, base + o))


class State:
    """The same on the GPU: every slot of every pool filled with what its place in
    the model's start says."""

    def __init__(self, m, pools):
        self.m = m
        self.refs, self.len = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (m.n_pages, m.B))
        self.table = torch.full((m.B, m.width), -1, dtype=torch.int32, device="cuda")
        self.ws = ops.Workspace(ops.pages_workspace_bytes(m.B, m.n_pages))
        g = torch.Generator().manual_seed(m.n_pages)
        self.start, self.pools = [], []
        for kind, *shape in pools:
            if kind == "kv4":
                heads, D = shape
                t = torch.randint(0, 256, ops.kv4_shape(m.n_pages, m.page, heads, D), generator=g, dtype=torch.uint8)
            else:
                t = torch.randint(-2 ** 15, 2 ** 15, (m.n_pages, m.page, *shape), generator=g).to(torch.int16)
            self.start.append(t)
            self.pools.append(t.cuda())

    def slots(self, t):
        """The bytes of every slot: [pages, page, n]."""
        if t.dim() == 3 and t.dtype is torch.uint8:
            n, heads, size = t.shape
            page, D = self.m.page, size // self.m.page * 16 // 17
            groups = D // 32
            codes = t[..., :page * D].view(n, heads, 2 * groups, page, 16).permute(0, 3, 1, 2, 4).flatten(2)
            scales = t[..., page * D:].view(n, heads, 2, page, groups).permute(0, 3, 1, 2, 4).flatten(2)
            return torch.cat([codes, scales], dim=2)
        return t.flatten(2)

    def check(self):
        m = self.m
        assert self.refs.tolist() == m.refs
        assert self.table.tolist() == m.table
        assert self.len.tolist() == m.len
        for start, pool in zip(self.start, self.pools):
            a, b = self.slots(start), self.slots(pool.cpu())
            src = torch.tensor([p * m.page + o for row in m.rows for _, p, o in row])
            want = a.reshape(m.n_pages * m.page, -1)[src]
            assert torch.equal(b.reshape(m.n_pages * m.page, -1), want)

    def resize(self, new):
        failed = self.m.resize(new)
        ops.pages_resize(self.refs, self.table, self.len, _i32(new), self.m.page, self.ws, caches=self.pools)
        self.check()
        assert self.ws.device_status() == ((ops.MOE_ERR_DEVICE_POOL, ops.INFO_POOL) if failed else (0, 0))

    def fork(self, pairs):
        failed = self.m.fork(pairs)
        ops.pages_fork(self.refs, self.table, self.len, _i32([s for s, _ in pairs]), _i32([d for _, d in pairs]),
                       self.m.page, self.ws, caches=self.pools)
        self.check()
        assert self.ws.device_status() == ((ops.MOE_ERR_DEVICE_POOL, ops.INFO_POOL) if failed else (0, 0))

    def compact(self, base, keep):
        n = max(k[-1] + 1 for k in keep if k)  # the block's tokens
        rows = [k + [-1] * (n - len(k)) for k in keep]
        for b, k in enumerate(keep):
            self.m.compact(b, base[b], k)
        new = ops.pages_compact(self.table, _i32(base), _i32(rows).view(len(base), n), self.m.page, self.ws,
                                caches=self.pools)
        self.check()
        assert new.tolist() == [a + len(k) for a, k in zip(base, keep)]
        assert self.ws.device_status() == (0, 0)
        return new.tolist()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


POOLS = [("kv4", 2, 64), ("rows", 3, 8), ("kv4", 3, 128), ("rows", 8), ("rows", 2, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,width,page,n_pages,seed", [(1, 4, 8, 5, 0), (4, 9, 8, 30, 1), (5, 6, 16, 24, 2),
                                                       (40, 5, 8, 150, 3), (13, 12, 32, 90, 4)])
def test_random_walk(B, width, page, n_pages, seed):
    """Growth, truncation into shared pages, forks, verify steps and ends, with
    and without free pages enough."""
    rng = random.Random(seed)
    s = State(Model(B, width, page, n_pages), POOLS)
    m = s.m
    s.check()
    for step in range(30):
        what = rng.choice(["grow", "any", "fork", "verify", "end"])
        if what == "fork":
            free = [b for b in range(B) if m.len[b] == 0]
            used = [b for b in range(B) if m.len[b] > 0]
            if free and used:
                s.fork([(rng.choice(used), d) for d in rng.sample(free, rng.randint(1, len(free)))])
        elif what == "verify":
            base = list(m.len)
            n = rng.randint(1, min(12, page + 3))
            s.resize([min(x + n, width * page) for x in base])
            if all(m.len[b] >= base[b] for b in range(B)):
                room = [m.len[b] - base[b] for b in range(B)]
                keep = [sorted(rng.sample(range(r), rng.randint(0, r))) for r in room]
                if any(keep):
                    s.resize(s.compact(base, keep))
        else:
            new = list(m.len)
            for b in range(B):
                if rng.random() < 0.6:
                    new[b] = {"grow": min(width * page, new[b] + rng.randint(0, 2 * page)), "end": 0,
                              "any": rng.randint(0, width * page)}[what]
            s.resize(new)


@pytest.mark.gpu
@pytest.mark.parametrize("page,pools", [(8, POOLS), (1024, [("rows", 512), ("kv4", 5, 128)]), (256, [("rows", 2048), ("kv4", 1, 64)])])
def test_shared_pages_that_are_written_on(page, pools):
    """Every request of a resize takes a copy of a page that others hold too: of small
    pools, and of pools so large that copies are a launch of their own."""
    s = State(Model(9, 2, page, 30), pools)
    s.resize([page // 2 + 1, page - 1, 1] + [0] * 6)
    s.fork([(0, 3), (1, 4), (2, 5), (0, 6), (0, 7), (1, 8)])
    m = s.m
    for b in range(9):  # shared once more, as a prefix that another table holds would be
        m.refs[m.table[b][0]] += 1
    s.refs.copy_(_i32(m.refs))
    s.resize([min(2 * page, n + 3) for n in m.len])
    assert len({t[0] for t in m.table}) == 9
    s.resize([n - 1 for n in m.len])


@pytest.mark.gpu
def test_many_pages_and_requests():
    """More pages and requests than a CTA has threads, in one call."""
    B, width, page, n_pages = 1500, 3, 8, 9000
    s = State(Model(B, width, page, n_pages), [("rows", 8)])
    rng = random.Random(5)
    s.resize([rng.randint(0, width * page) if b % 2 == 0 else 0 for b in range(B)])
    s.fork([(b - 1, b) for b in range(1, B, 2)])
    s.resize([rng.randint(0, width * page) for b in range(B)])
    s.resize([rng.randint(0, 5) for b in range(B)])


@pytest.mark.gpu
def test_one_long_request():
    s = State(Model(3, 3000, 8, 9000), [("rows", 8)])
    s.resize([5, 24000, 3])
    s.resize([24000, 7, 24000])
    s.resize([0, 0, 23999])


@pytest.mark.gpu
def test_pairs_that_are_not_made():
    m = Model(6, 4, 8, 20)
    s = State(m, [("rows", 8)])
    s.resize([13, 8, 0, 0, 0, 3])
    m.fork([(0, 2), (1, 3)])
    # padding; a child with tokens, one outside, a source outside, a child named twice (the first is made)
    src, dst = _i32([-1, 0, 0, 1, 9, 0]), _i32([4, 5, 2, 3, 4, 3])
    ops.pages_fork(s.refs, s.table, s.len, src, dst, m.page, s.ws, caches=s.pools)
    s.check()
    assert s.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_FORK)
    ops.pages_fork(s.refs, s.table, s.len, _i32([-1, 0]), _i32([4, -7]), m.page, s.ws, caches=s.pools)
    s.check()
    assert s.ws.device_status() == (0, 0)


@pytest.mark.gpu
def test_lengths_and_entries_outside():
    m = Model(4, 4, 8, 20)
    s = State(m, [("rows", 8)])
    s.resize([13, 8, 20, 0])
    m.resize([13, 8, 4, 9])
    ops.pages_resize(s.refs, s.table, s.len, _i32([-1, 33, 4, 9]), m.page, s.ws, caches=s.pools)
    s.check()
    assert s.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_LENGTH)
    # an entry outside the pool, and a page that no one holds, among those given back
    s.table[0, 1] = 20
    s.refs[s.table[1, 0].long()] = 0
    ops.pages_resize(s.refs, s.table, s.len, _i32([0, 0, 4, 9]), m.page, s.ws, caches=s.pools)
    assert s.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_PAGE)
    assert (s.refs >= 0).all() and s.len.tolist() == [0, 0, 4, 9] and s.table[0].tolist() == [-1] * 4


@pytest.mark.gpu
def test_kept_offsets_outside():
    m = Model(6, 4, 8, 30)
    s = State(m, POOLS)
    s.resize([32] * 5 + [0])
    base = [3, 28, 9, 40, 1, 0]
    keep = [[1, 1, 3], [1, 3, 4], [2, -1, 1], [0, 1, 2], [0, 2, 3], [0, 1, 2]]
    for b, k in enumerate([[1], [1, 3], [2], [], [0, 2, 3], []]):  # what comes before the fault moves
        m.compact(b, base[b], k)
    new = ops.pages_compact(s.table, _i32(base), _i32([k + [-1] * 2 for k in keep]), m.page, s.ws, caches=s.pools)
    s.check()
    # (the third offset of request 1 lies behind the table, the sixth request has no pages)
    assert new.tolist() == [4, 30, 10, 32, 4, 0]
    assert s.ws.device_status()[0] == ops.MOE_ERR_DEVICE_INDEX


@pytest.mark.gpu
def test_captured_steps():
    """One captured verify step, replayed as the requests grow."""
    B, width, page, n = 5, 20, 8, 6
    m = Model(B, width, page, 120)
    s = State(m, POOLS)
    rng = random.Random(9)
    s.resize([rng.randint(0, 30) for _ in range(B)])
    base, grown, keep, new = s.len.clone(), s.len + n, _i32([[0] * n] * B), _i32([0] * B)

    def step():
        base.copy_(s.len)
        torch.add(base, n, out=grown)
        ops.pages_resize(s.refs, s.table, s.len, grown, page, s.ws, caches=s.pools)
        ops.pages_compact(s.table, base, keep, page, s.ws, caches=s.pools, new_len=new)
        ops.pages_resize(s.refs, s.table, s.len, new, page, s.ws, caches=s.pools)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(8):
        at, kept = list(m.len), [sorted(rng.sample(range(n), rng.randint(0, n))) for _ in range(B)]
        m.resize([x + n for x in at])
        for b in range(B):
            m.compact(b, at[b], kept[b])
        m.resize([x + len(k) for x, k in zip(at, kept)])
        keep.copy_(torch.tensor([k + [-1] * (n - len(k)) for k in kept]))
        graph.replay()
        s.check()
    assert s.ws.device_status() == (0, 0)


@pytest.mark.gpu
def test_without_pools_or_pages():
    ws = ops.Workspace(ops.pages_workspace_bytes(2, 4))
    refs, table, own = _i32([0] * 4), _i32([[-1] * 3] * 2), _i32([0, 0])
    ops.pages_resize(refs, table, own, _i32([17, 1]), 8, ws)
    assert refs.tolist() == [1] * 4 and table.tolist() == [[0, 1, 2], [3, -1, -1]] and own.tolist() == [17, 1]
    new = ops.pages_compact(table, _i32([3, 0]), _i32([[0, 2], [-1, 1]]), 8, ws)
    assert new.tolist() == [5, 0] and ws.device_status() == (0, 0)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    own.zero_()
    ops.pages_resize(none, table[:, :0].contiguous(), own, _i32([0, 0]), 8, ws)
    assert ws.device_status() == (0, 0)
    with pytest.raises(ValueError, match="pages"):
        ops.pages_resize(refs, table, own, own + 1, 8, ws, caches=[torch.zeros((3, 8, 8), device="cuda")])
    with pytest.raises(ValueError, match="page_size"):
        ops.pages_resize(refs, table, own, own + 1, 8, ws, caches=[torch.zeros((4, 16, 8), device="cuda")])
    with pytest.raises(TypeError):
        ops.pages_resize(refs.long(), table, own, own + 1, 8, ws)
    with pytest.raises(ops.MoeError):
        ops.pages_resize(refs, table, own, own, 8, ws)
