"""PagedRequests.keep behind a block that found no pages: the request keeps its tokens and no
others, and nothing is moved in a page that another request holds too.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import decoder, ops
from moe_ffn_speculative_gb300.build import build

PAGE, PAGES = 8, 3


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _requests(rows):
    a = decoder.AttentionConfig(q_heads=4, kv_heads=2, head_dim=64)
    cache = decoder.KVCache4(PAGES, PAGE, a)
    cache.data.copy_(torch.randint(0, 256, cache.data.shape, generator=torch.Generator().manual_seed(rows)))
    return decoder.PagedRequests(rows, 2, PAGES, PAGE, [cache.data]), cache.data


def _keep(r, captured, base, kept):
    if not captured:
        return r.keep(base, kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.keep(base, kept)
    graph.replay()


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_kept_tokens_that_would_fit_the_last_page(captured):
    """A block of six behind five tokens needs a page that there is not; two kept ones would
    not, but were never written."""
    r, data = _requests(2)
    r.resize(_i32(5, 16))                 # all three pages
    before = data.clone()
    _, base = r.block(6)
    assert r.ws.device_status()[0] != ops.MOE_OK
    _keep(r, captured, base, _i32(*[[0, 1, -1, -1, -1, -1]] * 2))
    assert r.own_len.tolist() == [5, 16] and r.refs.tolist() == [1] * PAGES
    assert torch.equal(data, before) and r.ws.device_status() == (ops.MOE_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_a_shared_page_that_could_not_be_copied(captured):
    """A child cut back into a full page that it shares, without a page to copy it to: its
    tokens behind the cut are the parent's, before and after it keeps some."""
    r, data = _requests(3)
    r.resize(_i32(8, 16, 0))              # all three pages
    r.fork(_i32(0), _i32(2))              # shares the full page
    r.resize(_i32(8, 16, 3))
    assert r.ws.device_status()[0] == ops.MOE_ERR_DEVICE_POOL
    shared = r.table[0, 0].item()
    assert r.table[2, 0].item() == shared and r.refs[shared].item() == 2
    before, base = data.clone(), r.own_len.clone()
    b, base = r.block(3)
    assert base.tolist() == [8, 16, 3] and b.slots.tolist() == [-1] * 9
    assert r.ws.device_status()[0] != ops.MOE_OK
    _keep(r, captured, base, _i32(*[[0, 2, -1]] * 3))
    assert torch.equal(data, before)
    assert r.own_len.tolist() == [8, 16, 3] and r.table[2, 0].item() == shared
    # once a page is free the child copies its tokens and goes on by itself
    r.resize(_i32(8, 0, 3))
    r.ws.device_status()
    b, base = r.block(3)
    mine = r.table[2, 0].item()
    assert r.own_len.tolist()[2] == 6 and mine != shared
    _keep(r, captured, base, _i32([-1] * 3, [-1] * 3, [0, 2, -1]))
    assert r.own_len.tolist() == [8, 0, 5] and torch.equal(data[shared], before[shared])
    k, v = ops.kv4_read(data, 64, r.ws, pages=_i32(shared, mine))
    assert torch.equal(k[0, :3].nan_to_num(), k[1, :3].nan_to_num()) and torch.equal(v[0, :3].nan_to_num(), v[1, :3].nan_to_num())


@pytest.mark.gpu
def test_requests_that_got_theirs_keep_them():
    r, data = _requests(2)
    r.resize(_i32(5, 8))
    _, base = r.block(3)
    rows = [x.flatten(0, 1).nan_to_num().clone() for x in ops.kv4_read(data, 64, r.ws)]
    t = r.table.tolist()
    r.keep(base, _i32([0, 2, -1], [1, -1, 2]))
    assert r.own_len.tolist() == [7, 9]
    now = [x.flatten(0, 1).nan_to_num() for x in ops.kv4_read(data, 64, r.ws)]
    for x, y in zip(rows, now):
        x[t[0][0] * PAGE + 6] = x[t[0][0] * PAGE + 7]
        x[t[1][1] * PAGE] = x[t[1][1] * PAGE + 1]
        assert torch.equal(x, y)
    assert r.ws.device_status() == (ops.MOE_OK, 0)
