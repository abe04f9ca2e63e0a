"""moe_prefix_attention_kv4: NaN in a query, or in a key that a row sees, makes the row NaN
(out and lse) however few keys it sees; a row that sees no key is zeros and -infinity
whatever its query, and every other row keeps its bits.
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_prefix_attention import BF, HF, NAN
from test_prefix_attention_kv4 import Batch4


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


def _seen(b, causal):
    """Own keys that every token sees."""
    return torch.tensor([max(0, own - n + i + 1) if causal else own for n, own in b.blocks for i in range(n)], device="cuda")


def _check(b, causal, bad, want):
    """Rows `bad` [T, Hq] are NaN, the others `want` (out, lse)."""
    out, lse = b.run(causal)
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])
    assert b.ws.device_status() == (ops.MOE_OK, 0)


def _queries(b, causal):
    """NaN in one query head, in a whole token, in a whole block, in every query."""
    T, Hq, _ = b.q.shape
    want = b.run(causal)
    some = ((_seen(b, causal) + b.P) > 0)[:, None]
    q = b.q.clone()
    for rows, heads in ((slice(T // 2, T // 2 + 1), slice(1, 2)), (slice(T - 1, T), slice(0, Hq)),
                        (slice(0, b.blocks[0][0]), slice(0, Hq)), (slice(0, T), slice(0, Hq))):
        hit = torch.zeros((T, Hq), dtype=torch.bool, device="cuda")
        hit[rows, heads] = True
        b.q[rows, heads, 5] = NAN
        _check(b, causal, hit & some, want)
        b.q.copy_(q)


def _last_key(b, causal):
    """The last own key of request 0 is a NaN group of key head 0."""
    T, Hq, D = b.q.shape
    want = b.run(causal)
    n, own = b.blocks[0]
    k, v = (x[own - 1:own].to(b.q.dtype) for x in b.keys[1])
    k[:, 0, 3] = NAN
    slot = (b.table[0, (own - 1) // b.page] * b.page + (own - 1) % b.page)[None]
    ops.kv4_write(k, v, slot, b.cache, b.ws)
    assert b.ws.device_status() == (ops.MOE_ERR_DEVICE_RANGE, ops.INFO_KV_RANGE)
    hit = torch.zeros((T, Hq), dtype=torch.bool, device="cuda")
    hit[(n - 1 if causal else 0):n, :Hq // b.Hkv] = True
    _check(b, causal, hit, want)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF)])
@pytest.mark.parametrize("n,own,P", [(5, 5, 0), (8, 1, 0), (12, 5, 0), (16, 130, 0), (5, 6, 3), (12, 20, 130), (9, 200, 128)])
def test_many_rows(n, own, P, D, dtype, causal):
    """Blocks of 20 to 64 rows a key head (few and many of a softmax group), fewer keys than
    a tile and more."""
    for f in (_queries, _last_key):
        f(Batch4(8, 2, D, dtype, 16, P, [(n, own), (n, own + 3)], seed=n), causal)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF)])
@pytest.mark.parametrize("Hq,Hkv,n,own,P", [(64, 8, 1, 5, 0), (64, 8, 1, 1, 0), (64, 8, 1, 300, 0), (64, 8, 2, 5, 0),
                                            (32, 8, 1, 5, 0), (32, 8, 4, 3, 0), (32, 8, 2, 700, 3), (16, 1, 1, 5, 3)])
def test_few_rows(Hq, Hkv, n, own, P, D, dtype, causal):
    """Blocks of 4, 8 and 16 rows a key head, all of them NaN and some, keys for one warp and
    for several."""
    for f in (_queries, _last_key):
        f(Batch4(Hq, Hkv, D, dtype, 16, P, [(n, own), (n, own + 3)], seed=n), causal)
