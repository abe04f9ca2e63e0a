"""moe_pages_compact: kept offsets out of order near a table's end.  An entry behind one
that does not grow may be small and far down its list at once, so that the place it would
go to lies behind the table: it is recorded and nothing is read there.  (Only the outcome
is visible: what comes before the fault moves, the list ends there.)
"""
import pytest
import torch

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_pages import POOLS, Model, State, _i32


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [8, 32])
def test_places_behind_the_table(page):
    m = Model(5, 2, page, 12)
    s = State(m, POOLS)
    cap = 2 * page
    s.resize([cap] * 5)
    base = [cap - 2, cap - 3, cap - 1, 0, cap - 2]
    n = 1024
    keep = [[5, 0, 1], [1, 2, 0, 1, 2], [0, 0] * 512, [0, 1] * 512, [0, 1] * 512]
    for b, k in enumerate([[], [1, 2], [0], [0, 1], [0, 1]]):
        m.compact(b, base[b], k)
    new = ops.pages_compact(s.table, _i32(base), _i32([k + [-1] * (n - len(k)) for k in keep]), page, s.ws, caches=s.pools)
    s.check()
    assert new.tolist() == [cap - 2, cap - 1, cap, 2, cap]
    assert s.ws.device_status() == (ops.MOE_ERR_DEVICE_INDEX, ops.INFO_KEEP)


@pytest.mark.gpu
def test_a_list_that_grows_to_the_tables_end():
    m = Model(2, 2, 8, 6)
    s = State(m, POOLS)
    s.resize([16, 16])
    assert s.compact([3, 15], [[0, 2, 5, 12], [0]]) == [7, 16]
    assert s.compact([0, 14], [list(range(16)), [1]]) == [16, 15]
