"""Outputs of the attention side's calls that lie in what the call reads, or in one
another: refused on the host, before any launch (no GPU).  Slices of one buffer
that only lie next to each other pass that check: they get as far as the
workspace's."""
import pytest

from moe_ffn_speculative_gb300 import ops
from moe_ffn_speculative_gb300.build import build
from test_linear import _call as _linear
from test_prefix_attention import _call as _attention
from test_qk_norm_rope import _call as _rope

BAD, PASS = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_WORKSPACE
M = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()
    ops.lib()


@pytest.mark.parametrize("change,status", [
    # x [4, 64] at 1 MB, w [128, 64] at 2 MB, y [4, 128] at 3 MB
    (dict(y=M + 128), BAD),                                  # over x's second row
    (dict(y=M - 1024 + 16), BAD), (dict(y=M - 1024), PASS),  # its end over x's start, or up to it
    (dict(y=2 * M + 128 * 64 * 2 - 16), BAD), (dict(y=2 * M + 128 * 64 * 2), PASS),
    (dict(xs=192, ys=192, y=M + 128), PASS), (dict(xs=192, ys=192, y=M + 112), BAD),  # columns next to x's, and into them
    (dict(xs=200, ys=192, y=M + 128), BAD),                  # rows that drift into one another
    (dict(bias=3 * M + 512), BAD), (dict(bias=3 * M + 1024), PASS),
    (dict(ys=512, bias=3 * M + 256), PASS),                  # in the gap between y's rows
    (dict(res=3 * M, rs=128), PASS), (dict(res=3 * M + 256, rs=128), BAD), (dict(res=3 * M + 512, rs=0), BAD),
    (dict(ys=256, res=3 * M + 256, rs=256), PASS),
])
def test_linear(change, status):
    assert _linear(**{**change, "wb": 0}) == status


@pytest.mark.parametrize("change,status", [
    # q [4, 4 x 128] at 1 MB, caches of 8 x 16 x 128 at 3 and 4 MB, out [4, 4, 128] at 9 MB
    (dict(out=M + 1024), BAD), (dict(out=M + 4096), PASS), (dict(qs=1024, out=M + 1024), BAD),
    (dict(out=3 * M + 32768 - 16), BAD), (dict(out=3 * M + 32768), PASS), (dict(out=4 * M - 4096 + 16), BAD),
    (dict(lse=9 * M + 64), BAD), (dict(lse=9 * M + 4096), PASS), (dict(lse=4 * M), BAD), (dict(lse=M), BAD),
    (dict(cap=0, width=0, out=3 * M), PASS),  # no pages: the caches are not read
])
def test_attention(change, status):
    assert _attention(**{**change, "wb": 0}) == status


@pytest.mark.parametrize("change,status", [
    # q [4, 4 x 128] at 1 MB, k, v [4, 128] at 2 and 3 MB, q_out at 6 MB, caches of 16 x 128 at 7 and 8 MB
    (dict(qo=M), PASS), (dict(qs=1024, qo=M), BAD), (dict(T=1, qs=1024, qo=M), PASS),  # in place, with q's stride
    (dict(qo=M + 1024), BAD), (dict(qo=M + 4096), PASS),
    (dict(qs=768, k=M + 1024, ks=768, v=M + 1280, vs=768, qo=M, qos=768), PASS),       # in place in a fused projection
    (dict(qs=768, k=M + 1024, ks=768, v=M + 1280, vs=768, qo=M + 256, qos=768), BAD),
    (dict(k=6 * M), BAD), (dict(v=6 * M + 2048), BAD), (dict(kc=6 * M), BAD), (dict(vc=6 * M + 4096 - 16), BAD),
    (dict(vc=7 * M), BAD), (dict(vc=7 * M + 4096), PASS), (dict(v=None, vc=None), PASS),
    (dict(k=7 * M), PASS),                                   # keys that lie in the cache: the caller's rows
])
def test_rope(change, status):
    assert _rope(**{**change, "wb": 0}) == status
