"""What the launchers of the 8-bit row operators choose, on the host."""

import math
import os
import random

import pytest

from quantized_base_rank_amd import _lib
from tests import q8_plans as P

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libqlin.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("M", [65, 96, 100, 128])
@pytest.mark.parametrize("N,K", [(8192, 28672), (16384, 16384), (8192, 8192), (12288, 24576)])
def test_few_row_tiles_fit_their_rows(M, N, K):
    """Where the weights' stream bounds the product, 65 to 128 tokens take one tile of 128 rows: a taller one would be
    padding, a lower one would read the weights twice."""
    assert P.gemm_shape(M, N, K)[0] == 2


def test_shares_fill_the_card_where_the_stream_bounds():
    """128 x 8192 x 28672: eight shares (256 workgroups) measured faster than six (192)."""
    assert P.gemm_shape(128, 8192, 28672) == (2, 8)


def test_large_products_keep_their_tiles():
    assert P.gemm_shape(4096, 8192, 28672) == (4, 1)
    assert P.gemm_shape(333, 32003, 4096) == (3, 1)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def test_gpu_cases_take_every_path_of_the_product():
    rng = random.Random(5)
    seen = {P.product_path(_log(rng, 1, 4200), _log(rng, 16, 40000), 16 * _log(rng, 1, 2500)) for _ in range(20000)}
    seen |= {P.product_path(rng.randint(1, 64), rng.randint(8129, 8192), 16 * rng.randint(1024, 2048)) for _ in range(200)}
    taken = {P.product_path(*c) for c in P.PRODUCTS}
    assert seen <= taken, seen - taken
    # ... with rows and columns that end inside a tile
    ragged = {P.product_path(M, N, K) for M, N, K in P.PRODUCTS if N % 8 and M % 16}
    assert {p for p in taken if p[0] == "many"} <= ragged and len([p for p in ragged if p[0] == "few"]) == 15


def test_gpu_cases_take_every_path_of_the_backward():
    rng = random.Random(6)
    sizes = [(_log(rng, 1, 20000), 16 * _log(rng, 1, 700), 64 * _log(rng, 1, 450), rng.randint(1, 128)) for _ in range(20000)]
    seen, taken = ({P.token_path(*c) for c in cs} for cs in (sizes, [c[:4] for c in P.BACKWARDS]))
    assert seen <= taken, seen - taken
    seen, taken = ({P.du_path(M, N, r) for M, N, _, r, *_ in cs} for cs in (sizes, P.BACKWARDS))
    assert seen <= taken, seen - taken
    for path in {P.token_path(*c[:4]) for c in P.BACKWARDS}:  # pooled and not, where dA is in shares
        pools = {c[4] for c in P.BACKWARDS if P.token_path(*c[:4]) == path}
        assert pools <= {1, 32}
    assert {c[4] for c in P.BACKWARDS if P.token_path(*c[:4])[2]} == {1, 32}
