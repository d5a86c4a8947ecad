"""What the launchers of the 8-bit row operators choose, on the host."""

import os

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
