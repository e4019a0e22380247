"""Refusals of the feed-forward entry points that a later call would have to make."""
import pytest

import expert_adapter_gemms_gb300 as m
from test_ffn_cpu import INVALID, OK, P, UNSUPPORTED, L  # noqa: F401


@pytest.mark.parametrize("K", [1, 12, 129, 4100, 16392, 1 << 20])
def test_w4_pack_refuses_what_the_product_refuses(L, K):  # noqa: F811
    """A weight whose columns no product takes is refused when it is packed."""
    N, group = 16, 32
    product = L.moe_w4_matvec(P, 0, P, 1, N, K, group, 0, 0, 0, 4, None, 0, P, 0, 0)
    assert product == UNSUPPORTED
    assert L.moe_w4_pack(P, P, 0, 1, N, K, group, 0, P, 0) == UNSUPPORTED


def test_w4_pack_takes_what_the_product_takes(L):  # noqa: F811
    """Arguments that both take: the pointers are looked at next."""
    for K in (8, 2880, 16384):
        assert L.moe_w4_pack(0, P, 0, 1, 16, K, 32, 0, P, 0) == INVALID
        assert L.moe_w4_matvec(0, 0, P, 1, 16, K, 32, 0, 0, 0, 4, None, 0, P, 0, 0) == INVALID
        assert L.moe_w4_matvec(0, 0, 0, 1, 16, K, 32, 0, 0, 0, 0, None, 0, 0, 0, 0) == OK
