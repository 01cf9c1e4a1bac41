"""Sizes at the end of the integers, on the host: refused before anything is enqueued."""
import ctypes

import pytest

from score_top_expert_gb300 import build as Build

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks
MOST = 2_000_000_000            # MR_MAX_ROWS
PAST = [MOST + 1, 2 ** 31 - 10_000, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def L():
    Build.build()
    import score_top_expert_gb300.router as r
    return r.lib()


@pytest.mark.parametrize("T", PAST)
def test_balance_refuses_more_rows_than_its_row_numbers_hold(L, T):
    assert L.router_balance_loss_workspace_bytes(T, 1, 1) == 0
    assert L.router_balance_loss_fwd(FAKE, 1, FAKE, 1, None, T, 1, 1, 1, 0, 1.0, 0.0, FAKE, FAKE, FAKE,
                                     FAKE, 1 << 62, None) == -2
    assert L.router_balance_loss_bwd(FAKE, FAKE, 1, FAKE, FAKE, None, T, 1, 1, 1, 0, 1.0, 0.0, FAKE,
                                     None) == -2


@pytest.mark.parametrize("T", PAST)
def test_norms_refuse_more_rows_than_their_row_numbers_hold(L, T):
    assert L.router_combine_norm_bwd_workspace_bytes(T, 1) == 0
    assert L.router_combine_norm_fwd(FAKE, 1, None, None, 0, FAKE, FAKE, None, 0, 1.0, FAKE, 1e-6, T, 1,
                                     1, FAKE, FAKE, None, None, None) == -2
    assert L.router_combine_norm_bwd(FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, None, 0, 1.0, FAKE, T, 1,
                                     FAKE, FAKE, None, FAKE, FAKE, FAKE, 1 << 62, None) == -2


@pytest.mark.parametrize("P", PAST)
def test_products_refuse_more_rows_than_their_tiles_count(L, P):
    assert L.router_expert_matmul_w8(FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, P, 1, 1, 1, FAKE, 1,
                                     None) == -2
    assert L.router_expert_matmul_w8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, P, 2304, 1, 16, FAKE, 0,
                                     None) == -2
    assert L.router_expert_matmul(FAKE, 1, FAKE, FAKE, None, 0, P, 1, 1, 1, FAKE, 1, None) == -2
    assert L.router_expert_matmul_bwd_input(FAKE, 1, FAKE, FAKE, P, 1, 1, 1, FAKE, 1, None) == -2
    assert L.router_expert_matmul_bwd_weight(FAKE, 1, FAKE, FAKE, None, 0, P, 1, 1, 1, FAKE, 0,
                                             None) == -2


def test_the_largest_row_counts_have_workspaces(L):
    assert L.router_balance_loss_workspace_bytes(MOST, 1, 1) > 0
    assert L.router_combine_norm_bwd_workspace_bytes(MOST, 1) > 0
