"""glu_gemm_backward where grad_gate and grad_up are split over the rows: tiles left
over from full rounds of SM pairs, in ranges whose partial sums are joined."""
import pytest
import torch

import memory_bound_glu_gb300 as mb
from test_block_plan_model import TILE, ceil_div, pair_plan
from test_glu_gemm_gpu import check_backward, operands, rand

pytestmark = pytest.mark.gpu


def plans(M, N, K):
    """(grad_h's, grad_gate's and grad_up's)"""
    return (pair_plan(M, K, 256, 1, 2 * ceil_div(N, 64), True), pair_plan(N, K, 256, 2, ceil_div(M, 64), True))


def workspace(M, N, K):
    parts = [p["rest"] * p["splits"] * TILE * TILE * 4 for p in plans(M, N, K)]
    return ceil_div(4 * M * ceil_div(N, 64) * 64, 256) * 256 + max(parts)


# only ranges, of both outputs; full rounds and ranges; rows of the outputs that lie on
# 8 bytes, and that do not
@pytest.mark.parametrize("M,N,K,pad,whole,rest", [(2500, 300, 264, 0, 0, 8), (2000, 72, 136, 0, 0, 2), (2333, 257, 515, 5, 0, 12),
                                                  (2500, 2500, 1000, 0, 76, 4), (3100, 2001, 1703, 1, 76, 36)])
@pytest.mark.parametrize("gu", [False, True])
def test_split_weight_gradients(M, N, K, pad, whole, rest, gu):
    p = plans(M, N, K)[1]
    assert (p["whole"], p["rest"]) == (whole, rest) and p["splits"] > 1
    assert mb.glu_gemm_backward_workspace_bytes(M, N, K) == workspace(M, N, K)
    ops = operands(M, N, K, seed=M, pad=pad)
    d = rand(M, N, seed=5)
    whole_call = check_backward(*ops, d, gu=gu)
    assert mb.last_backward_path() == 4
    again = check_backward(*ops, d, gu=gu, want_h=False)
    assert again[0] is None and all(torch.equal(a, b) for a, b in zip(again[1:], whole_call[1:]))
