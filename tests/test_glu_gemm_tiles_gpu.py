"""glu_gemm's kernel with the weights on the 256-row side, at every width of tokens
and of outputs that its rule chooses: both modes, with and without g and u."""
import pytest

import memory_bound_glu_gb300 as mb
from test_glu_gemm_gpu import check_forward, operands

pytestmark = pytest.mark.gpu

SIZES = [
    (32, 80, 877, 130, 136), (32, 96, 71, 2220, 72), (32, 128, 195, 962, 64), (64, 80, 422, 642, 64), (64, 96, 133, 2377, 64),
    (64, 128, 260, 1446, 64), (96, 80, 81, 5097, 208), (96, 96, 529, 1039, 72), (96, 128, 389, 1496, 64),
    (128, 80, 121, 5606, 264), (128, 96, 107, 6513, 272), (128, 128, 102, 7821, 272), (160, 80, 131, 5734, 712),
    (160, 96, 285, 3355, 712), (160, 128, 136, 7454, 728), (192, 80, 173, 5221, 1624), (192, 96, 325, 3398, 1512),
    (192, 128, 339, 3702, 1488), (224, 96, 402, 3353, 3104), (224, 128, 579, 2444, 3104), (224, 128, 869, 2432, 3176)]


@pytest.mark.parametrize("tn,wt,M,N,K", SIZES)
def test_each_width(tn, wt, M, N, K):
    assert mb.block_plan("glu_gemm", M, N, K)[:3] == (1, tn, wt)
    for mode, gu in (("fused", False), ("hf", True)):
        check_forward(*operands(M, N, K, seed=M), mode=mode, gu=gu)
        assert mb.last_variant() == 11


@pytest.mark.parametrize("M,N", [(671, 2433), (672, 2433), (671, 2559), (672, 2559), (671, 2560)])
def test_edges_of_the_widest_tile(M, N):
    """Three tiles of 224 tokens, full or one short; the last tile of outputs with one, all but one, all."""
    K = 3176
    assert mb.block_plan("glu_gemm", M, N, K)[:3] == (1, 224, 128)
    check_forward(*operands(M, N, K, seed=M + N), gu=True)
