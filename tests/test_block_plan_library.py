"""The plans that the library makes against the CPU models of them, and the models'
exchange between the warps of g and u."""
import itertools

import pytest

import memory_bound_glu_gb300 as mb
import test_block_plan_model as model
from test_block_plan_model import PAIRS, TILE, ceil_div, pair_plan

ROWS = (1, 16, 17, 48, 64, 65, 100, 129, 200, 333, 448, 500, 768, 1000, 2100, 4096, 100000)
COLS = (1, 79, 128, 300, 1000, 2504, 4096, 9728, 11008, 14336)
INNER = (1, 64, 72, 128, 1000, 2560, 4096, 9728)


def of_pair(p, tile_cols):
    return 0, TILE, tile_cols, p["whole"], p["rest"], p["splits"]


def modelled(product, M, N, K):
    if product == "glu_gemm":
        tn = model.gemm_tokens(M, N, K)
        if tn:
            wt = model.gemm_outputs(M, N, tn)
            return 1, tn, wt, ceil_div(N, wt) * ceil_div(M, tn), 0, 1
        return of_pair(pair_plan(M, N, 128, 1, ceil_div(K, 64), False), 128)
    if product == "grad_h":
        return of_pair(pair_plan(M, K, 256, 1, 2 * ceil_div(N, 64), True), 256)
    if product == "grad_w":
        return of_pair(pair_plan(N, K, 256, 2, ceil_div(M, 64), True), 256)
    dual = product == "glu_fp8"
    kind, *rest = model.fp8_plan(M, N, K, dual)
    if kind == "pair":
        return of_pair(rest[0], 128 if dual else 256)
    tn, ks = rest
    tiles = ceil_div(N, 128) * ceil_div(M, tn)
    return (1, tn, 128, tiles, 0, 1) if ks == 1 else (1, tn, 128, 0, tiles, ks)


@pytest.mark.parametrize("product", mb.binding.PRODUCTS)
def test_every_plan_is_the_models(product):
    seen = set()
    for M, N, K in itertools.product(ROWS, COLS, INNER):
        got = mb.block_plan(product, M, N, K)
        assert got == modelled(product, M, N, K), (M, N, K)
        seen.add((got[0], got[4] > 0))
    few, split = (1, True), (0, True)
    assert (0, False) in seen
    assert (few in seen) == ("fp8" in product) and (split in seen) == (product in ("grad_h", "grad_w", "matmul_fp8"))


@pytest.mark.parametrize("product", ["glu_fp8", "matmul_fp8"])
def test_few_row_tiles_of_e4m3(product):
    """Every width that the kernels are instantiated for is chosen somewhere, and no other."""
    got = {mb.block_plan(product, M, N, K)[1] for M in range(1, 500, 3) for N in (128, 1000, 2560, 9728, 11008)
           for K in (128, 1000, 2560, 9728)}
    assert got == {16, 32, 48, TILE} | ({64, 80, 96, 112, 128} if product == "matmul_fp8" else set())


def test_tiles_of_glu_gemm():
    got = {mb.block_plan("glu_gemm", M, N, K)[1:3] for M in range(17, 700, 3) for N in (300, 2504, 3350, 5500, 9728, 11008)
           for K in (72, 264, 1000, 1648, 2960, 3176)}
    assert {tn for tn, _ in got} == {*range(32, 256, 32), TILE} and {wt for _, wt in got} == {80, 96, 128}


def test_refusals():
    def status(product=0, M=5, N=5, K=5, plan=(mb.binding.ctypes.c_int * 6)()):
        return mb.lib().mbglu_block_plan(product, M, N, K, plan)
    assert status() == 0 and status(plan=None) == 1
    assert status(product=-1) == status(product=5) == 5
    for bad in (dict(M=0), dict(N=0), dict(K=0), dict(M=-1), dict(M=2 ** 31 - 1), dict(N=2 ** 30), dict(K=2 ** 31 - 511)):
        assert status(**bad) == 2
    for product, kw in enumerate((dict(M=2 ** 30, N=2 ** 29), dict(M=2 ** 30, K=2 ** 30), dict(N=2 ** 29, K=2 ** 30),
                                  dict(M=2 ** 30, N=2 ** 29), dict(M=2 ** 30, N=2 ** 29))):
        assert status(product=product, **kw) == 2
    for product in range(5):   # 2^36 elements
        assert status(product=product, M=2 ** 18, N=2 ** 18, K=2 ** 18) == 0
    with pytest.raises(ValueError):
        mb.block_plan("other", 1, 1, 1)


@pytest.mark.parametrize("tn", range(32, 256, 32))
def test_a_warp_reads_what_its_partner_wrote(tn):
    """Of 16 tokens the warp of g works on the first 8 and the warp of u on the others;
    each writes what the other needs where the other reads it."""
    for half, q0 in itertools.product((0, 1), (0, 1)):
        sets = 0
        for j in range(0, tn // 2, 16):
            first = half * (tn // 2) + j
            place = {}
            for side in (0, 1):   # g[tokens], u[tokens]; side 0 hands over the second eight, side 1 the first
                for i in range(8):
                    r = i if side else 8 + i
                    place[(sets & 1) * 512 + side * 256 + i * 32] = ("gu"[side], first + r)
            for side in (0, 1):
                for i in range(8):
                    token = first + side * 8 + i
                    own = ("gu"[side], first + (8 + i if side else i))
                    theirs = place[(sets & 1) * 512 + (side ^ 1) * 256 + i * 32]
                    assert {own, theirs} == {("g", token), ("u", token)}
            sets += 1


def test_rounds_count_the_pairs():
    assert PAIRS == 76 and all(mb.block_plan("grad_w", 4096, N, K)[3] % PAIRS == 0 or mb.block_plan("grad_w", 4096, N, K)[4] == 0
                               for N in (300, 2500, 9728) for K in (1000, 2560))
