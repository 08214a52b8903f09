"""Refusals of the gated block's wide and 8-bit entry points: host-side
validation (pointers are never dereferenced) and the binding's checks."""
import pytest
import torch

import memory_bound_glu_gb300 as mb

HUGE = 2 ** 31 - 511   # one more than the largest size
OK, NULL, SHAPE, STRIDE, ALIGN, MODE, ALIAS = range(7)
A, G, U, O, D, GH, GG, GU, WS, S1, S2, S3, S4, Q = (0x7F0000000000 + i * (1 << 36) for i in range(14))


def gemm(h=A, ldh=64, g=G, ldg=64, u=U, ldu=64, o=O, ldo=32, gu=0, ldgu=64, M=200, N=32, K=64, mode=0):
    return mb.lib().glu_gemm(h, ldh, g, ldg, u, ldu, o, ldo, gu, ldgu, M, N, K, mode, None)


@pytest.mark.parametrize("kw,code", [
    (dict(mode=2), MODE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(N=2 ** 30, ldo=2 ** 30), SHAPE),
    (dict(h=0), NULL), (dict(g=0), NULL), (dict(u=0), NULL), (dict(o=0), NULL),
    (dict(ldh=63), STRIDE), (dict(ldg=63), STRIDE), (dict(ldu=1), STRIDE), (dict(ldo=31), STRIDE), (dict(gu=GU, ldgu=63), STRIDE),
    (dict(h=A + 1), ALIGN), (dict(g=G + 1), ALIGN), (dict(u=U + 1), ALIGN), (dict(o=O + 1), ALIGN), (dict(gu=GU + 2), ALIGN),
    (dict(o=A + 2 * 64 * 199), ALIAS), (dict(o=G), ALIAS), (dict(o=U + 64), ALIAS), (dict(gu=O + 4), ALIAS), (dict(gu=G), ALIAS),
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, h=0, g=0, u=0, o=0), OK),
    (dict(M=HUGE), SHAPE), (dict(K=HUGE), SHAPE),
])
def test_glu_gemm(kw, code):
    assert gemm(**kw) == code
    assert mb.last_variant() == 0


def bwd(h=A, ldh=64, g=G, ldg=64, u=U, ldu=64, d=D, ldd=32, gu=0, ldgu=64, gh=GH, ldgh=64, gg=GG, ldgg=64, gw=GU, ldgw=64,
        M=200, N=32, K=64, ws=WS, wsb=1 << 30):
    return mb.lib().glu_gemm_backward(h, ldh, g, ldg, u, ldu, d, ldd, gu, ldgu, gh, ldgh, gg, ldgg, gw, ldgw, M, N, K, ws,
                                      wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(wsb=100), SHAPE),
    (dict(h=0), NULL), (dict(d=0), NULL), (dict(ws=0), NULL), (dict(gg=0), NULL), (dict(gw=0), NULL),
    (dict(ldh=63), STRIDE), (dict(ldd=31), STRIDE), (dict(ldgh=60), STRIDE), (dict(ldgw=1), STRIDE), (dict(gu=S1, ldgu=63), STRIDE),
    (dict(h=A + 1), ALIGN), (dict(gh=GH + 1), ALIGN), (dict(ws=WS + 128), ALIGN), (dict(gu=S1 + 2), ALIGN),
    (dict(gh=A), ALIAS), (dict(gg=G + 64), ALIAS), (dict(gw=D), ALIAS), (dict(ws=GG), ALIAS), (dict(gw=GG + 2 * 64 * 31), ALIAS),
    (dict(gu=GH), ALIAS),
    (dict(K=0), OK), (dict(M=0, N=0), OK), (dict(gh=0, gg=0, gw=0), OK),
    (dict(M=HUGE), SHAPE), (dict(K=HUGE), SHAPE),
])
def test_glu_gemm_backward(kw, code):
    assert bwd(**kw) == code
    assert mb.last_variant() == 0


def norm(x=A, ldx=256, r=G, ldr=256, ro=G, ldro=256, w=U, q=Q, ldq=256, s=S1, lds=2, M=3, K=256):
    return mb.lib().add_rmsnorm_fp8(x, ldx, r, ldr, ro, ldro, w, 1e-6, q, ldq, s, lds, M, K, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(M=HUGE), SHAPE), (dict(K=HUGE), SHAPE),
    (dict(x=0), NULL), (dict(r=0), NULL), (dict(ro=0), NULL), (dict(w=0), NULL), (dict(q=0), NULL), (dict(s=0), NULL),
    (dict(ldx=255), STRIDE), (dict(ldr=255, ro=O), STRIDE), (dict(ldro=255, ro=O), STRIDE), (dict(ldq=255), STRIDE), (dict(lds=1), STRIDE),
    (dict(x=A + 1), ALIGN), (dict(w=U + 1), ALIGN), (dict(s=S1 + 2), ALIGN),
    (dict(ro=G + 2), ALIAS), (dict(ro=G, ldro=264), ALIAS), (dict(ro=U), ALIAS), (dict(q=A), ALIAS), (dict(q=G), ALIAS),
    (dict(s=Q), ALIAS), (dict(s=U), ALIAS), (dict(q=O, ro=O), ALIAS),
    (dict(M=0), OK),
])
def test_add_rmsnorm_fp8(kw, code):
    assert norm(**kw) == code
    assert mb.last_variant() == 0


def matmul(a=A, lda=256, sa=S1, ldsa=2, w=G, ldw=256, sw=S2, ldsw=2, o=O, ldo=200, M=3, N=200, K=256, ws=WS, wsb=1 << 34):
    return mb.lib().matmul_fp8(a, lda, sa, ldsa, w, ldw, sw, ldsw, o, ldo, M, N, K, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(M=HUGE), SHAPE), (dict(N=HUGE), SHAPE), (dict(K=HUGE), SHAPE),
    (dict(a=0), NULL), (dict(sa=0), NULL), (dict(w=0), NULL), (dict(sw=0), NULL), (dict(o=0), NULL),
    (dict(lda=255), STRIDE), (dict(ldw=255), STRIDE), (dict(ldsa=1), STRIDE), (dict(ldsw=1), STRIDE), (dict(ldo=199), STRIDE),
    (dict(sa=S1 + 2), ALIGN), (dict(sw=S2 + 1), ALIGN), (dict(o=O + 1), ALIGN),
    (dict(o=A), ALIAS), (dict(o=G + 256), ALIAS), (dict(o=S1), ALIAS), (dict(o=S2 + 8), ALIAS),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_matmul_fp8(kw, code):
    assert matmul(**kw) == code
    assert mb.last_variant() == 0


def glu(a=A, lda=256, sa=S1, ldsa=2, g=G, ldg=256, sg=S2, ldsg=2, u=U, ldu=256, su=S3, ldsu=2, o=0, ldo=200, q=Q, ldq=200,
        qs=S4, ldqs=2, M=3, N=200, K=256):
    return mb.lib().glu_fp8(a, lda, sa, ldsa, g, ldg, sg, ldsg, u, ldu, su, ldsu, o, ldo, q, ldq, qs, ldqs, M, N, K, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(M=HUGE), SHAPE), (dict(N=HUGE), SHAPE), (dict(K=HUGE), SHAPE),
    (dict(o=O), NULL), (dict(q=0), NULL), (dict(qs=0), NULL), (dict(q=0, qs=0), NULL), (dict(o=O, q=0), NULL),
    (dict(a=0), NULL), (dict(sg=0), NULL), (dict(u=0), NULL),
    (dict(lda=255), STRIDE), (dict(ldg=255), STRIDE), (dict(ldsu=1), STRIDE), (dict(ldq=199), STRIDE), (dict(ldqs=1), STRIDE),
    (dict(o=O, ldo=199, q=0, qs=0), STRIDE),
    (dict(qs=S4 + 2), ALIGN), (dict(sa=S1 + 2), ALIGN), (dict(o=O + 1, q=0, qs=0), ALIGN),
    (dict(q=A), ALIAS), (dict(q=U + 256), ALIAS), (dict(qs=S3), ALIAS), (dict(qs=Q), ALIAS), (dict(o=G, q=0, qs=0), ALIAS),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_glu_fp8(kw, code):
    assert glu(**kw) == code
    assert mb.last_variant() == 0


def quant(w=A, ldw=256, q=Q, ldq=256, s=S1, lds=2, N=200, K=256):
    return mb.lib().quantize_weight_fp8(w, ldw, q, ldq, s, lds, N, K, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(N=HUGE), SHAPE), (dict(K=HUGE), SHAPE), (dict(w=0), NULL), (dict(q=0), NULL), (dict(s=0), NULL),
    (dict(ldw=255), STRIDE), (dict(ldq=255), STRIDE), (dict(lds=1), STRIDE), (dict(w=A + 1), ALIGN), (dict(s=S1 + 2), ALIGN),
    (dict(q=A + 5), ALIAS), (dict(s=A), ALIAS), (dict(s=Q + 4), ALIAS), (dict(N=0), OK), (dict(K=0), OK),
])
def test_quantize_weight_fp8(kw, code):
    assert quant(**kw) == code
    assert mb.last_variant() == 0


def test_workspace_bytes():
    lib = mb.lib()
    # dG and dU in bf16, rows padded to 64 elements, at least
    assert lib.glu_gemm_backward_workspace_bytes(100, 100, 64) >= 2 * 100 * 128 * 2
    for f in (lib.glu_gemm_backward_workspace_bytes, lib.matmul_fp8_workspace_bytes):
        assert f(0, 10, 10) == 0 and f(10, 0, 10) == 0 and f(-1, 10, 10) == 0 and f(HUGE, 10, 10) == 0


def test_binding_refuses():
    bf = torch.zeros(4, 128, dtype=torch.bfloat16)
    f8 = bf.to(torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    with pytest.raises(ValueError):
        mb.glu_gemm(bf, bf, bf)                      # not on a GPU
    with pytest.raises(TypeError):
        mb.matmul_fp8(bf, s, bf, s)                  # not e4m3
    with pytest.raises(ValueError):
        mb.matmul_fp8(f8, s, f8, s)                  # not on a GPU
    with pytest.raises(TypeError):
        mb.glu_fp8(f8, s, f8, s, f8, s, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mb.matmul_fp8(f8[0], s, f8, s)               # one dimension
    with pytest.raises(TypeError):
        mb.quantize_weight_fp8(bf.float())
