"""Refusals of glu_lora, linear_lora and moe_glu: host-side validation (pointers are
never dereferenced) and the binding's checks."""
import ctypes

import pytest
import torch

import memory_bound_glu_gb300 as mb
from memory_bound_glu_gb300.binding import _Adapters

HUGE = 2 ** 31 - 511
OK, NULL, SHAPE, STRIDE, ALIGN, MODE, ALIAS = range(7)
X, W, U, A, B, A2, B2, I, S, O, WS, D, R = (0x7F0000000000 + i * (1 << 36) for i in range(13))


def lora(x=X, ldx=64, w=W, ldw=64, u=U, ldu=64, a=A, aa=64 * 8, lda=64, b=B, ba=8 * 32, ldb=8, a2=A2, b2=B2, none=False, idx=I, scale=S,
         o=O, ldo=32, M=20, N=32, K=64, L=3, r=8, mode=0, ws=WS, wsb=1 << 30, second=False):
    q, q2 = _Adapters(a, aa, lda, b, ba, ldb), _Adapters(a2, aa, lda, b2, ba, ldb)
    two = mb.lib().glu_lora(x, ldx, w, ldw, u, ldu, None if none else ctypes.byref(q), None if none else ctypes.byref(q2), idx, scale,
                            o, ldo, M, N, K, L, r, mode, ws, wsb, None)
    assert mb.last_variant() == 0
    if not second:   # what is wrong is not the second projection
        assert two == mb.lib().linear_lora(x, ldx, w, ldw, None if none else ctypes.byref(q), idx, scale, o, ldo, M, N, K, L, r, ws, wsb, None)
        assert mb.last_variant() == 0
    return two


@pytest.mark.parametrize("kw,code", [
    (dict(mode=2, second=True), MODE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(L=-1), SHAPE), (dict(r=-1), SHAPE),
    (dict(r=129), SHAPE), (dict(M=HUGE), SHAPE), (dict(K=HUGE), SHAPE), (dict(L=HUGE), SHAPE), (dict(N=2 ** 30, ldo=2 ** 30), SHAPE),
    (dict(wsb=20 * 16 * 4 - 1, second=True), SHAPE), (dict(wsb=0), SHAPE),
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(u=0, second=True), NULL), (dict(o=0), NULL), (dict(a=0), NULL), (dict(b=0), NULL), (dict(a2=0, second=True), NULL),
    (dict(b2=0, second=True), NULL), (dict(none=True), NULL), (dict(idx=0), NULL), (dict(ws=0), NULL),
    (dict(ldx=63), STRIDE), (dict(ldw=1), STRIDE), (dict(ldu=63, second=True), STRIDE), (dict(ldo=31), STRIDE), (dict(lda=63), STRIDE), (dict(ldb=7), STRIDE),
    (dict(aa=-1), STRIDE), (dict(ba=-8), STRIDE),
    (dict(x=X + 1), ALIGN), (dict(w=W + 1), ALIGN), (dict(u=U + 1, second=True), ALIGN), (dict(o=O + 1), ALIGN), (dict(a=A + 1), ALIGN),
    (dict(b2=B2 + 1, second=True), ALIGN), (dict(idx=I + 2), ALIGN), (dict(scale=S + 1), ALIGN), (dict(ws=WS + 128), ALIGN),
    (dict(o=X + 2 * 64 * 19), ALIAS), (dict(o=W), ALIAS), (dict(o=U + 64, second=True), ALIAS), (dict(o=A + 2 * 3 * 8 * 64 - 2), ALIAS), (dict(o=B2, second=True), ALIAS),
    (dict(o=I), ALIAS), (dict(o=S + 8), ALIAS), (dict(o=WS), ALIAS), (dict(ws=X), ALIAS), (dict(ws=A), ALIAS), (dict(ws=B2, second=True), ALIAS),
    (dict(ws=I), ALIAS), (dict(ws=U, second=True), ALIAS),
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=0, w=0, u=0, o=0, none=True, idx=0, ws=0, wsb=0), OK),
])
def test_lora(kw, code):
    assert lora(**kw) == code


def moe(h=X, ldh=64, r=R, ldr=64, g=A, ge=64 * 40, ldg=64, u=U, ue=64 * 40, ldu=64, d=D, de=64 * 40, ldd=40, o=O, ldo=64, ids=I, w=S,
        T=20, E=6, k=2, N=40, K=64, ws=WS, wsb=1 << 30):
    st = mb.lib().moe_glu(h, ldh, r, ldr, g, ge, ldg, u, ue, ldu, d, de, ldd, o, ldo, ids, w, T, E, k, N, K, 1, ws, wsb, None)
    assert mb.last_variant() == 0
    return st


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(T=65), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE), (dict(k=0), SHAPE), (dict(k=7), SHAPE),
    (dict(E=100, k=17), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(N=HUGE), SHAPE), (dict(K=HUGE), SHAPE), (dict(wsb=256), SHAPE),
    (dict(h=0), NULL), (dict(r=0), NULL), (dict(g=0), NULL), (dict(u=0), NULL), (dict(d=0), NULL), (dict(o=0), NULL), (dict(ws=0), NULL),
    (dict(ldh=63), STRIDE), (dict(ldr=63), STRIDE), (dict(ldg=63), STRIDE), (dict(ldu=63), STRIDE), (dict(ldd=39), STRIDE),
    (dict(ldo=63), STRIDE), (dict(ge=-1), STRIDE), (dict(ue=-64), STRIDE), (dict(de=-1), STRIDE),
    (dict(h=X + 1), ALIGN), (dict(r=R + 1), ALIGN), (dict(d=D + 1), ALIGN), (dict(o=O + 1), ALIGN), (dict(ids=I + 2), ALIGN),
    (dict(w=S + 1), ALIGN), (dict(ws=WS + 16), ALIGN),
    (dict(o=X), ALIAS), (dict(o=R + 2), ALIAS), (dict(o=A + 2 * 6 * 64 * 40 - 2), ALIAS), (dict(o=U), ALIAS), (dict(o=D), ALIAS),
    (dict(ids=O), ALIAS), (dict(w=I + 4), ALIAS), (dict(w=D), ALIAS), (dict(ws=O), ALIAS), (dict(ws=D), ALIAS), (dict(ws=I), ALIAS),
    (dict(ws=A - 256), ALIAS),
    (dict(T=0), OK), (dict(T=0, h=0, r=0, g=0, u=0, d=0, o=0, ws=0, wsb=0), OK),
])
def test_moe(kw, code):
    assert moe(**kw) == code


def test_workspace_sizes():
    assert mb.glu_lora_workspace_bytes(0, 32, 64, 3, 8) == 0 and mb.glu_lora_workspace_bytes(4, 32, 64, 3, 0) == 0
    assert mb.linear_lora_workspace_bytes(4, 32, 64, 0, 8) == 0 and mb.linear_lora_workspace_bytes(4, 32, -1, 3, 8) == 0
    assert mb.glu_lora_workspace_bytes(7, 32, 64, 3, 8) >= 7 * 16 * 4
    assert mb.moe_glu_workspace_bytes(0, 6, 2, 40, 64) == 0 and mb.moe_glu_workspace_bytes(65, 6, 2, 40, 64) == 0
    sizes = [mb.moe_glu_workspace_bytes(T, 6, 2, 40, 64) for T in range(1, 65)]
    assert sizes == sorted(sizes) and sizes[0] > mb.MOE_COUNTER_BYTES


BF = torch.bfloat16


def test_binding_refuses():
    x, w = torch.zeros(4, 64, dtype=BF), torch.zeros(32, 64, dtype=BF)
    a, b, i = torch.zeros(3, 8, 64, dtype=BF), torch.zeros(3, 32, 8, dtype=BF), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mb.linear_lora(x, w, a, b, i)
    with pytest.raises(TypeError, match="bfloat16"):
        mb.linear_lora(x.float(), w, a, b, i)
    with pytest.raises(ValueError, match="CUDA"):
        mb.glu_lora(x, w, w, a, b, a, b, i)
    with pytest.raises(TypeError, match="Tensor"):
        mb.glu_lora(None, w, w, a, b, a, b, i)
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_glu(x, w, torch.zeros(32, 8, 64, dtype=BF), torch.zeros(32, 8, 64, dtype=BF), torch.zeros(32, 64, 8, dtype=BF), 2)
    with pytest.raises(TypeError, match="bfloat16"):
        mb.moe_glu(x.half(), w, None, None, None, 2)


gpu = pytest.mark.gpu


@gpu
def test_binding_refuses_on_the_gpu():
    def z(*s, dtype=BF):
        return torch.zeros(*s, dtype=dtype, device="cuda")

    x, w, a, b, i, s = z(4, 64), z(32, 64), z(3, 8, 64), z(3, 32, 8), z(4, dtype=torch.int32), z(3, dtype=torch.float32)
    mb.linear_lora(x, w, a, b, i, s)
    for bad in ((x, w[:, :32], a, b, i, s), (x, w, a[:, :, :32], b, i, s), (x, w, a, b[:2], i, s), (x, w, a, b[:, :, :4], i, s),
                (x, w, a, b, i[:3], s), (x, w, a, b, i.long(), s), (x, w, a, b, i, s[:2]), (x, w, a, b, i, s.double()),
                (x, w, a[0], b, i, s), (x, w, z(3, 136, 64), z(3, 32, 136), i, s), (x, w, a, b, i.cpu(), s), (x, w, a.transpose(1, 2), b, i, s),
                (x, w, a, b, torch.zeros(8, dtype=torch.int32, device="cuda")[::2], s)):
        with pytest.raises((ValueError, TypeError)):
            mb.linear_lora(*bad)
        with pytest.raises((ValueError, TypeError)):
            mb.glu_lora(bad[0], bad[1], bad[1], bad[2], bad[3], bad[2], bad[3], *bad[4:])
    with pytest.raises(mb.MbgluError, match="SHAPE"):
        mb.linear_lora(x, w, a, b, i, s, workspace=z(16, dtype=torch.uint8))
    with pytest.raises(mb.MbgluError, match="ALIAS"):
        mb.linear_lora(z(4, 32), z(32, 32), z(3, 8, 32), b, i, s, out=b.view(-1)[:128].view(4, 32))
    with pytest.raises(KeyError):
        mb.glu_lora(x, w, w, a, b, a, b, i, s, mode="other")
    h, r, g, d = z(4, 64), z(6, 64), z(6, 16, 64), z(6, 64, 16)
    mb.moe_glu(h, r, g, g, d, 2)
    for bad in ((h, r[:5], g, g, d, 2), (h, r, g[:, :8], g, d, 2), (h, r, g, g, d[:, :32], 2), (h, r, g, g, d, 0), (h, r, g, g, d, 7),
                (z(65, 64), r, g, g, d, 2), (h, r, g, g.float(), d, 2), (h, r, g[0], g, d, 2), (h[0], r, g, g, d, 2),
                (h, r, g.transpose(1, 2), g, d, 2)):
        with pytest.raises((ValueError, TypeError)):
            mb.moe_glu(*bad)
    for bad in (dict(ids=z(4, 2)), dict(weights=z(4, 2)), dict(ids=z(4, 4, dtype=torch.int32)[:, ::2]), dict(out=z(4, 63))):
        with pytest.raises((ValueError, TypeError)):
            mb.moe_glu(h, r, g, g, d, 2, **bad)
    with pytest.raises(mb.MbgluError, match="SHAPE"):
        mb.moe_glu(h, r, g, g, d, 2, workspace=z(256, dtype=torch.uint8))
