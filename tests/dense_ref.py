"""The gated block's definitions in 64 bits, and how far a right kernel may be
from them.

Bounds (each from the arithmetic alone):
  * a rounding to a type is off by at most half a step: eps / 2 of the value
    (bf16 2^-8, e4m3 2^-4, with half the smallest step, 2^-10, near zero);
  * a sum of n products in fp32, in any order and with adds that may truncate
    (a tensor core's), is off by at most (n + 32) 2^-23 sum |a b|: each of the n
    products enters at most n adds of relative error 2^-23, and 32 covers the
    joins of partial sums;
  * SiLU and its derivative in fp32: a few roundings, 2^-20 of the value.
"""
import torch

EPS_BF16, EPS_E4M3, STEP_E4M3 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10
B = 128


def acc(n):
    return (n + 32) * 2.0 ** -23


def silu(g):
    return g * torch.sigmoid(g)


def dsilu(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


def blocks(n):
    return -(-n // B)


def spread_rows(s, K):
    return s.double().repeat_interleave(B, 1)[:, :K]


def spread_blocks(s, N, K):
    return s.double().repeat_interleave(B, 0)[:N].repeat_interleave(B, 1)[:, :K]


def glu(h, gw, uw):
    """(g, u, their error bounds), h and weights in 64 bits."""
    K = h.shape[1]
    return h @ gw.T, h @ uw.T, acc(K) * (h.abs() @ gw.abs().T), acc(K) * (h.abs() @ uw.abs().T)


def glu_out(g, u, eg, eu):
    """SiLU(g) u and its error bound before the last rounding: |SiLU'| <= 1.1."""
    v = silu(g) * u
    return v, 1.1 * eg * (u.abs() + eu) + (silu(g).abs() + 1.1 * eg) * eu + 2.0 ** -20 * v.abs()


def assert_bf16(got, ref, err, what=""):
    bound = EPS_BF16 * (ref.abs() + err) + err + 1e-37
    d = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    worst = (d / bound).max().item() if d.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def amax_groups(v):
    K = v.shape[1]
    pad = blocks(K) * B - K
    return torch.nn.functional.pad(v.abs(), (0, pad)).view(v.shape[0], -1, B).amax(2)


def assert_e4m3(q, scale, v, err, what=""):
    """q and its scales against the values v (64 bits) that they stand for;
    err bounds the values' own error."""
    K = v.shape[1]
    want = (amax_groups(v) / 448).clamp_min(2.0 ** -126)
    es = amax_groups(err) / 448 + 2.0 ** -22 * want
    d = (scale.double() - want).abs()
    assert (d <= es).all(), f"{what}: scale {(d / es).max().item():.3f} of the bound"
    s = spread_rows(scale, K)
    x = q.double() * s
    bound = EPS_E4M3 * (v.abs() + err) * (1 + 2.0 ** -20) + STEP_E4M3 * s + err + 2.0 ** -20 * v.abs()
    # a value that its scale's error lifts past 448 saturates there
    bound = bound + spread_rows(es, K) * 448
    d = (x - v).abs()
    worst = (d / bound).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def quantise_rows(v):
    s = (amax_groups(v) / 448).clamp_min(2.0 ** -126).float()
    return (v / spread_rows(s, v.shape[1])).float().to(torch.float8_e4m3fn), s


def quantise_blocks(w):
    N, K = w.shape
    nb, kb = blocks(N), blocks(K)
    a = torch.nn.functional.pad(w.abs(), (0, kb * B - K, 0, nb * B - N)).view(nb, B, kb, B).amax((1, 3))
    s = (a / 448).clamp_min(2.0 ** -126).float()
    return (w / spread_blocks(s, N, K)).float().to(torch.float8_e4m3fn), s
