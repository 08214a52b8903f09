"""Products with low-rank adapters and the expert layer: their definitions in 64 bits,
row by row, and how far a right kernel may be from them.

Bounds, beside dense_ref's for a rounding, an fp32 sum and SiLU:
  * a number carried as two bf16 terms is off by at most 2^-18 of it (each term is half
    a step, 2^-9, of what is left to it);
  * a softmax weight: expf of a difference d that was rounded, 2^-24 |d|, expf's two
    units and the sum of n such terms: (32 + |d| + n) 2^-23 of it, and below 2^-126,
    where fp32 numbers lie 2^-149 apart, two such steps for expf and one for the quotient.
"""
import torch

import dense_ref as R

TWO_TERMS = 2.0 ** -18


def adapted(x, w, a, b, adapter, scale):
    """(y, its error bound) of one projection with adapters, all in 64 bits."""
    x, w, a, b = x.double(), w.double(), a.double(), b.double()
    K, rank = x.shape[1], a.shape[1]
    y, e = x @ w.T, R.acc(K) * (x.abs() @ w.abs().T)
    for i in range(a.shape[0]):
        rows = torch.nonzero(adapter == i)[:, 0]
        if rows.numel() and rank and K:
            s = 1.0 if scale is None else scale[i].double()
            p = s * (x[rows] @ a[i].T)
            ep = abs(s) * R.acc(K) * (x[rows].abs() @ a[i].abs().T) + (TWO_TERMS + 2.0 ** -22) * p.abs()
            d = p @ b[i].T
            y[rows] += d
            e[rows] += ep @ b[i].abs().T + R.acc(2 * rank) * ((p.abs() + ep) @ b[i].abs().T) + 2.0 ** -22 * (y[rows].abs() + d.abs())
    return y, e


def assert_glu_lora(out, args, mode="fused"):
    h, gw, uw, ga, gb, ua, ub, adapter, scale = args
    g, eg = adapted(h, gw, ga, gb, adapter, scale)
    u, eu = adapted(h, uw, ua, ub, adapter, scale)
    if mode == "fused":
        R.assert_bf16(out, *R.glu_out(g, u, eg, eu), "out")
    else:   # g, u and SiLU(g) round to bf16 too
        eg, eu = eg + R.EPS_BF16 * (g.abs() + eg), eu + R.EPS_BF16 * (u.abs() + eu)
        v, e = R.glu_out(g, u, eg, eu)
        R.assert_bf16(out, v, e + R.EPS_BF16 * (v.abs() + e), "out (hf)")


def route(h, router, top_k, renormalize):
    """(ids, weights, the weights' error bound)."""
    logits = (h.double() @ router.double().T).float()
    order, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    v = order.double()
    n = top_k if renormalize else v.shape[1]
    w = torch.exp(v[:, :top_k] - torch.logsumexp(v[:, :n], 1, keepdim=True))
    return ids[:, :top_k], w, (32 + (v[:, :1] - v[:, :top_k]) + n) * 2.0 ** -23 * w + 3 * 2.0 ** -149


def assert_moe(got, h, router, gate, up, down, top_k, renormalize):
    out, ids, weights = got
    want, w, ew = route(h, router, top_k, renormalize)
    assert torch.equal(ids.long(), want), "ids"
    assert ((weights.double() - w).abs() <= ew).all(), "weights"
    K, N = h.shape[1], gate.shape[1]
    y, e = (torch.zeros(h.shape, dtype=torch.float64, device=h.device) for _ in range(2))
    for i in want.unique().tolist():
        rows, j = torch.nonzero(want == i, as_tuple=True)
        x, d = h[rows].double(), down[i].double()
        g, u, eg, eu = R.glu(x, gate[i].double(), up[i].double())
        v, ev = R.glu_out(g, u, eg, eu)
        ev = ev + TWO_TERMS * v.abs()
        z = v @ d.T
        # the sum's parts: 2 N products of two terms, joined
        ez = ev @ d.abs().T + R.acc(2 * N) * ((v.abs() + ev) @ d.abs().T)
        c, ec = w[rows, j][:, None], ew[rows, j][:, None]
        y.index_add_(0, rows, c * z)
        e.index_add_(0, rows, c * ez + ec * (z.abs() + ez) + (top_k + 2) * 2.0 ** -23 * c * (z.abs() + ez))
    R.assert_bf16(out, y, e, "out")
