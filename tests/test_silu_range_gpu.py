"""SiLU of the wide kernels where e^-|g| is no longer a normal number: an error that
is small beside the smallest normal number, whatever the up product makes of it."""
import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 20, 100, 300])
@pytest.mark.parametrize("mode", ["fused", "hf"])
def test_far_negative_gates(M, mode):
    """g = -60 to -128 exactly, u = 2^100.  Up to |g| = 87 the relative error of SiLU is below
    2^-20; beyond, e^-|g| is a subnormal with at most 3 roundings of 2^-149, and SiLU is
    that times |g|: below |g| 2^-146."""
    g = -torch.arange(60, 128.5, 0.5, device="cuda")
    N = g.numel()
    h, gw, uw = torch.zeros(M, 8, device="cuda"), torch.zeros(N, 8, device="cuda"), torch.zeros(N, 8, device="cuda")
    h[:, :2] = 1
    gw[:, 0], uw[:, 1] = g, 2.0 ** 100
    h, gw, uw = (t.bfloat16() for t in (h, gw, uw))
    assert (gw[:, 0].float() == g).all()
    s = R.silu(g.double())
    err = 2.0 ** -20 * s.abs() + g.double().abs() * 2.0 ** -146
    if mode == "hf":   # SiLU rounds to bf16, whose smallest step is 2^-133
        err = err + R.EPS_BF16 * (s.abs() + err) + 2.0 ** -134
    v = s * 2.0 ** 100
    bound = 2.0 ** 100 * err + R.EPS_BF16 * (v.abs() + 2.0 ** 100 * err)
    buf = torch.empty(M, 2 * N, device="cuda")
    for gu in (None, buf):
        out = mb.glu_gemm(h, gw, uw, mode=mode, gu=gu)
        assert ((out.double() - v).abs() <= bound).all()
    assert torch.equal(buf[:, :N], g.expand(M, N))
