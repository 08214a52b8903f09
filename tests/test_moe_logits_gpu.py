"""moe_glu's logits where large products cancel: the choice is the exact sums' in every
kernel and at every number of tokens, as far as the bound on the sum decides it."""
import pytest
import torch

import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def bound(h, router):
    """How far a logit may be from the exact sum before its rounding."""
    return (h.shape[1] / 32 + 32) ** 2 * 2.0 ** -48 * (h.double().abs() @ router.double().abs().T)


def experts(E, N, K, pad):
    return [torch.zeros(*s[:-1], s[-1] + pad, dtype=BF, device=DEV)[..., :s[-1]] for s in ((E, N, K), (E, N, K), (E, K, N))]


def view(t, pad):
    """The same values with rows that are not 16-byte aligned."""
    return torch.nn.functional.pad(t, (0, pad))[..., :t.shape[-1]]


def choices(h, router, k, weights=False):
    """ids of all tokens at once, of groups of 8, of single tokens and by the kernels for any alignment."""
    E, K = router.shape
    for pad, step in ((0, h.shape[0]), (0, 8), (0, 1), (1, 8)):
        x, r = view(h, pad), view(router, pad)
        got = [mb.moe_glu(x[i:i + step], r, *experts(E, 8, K, pad), k) for i in range(0, h.shape[0], step)]
        assert mb.last_variant() == (22 if pad else 21)
        yield torch.cat([g[1] for g in got]).long(), torch.cat([g[2] for g in got])


@pytest.mark.parametrize("E,K,k", [(20, 264, 4), (128, 2048, 8), (100, 4104, 7)])
def test_integers_that_cancel(E, K, k):
    """Sums of a few units beside products of 2^20 and more that cancel.  Every rounding is an integer,
    and their sum one below 2^24, so in any order each logit is exact, and equal ones go to the
    lowest index."""
    g = torch.Generator(device=DEV).manual_seed(K)
    T = 16
    h = torch.randint(-3, 4, (T, K), generator=g, device=DEV).double()
    router = torch.randint(-1, 2, (E, K), generator=g, device=DEV).double() * (torch.rand(E, K, generator=g, device=DEV) < 0.02)
    loud = torch.randperm(K, generator=g, device=DEV)[:8]
    for i in range(0, 8, 2):   # a channel and its opposite, far apart in the row
        h[:, loud[i]] = 2.0 ** 12 * torch.randint(1, 8, (T,), generator=g, device=DEV)
        h[:, loud[i + 1]] = -h[:, loud[i]]
        router[:, loud[i]] = 2.0 ** 6 * torch.randint(1, 5, (E,), generator=g, device=DEV)
        router[:, loud[i + 1]] = router[:, loud[i]]
    h, router = h.to(BF), router.to(BF)
    exact = h.double() @ router.double().T
    assert (2.0 ** -24 * (K / 32 + 32) * (h.double().abs() @ router.double().abs().T) < 2 ** 24).all()
    assert exact.abs().max() < 2 ** 20 and exact.unique().numel() < exact.numel() // 4
    order, want = torch.sort(exact, dim=1, descending=True, stable=True)
    for ids, weights in choices(h, router, k):
        assert torch.equal(ids, want[:, :k])
        assert torch.allclose(weights.double(), torch.softmax(order[:, :k], 1), rtol=1e-5, atol=1e-30)


@pytest.mark.parametrize("E,K,k", [(64, 520, 6), (128, 2048, 8)])
def test_loud_channels_that_cancel(E, K, k):
    """Random values with products of some 10^5 that cancel to the others' few units.  Experts whose
    logits differ by more than the bound and the rounding are chosen in their order."""
    g = torch.Generator(device=DEV).manual_seed(K + 1)
    T = 24
    h = torch.randn(T, K, generator=g, device=DEV)
    router = torch.randn(E, K, generator=g, device=DEV) * K ** -0.5
    at = torch.randperm(K, generator=g, device=DEV)[:6]
    for i in range(0, 6, 2):
        h[:, at[i]] = 3000 * (1 + torch.rand(T, generator=g, device=DEV))
        router[:, at[i]] = 30 * torch.randn(E, generator=g, device=DEV)
        h, router = h.to(BF).float(), router.to(BF).float()
        h[:, at[i + 1]], router[:, at[i + 1]] = h[:, at[i]], -router[:, at[i]]
    h, router = h.to(BF), router.to(BF)
    exact = h.double() @ router.double().T
    order, want = torch.sort(exact, dim=1, descending=True, stable=True)
    room = (bound(h, router) + 2.0 ** -24 * exact.abs()).max(1, keepdim=True).values
    clear = (order[:, :k] - order[:, 1:k + 1] > 2 * room).all(1)
    assert clear.sum() > T // 2
    for ids, _ in choices(h, router, k):
        assert torch.equal(ids[clear], want[clear][:, :k])
