"""Cases of the gated feed-forward block where each row chooses weights of its own: low-rank adapters of many requests
beside the shared projections, and a whole mixture-of-experts layer for a decode batch.

    glu_lora     SiLU(h Wg^T + p_g Bg[a]^T) * (h Wu^T + p_u Bu[a]^T), p = scale[a] (h A[a]^T), a the row's adapter or none
    linear_lora  x W^T + (scale[a] x A[a]^T) B[a]^T: the down projection beside it
    moe          router, top-k, the chosen experts' gated products, their down projections and the weighted sum

All of them serve: a batch of requests' tokens in, bf16 out. `own` selects the framework's calls; otherwise `run` is the
plain form in 32 bits.
"""
import math

import torch

own = False

NO_ADAPTER = 0.1   # the share of requests that use the shared weights alone


def listed():
    return [
        # one decoded token with an adapter: both shared weights are read once, the adapter's are small beside them
        dict(name="glu_lora_token", op="glu_lora", M=1, requests=1, K=2560, N=9728, R=16, L=32, mode="fused"),
        # a decode batch of 48 requests with adapters of their own: the adapters' bytes count
        dict(name="glu_lora_batch48", op="glu_lora", M=48, requests=48, K=2560, N=9728, R=16, L=64, mode="hf"),
        # a chunk of some prompts and decoded tokens together, ragged in every dimension
        dict(name="glu_lora_ragged", op="glu_lora", M=333, requests=37, K=1000, N=2504, R=24, L=40, mode="fused"),
        # a long prompt's chunk of few requests, adapters of a larger rank: arithmetic-bound
        dict(name="glu_lora_prompt", op="glu_lora", M=4096, requests=5, K=2560, N=9728, R=64, L=8, mode="fused"),
        # the down projection of a decode batch of 8
        dict(name="linear_lora_batch8", op="linear_lora", M=8, requests=8, K=9728, N=2560, R=16, L=32),
        # the down projection of a long prompt's chunk
        dict(name="linear_lora_prompt", op="linear_lora", M=2048, requests=6, K=9728, N=2560, R=32, L=16),
        # a small layer at ragged sizes
        dict(name="moe_ragged", op="moe", T=13, E=20, top_k=3, K=1000, N=408, renormalize=False),
        # one decoded token through a layer of many small experts: latency and the chosen experts' bytes
        dict(name="moe_token", op="moe", T=1, E=128, top_k=8, K=2048, N=768, renormalize=True),
        # a decode batch of 8: some fifty experts of one or two rows each
        dict(name="moe_batch8", op="moe", T=8, E=128, top_k=8, K=2048, N=768, renormalize=True),
        # a decode batch of 64: nearly every expert is read
        dict(name="moe_batch64", op="moe", T=64, E=128, top_k=8, K=2048, N=768, renormalize=True),
        # four tokens through a layer of few large experts
        dict(name="moe_large4", op="moe", T=4, E=8, top_k=2, K=4096, N=11008, renormalize=True),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["glu_lora", "glu_lora", "linear_lora", "moe", "moe"])
    if op == "moe":
        K, E = 8 * log_int(32, 512), log_int(4, 128)
        N = 8 * log_int(16, max(16, min(1376, 128 * 768 * 2048 // (8 * K * E))))
        return dict(op=op, T=log_int(1, 64), E=E, top_k=rng.randint(1, min(8, E)), K=K, N=N, renormalize=rng.random() < 0.7)
    M = log_int(1, 4096)
    d = dict(op=op, M=M, requests=min(M, log_int(1, 64)), R=8 * log_int(1, 8), L=log_int(1, 64))
    if op == "glu_lora":
        return dict(d, K=8 * log_int(32, 320), N=log_int(128, 9728), mode=rng.choice(["hf", "fused"]))
    return dict(d, K=8 * log_int(32, 1216), N=log_int(128, 2560))


def _inputs(case, seed):
    """The inputs, from the seed alone: activations with a few loud channels, weights N(0, 1/K)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 6733 + 29)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).bfloat16()

    K, N = case["K"], case["N"]
    loud = torch.ones(K, device=dev)
    loud[torch.randint(K, (max(1, K // 200),), generator=gen, device=dev)] = 6.0
    if case["op"] == "moe":
        E = case["E"]
        return dict(h=(normal(case["T"], K).float() * loud).bfloat16(), router=normal(E, K, scale=K ** -0.5),
                    gate=normal(E, N, K, scale=K ** -0.5), up=normal(E, N, K, scale=K ** -0.5),
                    down=normal(E, K, N, scale=N ** -0.5))
    M, R, L, q = case["M"], case["R"], case["L"], case["requests"]
    d = dict(x=(normal(M, K).float() * loud).bfloat16())
    # the rows of one request lie together and share its adapter
    chosen = torch.randint(L, (q,), generator=gen, device=dev)
    chosen[torch.rand(q, generator=gen, device=dev) < NO_ADAPTER] = -1
    if q < M:
        cuts = torch.randint(M, (q - 1,), generator=gen, device=dev)
        of = (torch.arange(M, device=dev)[:, None] >= cuts[None, :]).sum(1)
    else:
        of = torch.arange(M, device=dev)
    d["adapter"] = chosen[of].int()
    d["scale"] = 0.5 + 1.5 * torch.rand(L, generator=gen, device=dev)
    for side in ("gate", "up") if case["op"] == "glu_lora" else ("",):
        d["w" + side] = normal(N, K, scale=K ** -0.5)
        d["a" + side] = normal(L, R, K, scale=K ** -0.5)
        d["b" + side] = normal(L, N, R, scale=0.3 * R ** -0.5)
    return d


def prepare(case, seed):
    s = dict(case=dict(case), **_inputs(case, seed))
    # the one buffer that a serving loop keeps for all its calls: every call may write any of it, its first bytes start at 0
    s["workspace"] = torch.zeros(_workspace_bytes(case), dtype=torch.uint8, device="cuda")
    return s


def _workspace_bytes(case):
    """Room for any of the calls of a case: products of single rows in 32 bits, and parts of sums."""
    if case["op"] == "moe":
        slots, pad = case["T"] * case["top_k"], case["T"] + 15
        return 4 * slots * (5 * case["N"] + 2 * case["K"]) + 4 * 1024 * 128 * pad + 4 * case["T"] * case["E"] + (1 << 20)
    return 8 * case["M"] * case["R"] * 2 + (1 << 20)


def _silu(g):
    return g / (1 + torch.exp(-g))


def _adapted(s, side):
    """x W^T and the adapters' term: every adapter's, and of each row the one it uses."""
    x, a, b = s["x"].float(), s["a" + side].float(), s["b" + side].float()
    L, R, K = a.shape
    p = (x @ a.view(L * R, K).T).view(-1, L, R) * s["scale"][None, :, None]
    uses = s["adapter"][:, None] == torch.arange(L, device=x.device)[None, :]
    p = torch.where(uses[:, :, None], p, torch.zeros((), device=x.device)).view(-1, L * R)
    return x @ s["w" + side].float().T + p @ b.permute(0, 2, 1).reshape(L * R, -1)


def _route(h, router, top_k, renormalize):
    """(ids, weights): the top_k experts of each row by their logits, ties to the lowest index."""
    # a border between two experts lies anywhere: the logits in 64 bits, rounded once
    logits = (h.double() @ router.double().T).float()
    order, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp(order - order[:, :1])
    w = e[:, :top_k] / (e[:, :top_k] if renormalize else e).sum(1, keepdim=True)
    return ids[:, :top_k], w


def _plain_moe(s):
    case = s["case"]
    ids, w = _route(s["h"], s["router"], case["top_k"], case["renormalize"])
    h = s["h"].float()
    if ids.numel() < case["E"]:   # the chosen experts' weights, for each row
        g = torch.einsum("tk,tjnk->tjn", h, s["gate"][ids].float())
        u = torch.einsum("tk,tjnk->tjn", h, s["up"][ids].float())
        y = torch.einsum("tjn,tjkn->tjk", _silu(g) * u, s["down"][ids].float())
    else:                         # every expert on every row, and of those the chosen ones
        g = torch.einsum("tk,enk->etn", h, s["gate"].float())
        u = torch.einsum("tk,enk->etn", h, s["up"].float())
        y = torch.einsum("etn,ekn->etk", _silu(g) * u, s["down"].float())
        y = y[ids, torch.arange(h.shape[0], device=h.device)[:, None]]
    return dict(out=(y * w[:, :, None]).sum(1).bfloat16(), ids=ids.int(), weights=w)


def _plain(s):
    op = s["case"]["op"]
    if op == "moe":
        return _plain_moe(s)
    if op == "linear_lora":
        return dict(out=_adapted(s, "").bfloat16())
    g, u = _adapted(s, "gate"), _adapted(s, "up")
    if s["case"]["mode"] == "hf":
        return dict(out=_silu(g.bfloat16().float()).bfloat16() * u.bfloat16())
    return dict(out=(_silu(g) * u).bfloat16())


def run(state):
    if not own:
        return _plain(state)
    import memory_bound_glu_gb300 as mb
    s, case = state, state["case"]
    if case["op"] == "moe":
        out, ids, weights = mb.moe_glu(s["h"], s["router"], s["gate"], s["up"], s["down"], case["top_k"],
                                       renormalize=case["renormalize"], workspace=s["workspace"])
        return dict(out=out, ids=ids, weights=weights)
    if case["op"] == "linear_lora":
        return dict(out=mb.linear_lora(s["x"], s["w"], s["a"], s["b"], s["adapter"], s["scale"], workspace=s["workspace"]))
    return dict(out=mb.glu_lora(s["x"], s["wgate"], s["wup"], s["agate"], s["bgate"], s["aup"], s["bup"], s["adapter"],
                                s["scale"], mode=case["mode"], workspace=s["workspace"]))


def work(case):
    K, N = case["K"], case["N"]
    if case["op"] == "moe":
        T, E, k = case["T"], case["E"], case["top_k"]
        used = E * (1 - (1 - k / E) ** T)   # experts that some row chooses, where each row's choice is any k of them
        return dict(bytes=2 * (2 * T * K + E * K + used * 3 * N * K) + 8 * T * k, flops=6 * T * k * N * K + 2 * T * E * K)
    M, R, L = case["M"], case["R"], case["L"]
    sides = 2 if case["op"] == "glu_lora" else 1
    used = L * (1 - (1 - (1 - NO_ADAPTER) / L) ** case["requests"])
    return dict(bytes=2 * (M * K + M * N + sides * N * K + sides * used * R * (K + N)) + 4 * M + 4 * L,
                flops=2 * M * sides * (N * K + (1 - NO_ADAPTER) * R * (K + N)))


def exact(case, seed):
    """The definitions in 64 bits, adapter by adapter and expert by expert."""
    s = _inputs(case, seed)

    def silu(g):
        return g * torch.sigmoid(g)

    if case["op"] == "moe":
        T, k = case["T"], case["top_k"]
        h = s["h"].double()
        logits = torch.einsum("tk,ek->te", h, s["router"].double())
        rounded = logits.float()   # the choice goes by the logits as fp32 holds them
        ids = torch.empty(T, k, dtype=torch.int32, device=h.device)
        left = rounded.clone()
        for j in range(k):
            best = left.max(1, keepdim=True).values
            at = (left == best).int().argmax(1)   # the first of the largest
            ids[:, j] = at.int()
            left[torch.arange(T, device=h.device), at] = -math.inf
        v = rounded.double()
        chosen = torch.gather(v, 1, ids.long())
        w = torch.softmax(chosen, 1) if case["renormalize"] else torch.exp(chosen - torch.logsumexp(v, 1, keepdim=True))
        out = torch.zeros(T, case["K"], dtype=torch.float64, device=h.device)
        for e in range(case["E"]):
            rows, j = torch.nonzero(ids == e, as_tuple=True)
            if rows.numel():
                x = h[rows]
                y = (silu(x @ s["gate"][e].double().T) * (x @ s["up"][e].double().T)) @ s["down"][e].double().T
                out.index_add_(0, rows, y * w[rows, j][:, None])
        return dict(out=out, ids=ids, weights=w)

    x = s["x"].double()

    def adapted(side):
        y = x @ s["w" + side].double().T
        for i in range(case["L"]):
            rows = torch.nonzero(s["adapter"] == i)[:, 0]
            if rows.numel():
                p = s["scale"][i].double() * (x[rows] @ s["a" + side][i].double().T)
                y[rows] += p @ s["b" + side][i].double().T
        return y

    if case["op"] == "linear_lora":
        return dict(out=adapted(""))
    g, u = adapted("gate"), adapted("up")
    if case["mode"] == "hf":   # the mode's roundings of g, u and SiLU(g) are part of its definition
        g, u = g.bfloat16().double(), u.bfloat16().double()
        return dict(out=silu(g).bfloat16().double() * u)
    return dict(out=silu(g) * u)
