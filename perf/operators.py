"""Cases of the gated feed-forward block beyond the decode batch: its bf16 form at any number of tokens with its
backward pass, and its 8-bit form for serving (norm, gated projections, down projection).

    glu      out = SiLU(h Wg^T) * (h Wu^T), bf16, any number of tokens (a prompt, a chunk of one)
    train    the same with the gradients of h, Wg and Wu: one training step of the block
    norm8    residual' = bf16(x + residual); q, scale = e4m3 of the zero-centred RMSNorm of residual', a scale per 128
    glu8     SiLU(a Wg^T) * (a Wu^T) of e4m3 operands with block scales; out bf16, or e4m3 with a scale per 128
    matmul8  a w^T of e4m3 operands: a has a scale per row and 128 columns, w one per 128 x 128 block; out bf16

`own` selects the framework's calls; otherwise `run` is the plain form in 32 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126   # the smallest scale a group gets (a group of zeros has it)
BLOCK = 128
EPS = 1e-6


def listed():
    return [
        # one decoded token: the norm in front of the block, where only latency counts
        dict(name="norm8_token", op="norm8", M=1, K=2560),
        # a prompt's chunk through the same norm: memory-bound
        dict(name="norm8_prompt", op="norm8", M=4096, K=4096),
        # one decoded token through the gate and up projections: both 8-bit weights are read once
        dict(name="glu8_token", op="glu8", M=1, K=2560, N=9728, quant=True),
        # a decode batch of 48 requests
        dict(name="glu8_batch48", op="glu8", M=48, K=2560, N=9728, quant=True),
        # a long prompt: arithmetic-bound
        dict(name="glu8_prompt", op="glu8", M=4096, K=4096, N=11008, quant=True),
        # the down projection of a decode batch of 8
        dict(name="matmul8_batch8", op="matmul8", M=8, K=9728, N=2560),
        # a ragged chunk: few output tiles over a long inner dimension
        dict(name="matmul8_ragged", op="matmul8", M=333, K=9728, N=2560),
        # the down projection of a long prompt
        dict(name="matmul8_prompt", op="matmul8", M=4096, K=11008, N=4096),
        # a short prompt in bf16, with the roundings of the composite
        dict(name="glu_chunk", op="glu", M=333, K=2560, N=9728, mode="hf"),
        # a long prompt in bf16
        dict(name="glu_prompt", op="glu", M=4096, K=4096, N=14336, mode="fused"),
        # a small ragged training step
        dict(name="train_ragged", op="train", M=333, K=1000, N=2504),
        # a training step of 4096 tokens
        dict(name="train_step", op="train", M=4096, K=2560, N=9728),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm8", "glu8", "glu8", "matmul8", "matmul8", "glu", "train"])
    if op == "norm8":
        return dict(op=op, M=log_int(1, 4096), K=16 * log_int(8, 256))
    if op == "glu8":
        return dict(op=op, M=log_int(1, 4096), K=16 * log_int(16, 256), N=log_int(128, 11008), quant=rng.random() < 0.6)
    if op == "matmul8":
        return dict(op=op, M=log_int(1, 4096), K=16 * log_int(16, 688), N=log_int(128, 4096))
    if op == "glu":
        return dict(op=op, M=log_int(65, 4096), K=8 * log_int(32, 512), N=log_int(128, 14336), mode=rng.choice(["hf", "fused"]))
    return dict(op=op, M=log_int(65, 4096), K=8 * log_int(32, 320), N=log_int(128, 9728))


def _blocks(n):
    return -(-n // BLOCK)


def _spread_rows(s, K):
    """[M, blocks] -> [M, K]: each scale over its 128 columns."""
    return s.repeat_interleave(BLOCK, dim=1)[:, :K]


def _spread_blocks(s, N, K):
    return s.repeat_interleave(BLOCK, dim=0)[:N].repeat_interleave(BLOCK, dim=1)[:, :K]


def _row_scales(v):
    """The scale of each 128 columns of a row: amax / 448, at least 2^-126."""
    M, K = v.shape
    pad = _blocks(K) * BLOCK - K
    a = torch.nn.functional.pad(v.abs(), (0, pad)).view(M, _blocks(K), BLOCK).amax(dim=2)
    return (a / E4M3_MAX).clamp_min(SCALE_MIN)


def _quant_rows(v):
    s = _row_scales(v)
    return (v / _spread_rows(s, v.shape[1])).to(torch.float8_e4m3fn), s


def _quant_blocks(w):
    N, K = w.shape
    nb, kb = _blocks(N), _blocks(K)
    a = torch.nn.functional.pad(w.abs(), (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK).amax(dim=(1, 3))
    s = (a / E4M3_MAX).clamp_min(SCALE_MIN)
    return (w / _spread_blocks(s, N, K)).to(torch.float8_e4m3fn), s


def _inputs(case, seed):
    """The inputs, from the seed alone: activations with a few loud channels, weights N(0, 1/K) with loud entries."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    op, M, K = case["op"], case["M"], case["K"]
    loud = torch.ones(K, device=dev)
    loud[torch.randint(K, (max(1, K // 200),), generator=gen, device=dev)] = 12.0
    d = {}
    if op == "norm8":
        d["x"] = (normal(M, K) * loud).bfloat16()
        d["residual"] = (normal(M, K) * 2 * loud).bfloat16()
        d["norm_w"] = (normal(K) * 0.1).bfloat16()
        return d
    N = case["N"]
    if op in ("glu8", "matmul8"):
        d["a"], d["a_scale"] = _quant_rows(normal(M, K) * loud)

        def weight():
            return _quant_blocks((normal(N, K) / math.sqrt(K)).bfloat16().float())

        if op == "glu8":
            d["gate"], d["gate_scale"] = weight()
            d["up"], d["up_scale"] = weight()
        else:
            d["w"], d["w_scale"] = weight()
        return d
    d["h"] = normal(M, K).bfloat16()
    d["gate"] = (normal(N, K) / math.sqrt(K)).bfloat16()
    d["up"] = (normal(N, K) / math.sqrt(K)).bfloat16()
    if op == "train":
        d["dout"] = normal(M, N).bfloat16()
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "norm8":
        d["residual_out"] = torch.empty_like(d["residual"])
    if case["op"] == "train":
        for name in ("h", "gate", "up"):   # the leaves of the step
            d[name].requires_grad_(True)
    return dict(case=dict(case), **d)


def _silu(g):
    return g / (1 + torch.exp(-g))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm8":
        r = (s["x"].float() + s["residual"].float()).bfloat16()
        v = r.float()
        h = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * (1 + s["norm_w"].float())
        q, scale = _quant_rows(h)
        return dict(residual=r, q=q, scale=scale)
    if op in ("glu8", "matmul8"):
        a = s["a"].float() * _spread_rows(s["a_scale"], case["K"])
        if op == "matmul8":
            return dict(out=(a @ (s["w"].float() * _spread_blocks(s["w_scale"], case["N"], case["K"])).T).bfloat16())
        g = a @ (s["gate"].float() * _spread_blocks(s["gate_scale"], case["N"], case["K"])).T
        u = a @ (s["up"].float() * _spread_blocks(s["up_scale"], case["N"], case["K"])).T
        v = _silu(g) * u
        if not case["quant"]:
            return dict(out=v.bfloat16())
        q, scale = _quant_rows(v)
        return dict(q=q, scale=scale)
    with torch.no_grad():
        h, gw, uw = s["h"].float(), s["gate"].float(), s["up"].float()
        g, u = h @ gw.T, h @ uw.T
        if op == "glu":
            if case["mode"] == "hf":
                return dict(out=_silu(g.bfloat16().float()).bfloat16() * u.bfloat16())
            return dict(out=(_silu(g) * u).bfloat16())
        d = s["dout"].float()
        sig = 1 / (1 + torch.exp(-g))
        dg, du = d * u * sig * (1 + g * (1 - sig)), d * g * sig
        return dict(out=(g * sig * u).bfloat16(), grad_h=(dg @ gw + du @ uw).bfloat16(), grad_gate=(dg.T @ h).bfloat16(),
                    grad_up=(du.T @ h).bfloat16())


def run(state):
    if not own:
        return _plain(state)
    import memory_bound_glu_gb300 as mb
    s, case = state, state["case"]
    op = case["op"]
    if op == "norm8":
        q, scale = mb.add_rmsnorm_fp8(s["x"], s["residual"], s["norm_w"], EPS, residual_out=s["residual_out"])
        return dict(residual=s["residual_out"], q=q, scale=scale)
    if op == "glu8":
        if case["quant"]:
            q, scale = mb.glu_fp8(s["a"], s["a_scale"], s["gate"], s["gate_scale"], s["up"], s["up_scale"],
                                  out_dtype=torch.float8_e4m3fn)
            return dict(q=q, scale=scale)
        return dict(out=mb.glu_fp8(s["a"], s["a_scale"], s["gate"], s["gate_scale"], s["up"], s["up_scale"]))
    if op == "matmul8":
        return dict(out=mb.matmul_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"]))
    if op == "glu":
        return dict(out=mb.glu_gemm(s["h"], s["gate"], s["up"], mode=case["mode"]))
    out = mb.DualWeightGlu.apply(s["h"], s["gate"], s["up"])
    gh, gg, gu = torch.autograd.grad(out, (s["h"], s["gate"], s["up"]), s["dout"])
    return dict(out=out, grad_h=gh, grad_gate=gg, grad_up=gu)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    kb = _blocks(K)
    if op == "norm8":   # x and residual in, residual and q out, the scales, the norm's weight
        return dict(bytes=M * K * 7 + M * kb * 4 + K * 2, flops=8 * M * K)
    N = case["N"]
    nb = _blocks(N)
    if op == "glu8":
        out = M * N + M * nb * 4 if case["quant"] else M * N * 2
        return dict(bytes=M * K + M * kb * 4 + 2 * (N * K + nb * kb * 4) + out, flops=4 * M * N * K)
    if op == "matmul8":
        return dict(bytes=M * K + M * kb * 4 + N * K + nb * kb * 4 + M * N * 2, flops=2 * M * N * K)
    if op == "glu":
        return dict(bytes=2 * (M * K + 2 * N * K + M * N), flops=4 * M * N * K)
    # train: out, three gradients; the products g, u, grad_h (two), grad_gate, grad_up
    return dict(bytes=2 * (M * K + 2 * N * K + M * N) + 2 * (M * N + M * K + 2 * N * K), flops=12 * M * N * K)


def exact(case, seed):
    """The definitions in 64 bits. An e4m3 output is the value that is rounded to it, its scale taken out."""
    d = {k: v.double() for k, v in _inputs(case, seed).items()}
    op, M, K = case["op"], case["M"], case["K"]

    def quantised(v):
        s = torch.stack([c.abs().amax(dim=1) for c in v.split(BLOCK, dim=1)], dim=1) / E4M3_MAX
        s = torch.clamp(s, min=SCALE_MIN)
        return torch.cat([c / s[:, i:i + 1] for i, c in enumerate(v.split(BLOCK, dim=1))], dim=1), s

    def widened(w, s):
        out = w.clone()
        for i in range(s.shape[0]):
            for j in range(s.shape[1]):
                out[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= s[i, j]
        return out

    def rows_widened(a, s):
        return torch.cat([c * s[:, i:i + 1] for i, c in enumerate(a.split(BLOCK, dim=1))], dim=1)

    if op == "norm8":
        # the residual's sum is exact in 64 bits; the norm is taken of its bf16 rounding, as the operator defines it
        r = d["x"] + d["residual"]
        v = r.bfloat16().double()
        h = v / torch.sqrt(v.square().sum(dim=1, keepdim=True) / K + EPS) * (1.0 + d["norm_w"])
        q, s = quantised(h)
        return dict(residual=r, q=q, scale=s)
    if op == "matmul8":
        return dict(out=torch.einsum("mk,nk->mn", rows_widened(d["a"], d["a_scale"]), widened(d["w"], d["w_scale"])))
    if op == "glu8":
        a = rows_widened(d["a"], d["a_scale"])
        g = torch.einsum("mk,nk->mn", a, widened(d["gate"], d["gate_scale"]))
        u = torch.einsum("mk,nk->mn", a, widened(d["up"], d["up_scale"]))
        v = g * torch.sigmoid(g) * u
        if not case["quant"]:
            return dict(out=v)
        q, s = quantised(v)
        return dict(q=q, scale=s)
    g = torch.einsum("mk,nk->mn", d["h"], d["gate"])
    u = torch.einsum("mk,nk->mn", d["h"], d["up"])
    if op == "glu":
        if case["mode"] == "hf":   # the mode's roundings of g, u and SiLU(g) are part of its definition
            g, u = g.bfloat16().double(), u.bfloat16().double()
            return dict(out=(g * torch.sigmoid(g)).bfloat16().double() * u)
        return dict(out=g * torch.sigmoid(g) * u)
    sg = torch.sigmoid(g)
    dg = d["dout"] * u * (sg + g * sg * (1.0 - sg))
    du = d["dout"] * g * sg
    return dict(out=g * sg * u, grad_h=torch.einsum("mn,nk->mk", dg, d["gate"]) + torch.einsum("mn,nk->mk", du, d["up"]),
                grad_gate=torch.einsum("mn,mk->nk", dg, d["h"]), grad_up=torch.einsum("mn,mk->nk", du, d["h"]))
