"""ctypes binding of libmbglu.so (C ABI in include/mbglu.h).

Argument marshalling only: tensors become device pointers, row strides and
the current CUDA stream; every step of the computation runs in the library's
kernels.  The wide and the e4m3 calls marshal their common case in an extension
module (csrc/bind_torch.cpp), and here where that is not built.  There is no
fallback for the library: if it is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib
import os
import warnings

import torch

from . import _build

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmbglu.so")

MODE_FUSED = 0
MODE_HF = 1
_MODES = {"fused": MODE_FUSED, "hf": MODE_HF, MODE_FUSED: MODE_FUSED, MODE_HF: MODE_HF}
MAX_M = 64        # batch rows per call (MBGLU_MAX_M)
BLOCK_M = 16      # batch rows per pass over the weights (MBGLU_BLOCK_M)
WORKSPACE_BYTES = 256
MAX_RANK = 128            # of an adapter (MBGLU_LORA_MAX_RANK)
MOE_MAX_EXPERTS = 512     # MBGLU_MOE_MAX_EXPERTS
MOE_MAX_TOP_K = 16        # MBGLU_MOE_MAX_TOP_K
MOE_COUNTER_BYTES = 256   # MBGLU_MOE_COUNTER_BYTES

# Every symbol include/mbglu.h declares.
EXPORTS = ("glu_gemv", "add_rmsnorm_glu", "add_rmsnorm_glu_ws", "add_rmsnorm_glu_strided", "add_rmsnorm_glu_noalloc",
           "silu_mul", "gdn_gates", "glu_backward", "glu_backward_workspace_bytes",
           "glu_gemm", "glu_gemm_backward", "glu_gemm_backward_workspace_bytes", "add_rmsnorm_fp8",
           "quantize_weight_fp8", "glu_fp8", "matmul_fp8", "matmul_fp8_workspace_bytes",
           "glu_lora", "glu_lora_workspace_bytes", "linear_lora", "linear_lora_workspace_bytes",
           "moe_glu", "moe_glu_workspace_bytes",
           "mbglu_set_launch_policy",
           "mbglu_get_launch_policy",
           "mbglu_status_string", "mbglu_abi_version", "mbglu_last_cuda_error", "mbglu_last_variant",
           "mbglu_last_single_kernel_blocks", "mbglu_block_plan", "mbglu_noalloc_scratch_read", "mbglu_read_device_error",
           "mbglu_last_backward_path")
POLICY_SERIAL, POLICY_PDL, POLICY_PREFETCH = 0, 1, 2

_lib = None
_quick_module = None


class MbgluError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().mbglu_status_string(status).decode()
        if status == 7:
            msg += f" (cudaError {lib().mbglu_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


class _Adapters(ctypes.Structure):
    """mbglu_adapters: one projection's A and B with their strides."""
    _fields_ = [("a", ctypes.c_void_p), ("a_adapter", ctypes.c_int64), ("lda", ctypes.c_int64),
                ("b", ctypes.c_void_p), ("b_adapter", ctypes.c_int64), ("ldb", ctypes.c_int64)]


def _bind(l):
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    l.glu_gemv.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32, i32, vp]
    l.glu_gemv.restype = i32
    l.add_rmsnorm_glu.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, vp, i32, i32, i32, i32, vp]
    l.add_rmsnorm_glu.restype = i32
    l.add_rmsnorm_glu_ws.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, vp, i32, i32, i32, i32, vp, ctypes.c_size_t, vp]
    l.add_rmsnorm_glu_ws.restype = i32
    l.add_rmsnorm_glu_noalloc.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, vp, i32, i32, i32, i32, vp]
    l.add_rmsnorm_glu_noalloc.restype = i32
    l.add_rmsnorm_glu_strided.argtypes = [vp, vp, vp, ctypes.c_float, vp, i64, vp, i64, vp, i64, i32, i32, i32, i32,
                                          vp, ctypes.c_size_t, vp]
    l.add_rmsnorm_glu_strided.restype = i32
    l.silu_mul.argtypes = [vp, i64, vp, i64, i32, i32, i32, vp]
    l.gdn_gates.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, i32, i32, vp]
    l.gdn_gates.restype = i32
    l.glu_backward_workspace_bytes.argtypes = [i32, i32, i32]
    l.glu_backward_workspace_bytes.restype = ctypes.c_size_t
    l.glu_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32,
                               vp, ctypes.c_size_t, vp]
    l.glu_backward.restype = i32
    l.silu_mul.restype = i32
    sz = ctypes.c_size_t
    l.glu_gemm.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32, i32, vp]
    l.glu_gemm.restype = i32
    l.glu_gemm_backward_workspace_bytes.argtypes = [i32, i32, i32]
    l.glu_gemm_backward_workspace_bytes.restype = sz
    l.glu_gemm_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32,
                                    i32, vp, sz, vp]
    l.glu_gemm_backward.restype = i32
    l.add_rmsnorm_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, ctypes.c_float, vp, i64, vp, i64, i32, i32, vp]
    l.add_rmsnorm_fp8.restype = i32
    l.quantize_weight_fp8.argtypes = [vp, i64, vp, i64, vp, i64, i32, i32, vp]
    l.quantize_weight_fp8.restype = i32
    l.glu_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32, vp]
    l.glu_fp8.restype = i32
    l.matmul_fp8_workspace_bytes.argtypes = [i32, i32, i32]
    l.matmul_fp8_workspace_bytes.restype = sz
    l.matmul_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, sz, vp]
    l.matmul_fp8.restype = i32
    ad = ctypes.POINTER(_Adapters)
    l.glu_lora.argtypes = [vp, i64, vp, i64, vp, i64, ad, ad, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, sz, vp]
    l.glu_lora.restype = i32
    l.linear_lora.argtypes = [vp, i64, vp, i64, ad, vp, vp, vp, i64, i32, i32, i32, i32, i32, vp, sz, vp]
    l.linear_lora.restype = i32
    l.moe_glu.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64, vp, vp, i32, i32, i32, i32, i32, i32,
                          vp, sz, vp]
    l.moe_glu.restype = i32
    for f in (l.glu_lora_workspace_bytes, l.linear_lora_workspace_bytes, l.moe_glu_workspace_bytes):
        f.argtypes = [i32, i32, i32, i32, i32]
        f.restype = sz
    l.mbglu_status_string.argtypes = [i32]
    l.mbglu_status_string.restype = ctypes.c_char_p
    l.mbglu_abi_version.restype = i32
    l.mbglu_last_cuda_error.restype = i32
    l.mbglu_last_variant.restype = i32
    l.mbglu_last_single_kernel_blocks.restype = i32
    l.mbglu_last_backward_path.restype = i32
    l.mbglu_block_plan.argtypes = [i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int)]
    l.mbglu_block_plan.restype = i32
    l.mbglu_noalloc_scratch_read.argtypes = [ctypes.POINTER(ctypes.c_int), i32]
    l.mbglu_noalloc_scratch_read.restype = i32
    l.mbglu_read_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
    l.mbglu_read_device_error.restype = i32
    l.mbglu_set_launch_policy.argtypes = [i32]
    l.mbglu_set_launch_policy.restype = i32
    l.mbglu_get_launch_policy.restype = i32
    return l


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


class _NoModule:
    """Stands in for the extension module where there is none: no call is its
    common case, so binding.py does them all."""

    def __getattr__(self, name):
        return lambda *args: None


def _quick():
    """The extension module that does the common case of the wide and the e4m3
    calls without Python's checks (csrc/bind_torch.cpp); None from one of its
    functions means that the call is not that case and comes here.  One that was
    built against another torch is not loaded."""
    global _quick_module
    if _quick_module is None:
        l = lib()
        if not _build.quick_is_current():
            warnings.warn(f"{_build.QUICK} is missing or was built against another torch: calls take 10 to 15 us more of host "
                          "time (build it with `python -c 'import __graft_entry__ as g; g.build()'`)")
            _quick_module = _NoModule()
            return _quick_module
        m = importlib.import_module("._mbglu_torch", __package__)
        m.bind(*(ctypes.cast(getattr(l, n), ctypes.c_void_p).value
                 for n in ("glu_gemm", "glu_gemm_backward", "glu_gemm_backward_workspace_bytes", "add_rmsnorm_fp8", "glu_fp8",
                           "matmul_fp8", "matmul_fp8_workspace_bytes", "glu_lora", "glu_lora_workspace_bytes", "linear_lora",
                           "linear_lora_workspace_bytes", "moe_glu")))
        _quick_module = m
    return _quick_module


def _on(dev):
    """The device context for a call on `dev`: none when it is already the
    current device (the common case; entering torch.cuda.device costs a few
    microseconds per call), else torch.cuda.device(dev)."""
    idx = dev.index
    if idx is None or idx == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _stream_handle(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check(t, name, dim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got shape {tuple(t.shape)}")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def glu_gemv(h, gate_w, up_w, out=None, mode="fused", stream=None):
    """out[M,N] = SiLU(h @ gate_w.T) * (h @ up_w.T) in one pass (bf16).

    h is [M,K] (or [K]); gate_w, up_w are [N,K] nn.Linear weights read in
    place; mode "fused" (one rounding) or "hf" (HF bf16 boundaries).  Row
    strides are passed through, so sliced views work without copies.
    """
    squeeze = h.dim() == 1
    h2 = h.unsqueeze(0) if squeeze else h
    _check(h2, "h", 2)
    _check(gate_w, "gate_w", 2)
    _check(up_w, "up_w", 2)
    M, K = h2.shape
    N = gate_w.shape[0]
    if tuple(gate_w.shape) != (N, K) or tuple(up_w.shape) != (N, K):
        raise ValueError(f"weights must be [N,K]=[{N},{K}], got {tuple(gate_w.shape)}, {tuple(up_w.shape)}")
    dev = h2.device
    if gate_w.device != dev or up_w.device != dev:
        raise ValueError("all tensors must be on one device")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    out2 = out.unsqueeze(0) if out.dim() == 1 else out
    _check(out2, "out", 2)
    if tuple(out2.shape) != (M, N) or out2.device != dev:
        raise ValueError(f"out must be [{M},{N}] on {dev}")
    with _on(dev):
        st = lib().glu_gemv(h2.data_ptr(), h2.stride(0), gate_w.data_ptr(), gate_w.stride(0),
                            up_w.data_ptr(), up_w.stride(0), out2.data_ptr(), out2.stride(0),
                            M, N, K, _MODES[mode], _stream_handle(dev, stream))
    if st != 0:
        raise MbgluError(st, "glu_gemv")
    return out2.view(N) if squeeze else out


def column_shard(N: int, world: int, rank: int):
    """Rows [lo, hi) of gate_w and up_w -- and columns of out -- that rank
    `rank` of `world` owns when the GLU GEMV is split column-parallel over N
    (DeepSpeed PR #8602, "Architecture Notes": the gate/up projections are
    column-parallel under AutoTP and the segment needs no communication; the
    all-reduce belongs to the row-parallel down projection after it).  The
    shares are balanced (sizes differ by at most one row), disjoint, in rank
    order, and cover [0, N).  Each rank then calls glu_gemv (or
    add_rmsnorm_glu, whose prologue every rank repeats) on its rows of both
    weights and writes out[:, lo:hi]; no collective is involved."""
    if world < 1 or not 0 <= rank < world or N < 0:
        raise ValueError(f"bad split: N={N}, world={world}, rank={rank}")
    return (N * rank) // world, (N * (rank + 1)) // world


def glu_backward(h, gate_w, up_w, dout, grad_h=None, grad_gate=None, grad_up=None, want_h=True, want_w=True,
                 workspace=None, stream=None):
    """Gradients of glu_gemv's SiLU(h @ gate_w.T) * (h @ up_w.T) for an
    upstream dout [M,N] (bf16): returns (grad_h [M,K], grad_gate [N,K],
    grad_up [N,K]), bf16, each None where not wanted.  Output tensors may be
    passed in (any row stride, contiguous last dimension); the workspace is a
    byte tensor of glu_backward_workspace_bytes(M, N, K), allocated here by
    torch's allocator when not given."""
    _check(h, "h", 2)
    _check(gate_w, "gate_w", 2)
    _check(up_w, "up_w", 2)
    _check(dout, "dout", 2)
    M, K = h.shape
    N = gate_w.shape[0]
    if tuple(gate_w.shape) != (N, K) or tuple(up_w.shape) != (N, K) or tuple(dout.shape) != (M, N):
        raise ValueError(f"expected gate_w, up_w [{N},{K}] and dout [{M},{N}]")
    dev = h.device
    if want_h and grad_h is None:
        grad_h = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    if want_w and grad_gate is None:
        grad_gate = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
    if want_w and grad_up is None:
        grad_up = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
    if not want_h:
        grad_h = None
    if not want_w:
        grad_gate = grad_up = None
    for t, name, shape in ((grad_h, "grad_h", (M, K)), (grad_gate, "grad_gate", (N, K)), (grad_up, "grad_up", (N, K))):
        if t is not None:
            _check(t, name, 2)
            if tuple(t.shape) != shape or t.device != dev:
                raise ValueError(f"{name} must be {list(shape)} on {dev}")
    need = lib().glu_backward_workspace_bytes(M, N, K)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wsp = workspace.data_ptr() if workspace is not None else None
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0

    def ptr(t):
        return (t.data_ptr(), t.stride(0)) if t is not None else (None, 0)

    with _on(dev):
        st = lib().glu_backward(h.data_ptr(), h.stride(0), gate_w.data_ptr(), gate_w.stride(0), up_w.data_ptr(),
                                up_w.stride(0), dout.data_ptr(), dout.stride(0), *ptr(grad_h), *ptr(grad_gate),
                                *ptr(grad_up), M, N, K, wsp, wsb, _stream_handle(dev, stream))
    if st != 0:
        raise MbgluError(st, "glu_backward")
    return grad_h, grad_gate, grad_up


class _GluNode(torch.autograd.Function):
    """The autograd node of DualWeightGlu.  keep: whether a backward can follow,
    which forward cannot see (grad mode is off inside it)."""

    @staticmethod
    def forward(ctx, h, gate_w, up_w, mode="fused", keep=True):
        if h.dim() == 2 and h.shape[0] > MAX_M:
            gu = torch.empty((h.shape[0], 2 * gate_w.shape[0]), dtype=torch.float32, device=h.device) if keep else None
            out = glu_gemm(h, gate_w, up_w, mode=mode, gu=gu)
            if keep:
                ctx.save_for_backward(h, gate_w, up_w, gu)
            return out
        if keep:
            ctx.save_for_backward(h, gate_w, up_w)
        return glu_gemv(h, gate_w, up_w, mode=mode)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        h, gate_w, up_w, *rest = ctx.saved_tensors
        squeeze = h.dim() == 1
        h2 = h.unsqueeze(0) if squeeze else h
        d2 = dout.reshape(h2.shape[0], -1).to(torch.bfloat16)
        # a broadcast gradient (of a sum) has stride 0; a single column or row may have any,
        # and counts as contiguous all the same: a copy has the strides of its shape
        if d2.stride(-1) != 1 or d2.stride(0) < d2.shape[1]:
            d2 = d2.clone(memory_format=torch.contiguous_format)
        want = dict(want_h=ctx.needs_input_grad[0], want_w=ctx.needs_input_grad[1] or ctx.needs_input_grad[2])
        if rest:
            gh, gg, gu = glu_gemm_backward(h2, gate_w, up_w, d2, gu=rest[0], **want)
        else:
            gh, gg, gu = glu_backward(h2, gate_w, up_w, d2, **want)
        if gh is not None and squeeze:
            gh = gh.view(-1)
        return gh, gg if ctx.needs_input_grad[1] else None, gu if ctx.needs_input_grad[2] else None, None, None


class DualWeightGlu(_GluNode):
    """out = SiLU(h @ gate_w.T) * (h @ up_w.T) with the weights read in place
    and gradients for h, gate_w and up_w ([8602/PlanB] "Plan B Design": the
    Function works on the model's own weight tensors, not on a copy, so their
    gradients land on those tensors).

    Up to MAX_M rows run glu_gemv and glu_backward; more run glu_gemm, which
    keeps g and u in fp32 (8 M N bytes) for glu_gemm_backward, whose gradients carry
    one bf16 rounding more (of the products' gradients dG and dU).  There is no second
    derivative and no forward-mode one: asking for either raises.  Where no
    gradient can follow, nothing is kept.  To capture a training step into a
    CUDA graph, run it on the capture's stream first and let no eager graph over
    the same leaves live meanwhile, as for any autograd Function."""

    @classmethod
    def apply(cls, h, gate_w, up_w, mode="fused"):
        tracing = torch.jit.is_tracing()   # what a trace runs on later may have gradients
        keep = tracing or torch.is_grad_enabled() and (h.requires_grad or gate_w.requires_grad or up_w.requires_grad)
        # the same node without Python, in its common case; a tracer does not see it and
        # torch's compiler does not know it
        if keep and not (tracing or torch.compiler.is_compiling()) and h.dim() == 2 and h.shape[0] > MAX_M:
            out = (_quick_module or _quick()).wide_glu(h, gate_w, up_w, _MODES[mode])
            if out is not None:
                return out
        return _GluNode.apply(h, gate_w, up_w, mode, keep)


def new_workspace(device=None):
    """A zeroed workspace for add_rmsnorm_glu (one per concurrently running stream)."""
    return torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=device or "cuda")


def add_rmsnorm_glu(x, residual, norm_w, eps, gate_w, up_w, out=None, mode="hf", stream=None, workspace=None):
    """residual <- bf16(x + residual); h = zero-centred RMSNorm(residual);
    out = GLU(h).  Returns out; residual is updated in place.  With a
    workspace (new_workspace()) the whole segment runs as one kernel.  x,
    residual and norm_w are contiguous; the weights and out may be row-strided
    views (contiguous last dimension)."""
    _check(x, "x", 2)
    _check(residual, "residual", 2)
    _check(norm_w, "norm_w", 1)
    _check(gate_w, "gate_w", 2)
    _check(up_w, "up_w", 2)
    M, K = x.shape
    N = gate_w.shape[0]
    for t, name in ((x, "x"), (residual, "residual"), (norm_w, "norm_w")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if tuple(residual.shape) != (M, K) or tuple(norm_w.shape) != (K,):
        raise ValueError("residual must be [M,K] and norm_w [K]")
    if tuple(gate_w.shape) != (N, K) or tuple(up_w.shape) != (N, K):
        raise ValueError("weights must be [N,K]")
    dev = x.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _check(out, "out", 2)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be a [{M},{N}] tensor")
    if workspace is not None and not (workspace.is_cuda and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on the operands' device")
    with _on(dev):
        if not (gate_w.is_contiguous() and up_w.is_contiguous() and out.is_contiguous()):
            wsp = workspace.data_ptr() if workspace is not None else None
            wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
            st = lib().add_rmsnorm_glu_strided(x.data_ptr(), residual.data_ptr(), norm_w.data_ptr(), float(eps),
                                               gate_w.data_ptr(), gate_w.stride(0), up_w.data_ptr(), up_w.stride(0),
                                               out.data_ptr(), out.stride(0), M, N, K, _MODES[mode], wsp, wsb,
                                               _stream_handle(dev, stream))
        elif workspace is None:
            st = lib().add_rmsnorm_glu(x.data_ptr(), residual.data_ptr(), norm_w.data_ptr(), float(eps),
                                       gate_w.data_ptr(), up_w.data_ptr(), out.data_ptr(), M, N, K, _MODES[mode],
                                       _stream_handle(dev, stream))
        else:
            st = lib().add_rmsnorm_glu_ws(x.data_ptr(), residual.data_ptr(), norm_w.data_ptr(), float(eps),
                                          gate_w.data_ptr(), up_w.data_ptr(), out.data_ptr(), M, N, K, _MODES[mode],
                                          workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                          _stream_handle(dev, stream))
    if st != 0:
        raise MbgluError(st, "add_rmsnorm_glu")
    return out


def _check_operand(t, name, dtype, shape, dev):
    """One operand of the wide and the e4m3 calls: dtype, device, shape and a
    contiguous last dimension; any row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a CUDA tensor on {dev}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _arg(t, name, dtype, rows, cols, dev):
    """(pointer, row stride) of a checked [rows, cols] operand.  A tensor of one
    row may carry any stride (a view's says nothing), so it gets its row's
    length.  The common case is decided in a few attribute reads: a decode step's
    kernels take microseconds, and so would the checks."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == (rows, cols):
        s0, s1 = t.stride()
        if s1 == 1:
            return t.data_ptr(), s0 if rows > 1 else cols
    _check_operand(t, name, dtype, (rows, cols), dev)
    return t.data_ptr(), t.stride(0) if rows > 1 else max(cols, 1)


def _dims(t, name, dtype):
    """(rows, cols, device) of a call's first operand, a 2-D CUDA tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if max(t.shape) > _MOST:
        raise ValueError(f"{name} has more than {_MOST} rows or columns: {tuple(t.shape)}")
    return (*t.shape, t.device)


def _out_rows(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if t.shape[0] > _MOST:
        raise ValueError(f"{name} has more than {_MOST} rows: {tuple(t.shape)}")
    return t.shape[0]


def _workspace(workspace, need, dev):
    """(pointer, bytes, tensor) of a workspace of `need` bytes, allocated here by
    torch's allocator on the current stream when not given."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace.data_ptr(), need, workspace
    if not (workspace.is_cuda and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


_here = contextlib.nullcontext()
_one_device = None   # whether the process sees one GPU, which then is the current one
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _allocate_on(dev, stream):
    """The context of a call's allocations and launch: they belong to the stream
    that the call runs on, whose order torch's allocator then hands their memory
    out again in."""
    global _one_device
    if stream is not None:
        return torch.cuda.stream(stream)
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    return _here if _one_device else _on(dev)


def _stream_of(dev, stream):
    """The handle of the stream that a call runs on."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev.index) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


_NONE = (None, 0)
_MOST = 2 ** 31 - 512   # what the C entry points take


def glu_gemm(h, gate_w, up_w, out=None, mode="fused", gu=None, stream=None):
    """out[M,N] = SiLU(h @ gate_w.T) * (h @ up_w.T) for any number of rows: a
    prompt or a training batch.  Arguments as glu_gemv; gu, a float32 [M, 2N]
    tensor, receives g and u for glu_gemm_backward.  Without gu, up to 16 rows
    (up to MAX_M of operands that are not 16-byte aligned) the call is glu_gemv."""
    if stream is None:
        r = (_quick_module or _quick()).glu_gemm(h, gate_w, up_w, out, _MODES[mode], gu)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "glu_gemm")
            return r
    bf16 = torch.bfloat16
    squeeze = isinstance(h, torch.Tensor) and h.dim() == 1
    h2 = h.unsqueeze(0) if squeeze else h
    M, K, dev = _dims(h2, "h", bf16)
    N = _out_rows(gate_w, "gate_w")
    ins = (*_arg(h2, "h", bf16, M, K, dev), *_arg(gate_w, "gate_w", bf16, N, K, dev), *_arg(up_w, "up_w", bf16, N, K, dev))
    with _allocate_on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=bf16, device=dev)
        out2 = out.unsqueeze(0) if out.dim() == 1 else out
        st = lib().glu_gemm(*ins, *_arg(out2, "out", bf16, M, N, dev),
                            *(_NONE if gu is None else _arg(gu, "gu", torch.float32, M, 2 * N, dev)), M, N, K, _MODES[mode],
                            _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "glu_gemm")
    return out2.view(N) if squeeze else out


def glu_gemm_backward(h, gate_w, up_w, dout, gu=None, grad_h=None, grad_gate=None, grad_up=None, want_h=True,
                      want_w=True, workspace=None, stream=None):
    """Gradients of glu_gemm for an upstream dout [M,N]: (grad_h, grad_gate,
    grad_up), each None where not wanted, as glu_backward but for any number of
    rows.  gu: what glu_gemm wrote there (computed again when not given).  The
    workspace is a byte tensor of glu_gemm_backward_workspace_bytes(M, N, K)
    bytes, 256-byte aligned, allocated here when not given."""
    if stream is None and grad_h is None and grad_gate is None and grad_up is None and workspace is None:
        r = (_quick_module or _quick()).glu_gemm_backward(h, gate_w, up_w, dout, gu, bool(want_h), bool(want_w))
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "glu_gemm_backward")
            return r
    bf16 = torch.bfloat16
    M, K, dev = _dims(h, "h", bf16)
    N = _out_rows(gate_w, "gate_w")
    ins = (*_arg(h, "h", bf16, M, K, dev), *_arg(gate_w, "gate_w", bf16, N, K, dev), *_arg(up_w, "up_w", bf16, N, K, dev),
           *_arg(dout, "dout", bf16, M, N, dev), *(_NONE if gu is None else _arg(gu, "gu", torch.float32, M, 2 * N, dev)))
    with _allocate_on(dev, stream):
        if not want_h:
            grad_h = None
        elif grad_h is None:
            grad_h = torch.empty((M, K), dtype=bf16, device=dev)
        if not want_w:
            grad_gate = grad_up = None
        else:
            if grad_gate is None:
                grad_gate = torch.empty((N, K), dtype=bf16, device=dev)
            if grad_up is None:
                grad_up = torch.empty((N, K), dtype=bf16, device=dev)
        outs = (*(_arg(grad_h, "grad_h", bf16, M, K, dev) if want_h else _NONE),
                *(_arg(grad_gate, "grad_gate", bf16, N, K, dev) if want_w else _NONE),
                *(_arg(grad_up, "grad_up", bf16, N, K, dev) if want_w else _NONE))
        wsp, wsb, keep = _workspace(workspace, lib().glu_gemm_backward_workspace_bytes(M, N, K), dev)
        st = lib().glu_gemm_backward(*ins, *outs, M, N, K, wsp, wsb, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "glu_gemm_backward")
    return grad_h, grad_gate, grad_up


E4M3 = torch.float8_e4m3fn
SCALE_BLOCK = 128   # columns (and rows, of a weight) per e4m3 scale


def _blocks(n):
    return -(-n // SCALE_BLOCK)


def _empty_e4m3(M, N, dev):
    """[M, N] e4m3 whose rows start on 16 bytes, as the products' tensor copies
    want their operands."""
    if N % 16 == 0:
        return torch.empty((M, N), dtype=E4M3, device=dev)
    return torch.empty((M, -(-N // 16) * 16), dtype=E4M3, device=dev)[:, :N]


def _scaled(t, scale, name, rows, cols, scale_rows, dev):
    """(pointer, row stride) of an e4m3 operand, then of its scales."""
    return (*_arg(t, name, E4M3, rows, cols, dev), *_arg(scale, name + "'s scale", torch.float32, scale_rows, _blocks(cols), dev))


def add_rmsnorm_fp8(x, residual, norm_w, eps, q=None, scale=None, residual_out=None, stream=None):
    """residual_out <- bf16(x + residual) (in place when not given); v = its
    zero-centred RMSNorm; returns (q, scale): v as e4m3 [M,K] with a float32
    scale per row and 128 columns [M, ceil(K/128)]."""
    if stream is None:
        r = (_quick_module or _quick()).add_rmsnorm_fp8(x, residual, norm_w, eps, q, scale, residual_out)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "add_rmsnorm_fp8")
            return r
    bf16 = torch.bfloat16
    M, K, dev = _dims(x, "x", bf16)
    if norm_w is None or norm_w.dim() != 1 or norm_w.shape[0] != K or norm_w.dtype is not bf16 or norm_w.device != dev \
            or not norm_w.is_contiguous():
        raise ValueError(f"norm_w must be a contiguous bfloat16 tensor of {K} elements on {dev}")
    ins = (*_arg(x, "x", bf16, M, K, dev), *_arg(residual, "residual", bf16, M, K, dev),
           *_arg(residual if residual_out is None else residual_out, "residual_out", bf16, M, K, dev), norm_w.data_ptr(), eps)
    with _allocate_on(dev, stream):
        if q is None:
            q = _empty_e4m3(M, K, dev)
        if scale is None:
            scale = torch.empty((M, _blocks(K)), dtype=torch.float32, device=dev)
        st = lib().add_rmsnorm_fp8(*ins, *_scaled(q, scale, "q", M, K, M, dev), M, K, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "add_rmsnorm_fp8")
    return q, scale


def quantize_weight_fp8(w, q=None, scale=None, stream=None):
    """A bf16 weight [N,K] as e4m3 with a float32 scale per 128 x 128 block:
    returns (q, scale), scale [ceil(N/128), ceil(K/128)]."""
    N, K, dev = _dims(w, "w", torch.bfloat16)
    ins = _arg(w, "w", torch.bfloat16, N, K, dev)
    with _allocate_on(dev, stream):
        if q is None:
            q = _empty_e4m3(N, K, dev)
        if scale is None:
            scale = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=dev)
        st = lib().quantize_weight_fp8(*ins, *_scaled(q, scale, "q", N, K, _blocks(N), dev), N, K, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "quantize_weight_fp8")
    return q, scale


def glu_fp8(a, a_scale, gate_w, gate_scale, up_w, up_scale, out=None, out_scale=None, out_dtype=torch.bfloat16,
            stream=None):
    """SiLU(a @ gate_w.T) * (a @ up_w.T) of e4m3 operands: a [M,K] with a scale
    per row and 128 columns (add_rmsnorm_fp8's), weights [N,K] with one per
    128 x 128 block (quantize_weight_fp8's).  out_dtype bfloat16 returns out;
    float8_e4m3fn returns (q, scale), the operand of matmul_fp8."""
    if out_dtype is not torch.bfloat16 and out_dtype is not E4M3:
        raise TypeError(f"out_dtype must be bfloat16 or float8_e4m3fn, got {out_dtype}")
    if stream is None:
        r = (_quick_module or _quick()).glu_fp8(a, a_scale, gate_w, gate_scale, up_w, up_scale, out, out_scale, out_dtype is E4M3)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "glu_fp8")
            return r
    M, K, dev = _dims(a, "a", E4M3)
    N = _out_rows(gate_w, "gate_w")
    nb = _blocks(N)
    ins = (*_scaled(a, a_scale, "a", M, K, M, dev), *_scaled(gate_w, gate_scale, "gate_w", N, K, nb, dev),
           *_scaled(up_w, up_scale, "up_w", N, K, nb, dev))
    quant = out_dtype is E4M3
    with _allocate_on(dev, stream):
        if quant:
            if out is None:
                out = _empty_e4m3(M, N, dev)
            if out_scale is None:
                out_scale = torch.empty((M, nb), dtype=torch.float32, device=dev)
            outs = (None, 0, *_scaled(out, out_scale, "out", M, N, M, dev))
        else:
            if out_scale is not None:
                raise ValueError("out_scale belongs to a float8_e4m3fn output")
            if out is None:
                out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
            outs = (*_arg(out, "out", torch.bfloat16, M, N, dev), None, 0, None, 0)
        st = lib().glu_fp8(*ins, *outs, M, N, K, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "glu_fp8")
    return (out, out_scale) if quant else out


def matmul_fp8(a, a_scale, w, w_scale, out=None, workspace=None, stream=None):
    """out[M,N] = a @ w.T (bf16) of e4m3 operands with the scales of glu_fp8.
    The workspace is a byte tensor of matmul_fp8_workspace_bytes(M, N, K)
    bytes, 256-byte aligned, allocated here when not given."""
    if stream is None and workspace is None:
        r = (_quick_module or _quick()).matmul_fp8(a, a_scale, w, w_scale, out)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "matmul_fp8")
            return r
    M, K, dev = _dims(a, "a", E4M3)
    N = _out_rows(w, "w")
    ins = (*_scaled(a, a_scale, "a", M, K, M, dev), *_scaled(w, w_scale, "w", N, K, _blocks(N), dev))
    with _allocate_on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        wsp, wsb, keep = _workspace(workspace, lib().matmul_fp8_workspace_bytes(M, N, K), dev)
        st = lib().matmul_fp8(*ins, *_arg(out, "out", torch.bfloat16, M, N, dev), M, N, K, wsp, wsb, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "matmul_fp8")
    return out


def glu_gemm_backward_workspace_bytes(M, N, K):
    """Bytes of glu_gemm_backward's workspace."""
    return lib().glu_gemm_backward_workspace_bytes(M, N, K)


def matmul_fp8_workspace_bytes(M, N, K):
    """Bytes of matmul_fp8's workspace (0: none needed)."""
    return lib().matmul_fp8_workspace_bytes(M, N, K)


def _arg3(t, name, shape, dev):
    """(pointer, outer stride, row stride) of a bf16 operand of three dimensions."""
    _check_operand(t, name, torch.bfloat16, shape, dev)
    count, rows, cols = shape
    row = t.stride(1) if rows > 1 else max(cols, 1)
    return t.data_ptr(), t.stride(0) if count > 1 else rows * row, row


def _vector(t, name, dtype, n, dev):
    """The pointer of a contiguous vector."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or t.shape != (n,) or n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {dev}")
    return t.data_ptr()


def _adapter_args(a, b, name, N, K, count, R, dev):
    """One projection's adapters, A [count, R, K] and B [count, N, R]."""
    return _Adapters(*_arg3(a, name + "_a", (count, R, K), dev), *_arg3(b, name + "_b", (count, N, R), dev))


def _ranks(a, name):
    """(adapters, R) of A [adapters, R, K]."""
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError(f"{name} must be a 3-D tensor [adapters, rank, K]")
    if a.shape[1] > MAX_RANK:
        raise ValueError(f"{name}'s rank {a.shape[1]} is above {MAX_RANK}")
    return a.shape[0], a.shape[1]


def glu_lora(h, gate_w, up_w, gate_a, gate_b, up_a, up_b, adapter, scale=None, out=None, mode="fused", workspace=None,
             stream=None):
    """SiLU(g) * u, [M,N], of the gated projections with low-rank adapters beside the
    shared weights: g = h @ gate_w.T + p @ gate_b[a].T with p = scale[a] * (h @
    gate_a[a].T) and a = adapter[m] the row's adapter; u likewise.  Any number of
    rows.  gate_a, up_a are [adapters,R,K], gate_b, up_b [adapters,N,R] (bf16, R <=
    MAX_RANK); adapter is int32 [M], a value outside [0, adapters) meaning none;
    scale float32 [adapters] or None for 1.  The workspace is a byte tensor, 256-byte
    aligned, of glu_lora_workspace_bytes(M, N, K, adapters, R) bytes (one for the most
    rows serves fewer) or of less, down to 16 R M + M / 8 + 2048, which may take longer;
    allocated here when not given.  No gradients."""
    if stream is None:
        r = (_quick_module or _quick()).glu_lora(h, gate_w, up_w, gate_a, gate_b, up_a, up_b, adapter, scale, out, _MODES[mode], workspace)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "glu_lora")
            return r
    bf16 = torch.bfloat16
    M, K, dev = _dims(h, "h", bf16)
    N = _out_rows(gate_w, "gate_w")
    count, R = _ranks(gate_a, "gate_a")
    ins = (*_arg(h, "h", bf16, M, K, dev), *_arg(gate_w, "gate_w", bf16, N, K, dev), *_arg(up_w, "up_w", bf16, N, K, dev),
           _adapter_args(gate_a, gate_b, "gate", N, K, count, R, dev), _adapter_args(up_a, up_b, "up", N, K, count, R, dev),
           _vector(adapter, "adapter", torch.int32, M, dev), None if scale is None else _vector(scale, "scale", torch.float32, count, dev))
    with _allocate_on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=bf16, device=dev)
        wsp, wsb, keep = _workspace(workspace, lib().glu_lora_workspace_bytes(M, N, K, count, R), dev)
        st = lib().glu_lora(*ins, *_arg(out, "out", bf16, M, N, dev), M, N, K, count, R, _MODES[mode], wsp, wsb, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "glu_lora")
    return out


def linear_lora(x, w, a, b, adapter, scale=None, out=None, workspace=None, stream=None):
    """x @ w.T + (scale[i] * (x @ a[i].T)) @ b[i].T, [M,N] bf16, with i = adapter[m]
    the row's adapter: one projection of glu_lora, such as the down projection.
    Arguments as there, a [adapters,R,K] and b [adapters,N,R]; the workspace is one of
    linear_lora_workspace_bytes(M, N, K, adapters, R) bytes, or of at least 8 R M + M / 8 +
    2048.  No gradients."""
    if stream is None:
        r = (_quick_module or _quick()).linear_lora(x, w, a, b, adapter, scale, out, workspace)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "linear_lora")
            return r
    bf16 = torch.bfloat16
    M, K, dev = _dims(x, "x", bf16)
    N = _out_rows(w, "w")
    count, R = _ranks(a, "a")
    ins = (*_arg(x, "x", bf16, M, K, dev), *_arg(w, "w", bf16, N, K, dev),
           _Adapters(*_arg3(a, "a", (count, R, K), dev), *_arg3(b, "b", (count, N, R), dev)),
           _vector(adapter, "adapter", torch.int32, M, dev), None if scale is None else _vector(scale, "scale", torch.float32, count, dev))
    with _allocate_on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=bf16, device=dev)
        wsp, wsb, keep = _workspace(workspace, lib().linear_lora_workspace_bytes(M, N, K, count, R), dev)
        st = lib().linear_lora(*ins, *_arg(out, "out", bf16, M, N, dev), M, N, K, count, R, wsp, wsb, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "linear_lora")
    return out


def new_moe_workspace(T, E, top_k, N, K, device=None):
    """A workspace for moe_glu calls of up to T tokens at these sizes (one per
    concurrently running stream), its counters zeroed.  After an error that
    read_device_error reports, its first MOE_COUNTER_BYTES have to be zeroed again."""
    need = moe_glu_workspace_bytes(T, E, top_k, N, K)
    ws = torch.empty(max(need, MOE_COUNTER_BYTES), dtype=torch.uint8, device=device or "cuda")
    ws[:MOE_COUNTER_BYTES].zero_()
    return ws


def moe_glu(h, router_w, gate_w, up_w, down_w, top_k, renormalize=True, out=None, ids=None, weights=None, workspace=None,
            stream=None):
    """A mixture-of-experts layer of up to MAX_M tokens: returns (out [T,K] bf16, ids
    [T,top_k] int32, weights [T,top_k] float32).  The logits h @ router_w.T are rounded
    once to float32, from sums that are off by (K / 32 + 32)^2 2^-48 of their products'
    magnitudes at most; each token takes the top_k experts (ties to the lowest index) with
    softmax weights, renormalised over the chosen or not; out is the weighted sum of
    (SiLU(h @ gate_w[e].T) * (h @ up_w[e].T)) @ down_w[e].T.  router_w is [E,K], gate_w
    and up_w [E,N,K], down_w [E,K,N].
    The workspace (new_moe_workspace(T, E, top_k, N, K), which a decode loop keeps)
    is allocated and its counters are zeroed here when not given; after a call that sets
    the device error word (read_device_error) one that is kept has to be zeroed again
    before calls on it succeed.  No gradients."""
    if stream is None:
        r = (_quick_module or _quick()).moe_glu(h, router_w, gate_w, up_w, down_w, top_k, bool(renormalize), out, ids, weights, workspace)
        if r is not None:
            if type(r) is int:
                raise MbgluError(r, "moe_glu")
            return r
    bf16 = torch.bfloat16
    T, K, dev = _dims(h, "h", bf16)
    if T > MAX_M:
        raise ValueError(f"h has more than {MAX_M} tokens: {T}")
    E = _out_rows(router_w, "router_w")
    if not isinstance(gate_w, torch.Tensor) or gate_w.dim() != 3 or gate_w.shape[1] > _MOST:
        raise ValueError("gate_w must be a 3-D tensor [experts, N, K]")
    N = gate_w.shape[1]
    top_k = int(top_k)
    if not 1 <= E <= MOE_MAX_EXPERTS or not 1 <= top_k <= min(E, MOE_MAX_TOP_K):
        raise ValueError(f"1 to {MOE_MAX_EXPERTS} experts and 1 to {MOE_MAX_TOP_K} of them per token, got {E} and {top_k}")
    ins = (*_arg(h, "h", bf16, T, K, dev), *_arg(router_w, "router_w", bf16, E, K, dev), *_arg3(gate_w, "gate_w", (E, N, K), dev),
           *_arg3(up_w, "up_w", (E, N, K), dev), *_arg3(down_w, "down_w", (E, K, N), dev))
    with _allocate_on(dev, stream):
        if out is None:
            out = torch.empty((T, K), dtype=bf16, device=dev)
        if ids is None:
            ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        if weights is None:
            weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        for t, name, dtype in ((ids, "ids", torch.int32), (weights, "weights", torch.float32)):
            _check_operand(t, name, dtype, (T, top_k), dev)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if workspace is None:
            workspace = new_moe_workspace(T, E, top_k, N, K, dev)
        wsp, wsb, keep = _workspace(workspace, 0, dev)
        st = lib().moe_glu(*ins, *_arg(out, "out", bf16, T, K, dev), ids.data_ptr(), weights.data_ptr(), T, E, top_k, N, K,
                           int(bool(renormalize)), wsp, wsb, _stream_of(dev, stream))
    if st != 0:
        raise MbgluError(st, "moe_glu")
    return out, ids, weights


def glu_lora_workspace_bytes(M, N, K, adapters, R):
    """Bytes with which glu_lora takes its fastest kernels at any number of rows up to M
    (0: none needed)."""
    return lib().glu_lora_workspace_bytes(M, N, K, adapters, R)


def linear_lora_workspace_bytes(M, N, K, adapters, R):
    """Bytes with which linear_lora takes its fastest kernels at any number of rows up to
    M (0: none needed)."""
    return lib().linear_lora_workspace_bytes(M, N, K, adapters, R)


def moe_glu_workspace_bytes(T, E, top_k, N, K):
    """Bytes of moe_glu's workspace; what holds for T tokens holds for fewer."""
    return lib().moe_glu_workspace_bytes(T, E, top_k, N, K)


def silu_mul(x, out=None, mode="fused", stream=None):
    """out[M,N] = SiLU(x[:, :N]) * x[:, N:2N] on the halves layout (the gate
    projection in the first half of each row, the up projection in the second,
    as a GEMM on the concatenated [gate; up] weight leaves them); mode "fused"
    (one rounding) or "hf" (SiLU rounded to bf16 first).  x is [M, 2N] (or
    [2N]) bf16 with a contiguous last dimension; any row stride."""
    squeeze = x.dim() == 1
    x2 = x.unsqueeze(0) if squeeze else x
    _check(x2, "x", 2)
    M, W = x2.shape
    if W % 2:
        raise ValueError(f"x must have an even number of columns (gate half, up half), got {W}")
    N = W // 2
    dev = x2.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    out2 = out.unsqueeze(0) if out.dim() == 1 else out
    _check(out2, "out", 2)
    if tuple(out2.shape) != (M, N) or out2.device != dev:
        raise ValueError(f"out must be [{M},{N}] on {dev}")
    with _on(dev):
        st = lib().silu_mul(x2.data_ptr(), x2.stride(0), out2.data_ptr(), out2.stride(0), M, N, _MODES[mode],
                            _stream_handle(dev, stream))
    if st != 0:
        raise MbgluError(st, "silu_mul")
    return out2.view(N) if squeeze else out


def gdn_gates(a, b, A_log, dt_bias, g=None, beta=None, stream=None):
    """Gated-delta-net gates: g = -exp(A_log) * softplus(a + dt_bias) (fp32)
    and beta = sigmoid(b) (bf16), per token and head.  a, b are [T, H] bf16
    (row-strided views allowed, contiguous last dimension); A_log, dt_bias are
    contiguous [H] float32.  Returns (g, beta)."""
    _check(a, "a", 2)
    _check(b, "b", 2)
    T, H = a.shape
    if tuple(b.shape) != (T, H):
        raise ValueError(f"b must be [{T},{H}]")
    for t, name in ((A_log, "A_log"), (dt_bias, "dt_bias")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != (H,) \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape [{H}]")
    dev = a.device
    if g is None:
        g = torch.empty((T, H), dtype=torch.float32, device=dev)
    if beta is None:
        beta = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if g.dtype != torch.float32 or tuple(g.shape) != (T, H) or (g.numel() and g.stride(-1) != 1):
        raise ValueError(f"g must be a float32 [{T},{H}] tensor with a contiguous last dimension")
    _check(beta, "beta", 2)
    if tuple(beta.shape) != (T, H):
        raise ValueError(f"beta must be [{T},{H}]")
    with _on(dev):
        st = lib().gdn_gates(a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(0), A_log.data_ptr(),
                             dt_bias.data_ptr(), g.data_ptr(), g.stride(0), beta.data_ptr(), beta.stride(0), T, H,
                             _stream_handle(dev, stream))
    if st != 0:
        raise MbgluError(st, "gdn_gates")
    return g, beta


def last_variant() -> int:
    """Kernel the calling thread's last call launched: 0 none, 1 streaming
    (CUDA-core), 2 generic, 3 zero fill, 4 tensor cores with h in shared
    memory (batch >= 3), 5 silu_mul, 6 gdn_gates, 7 row blocks, 8
    glu_backward, 9 tcgen05, 10 the K-slice tensor-core kernel (batch 1..16),
    11 glu_gemm on the CTA-pair tcgen05 kernel, 12 glu_gemm at any alignment,
    13 glu_gemm_backward, 14 add_rmsnorm_fp8, 15..17 an e4m3 product (CTA pairs,
    few rows, any alignment), 18 quantize_weight_fp8, 19 and 20 glu_lora and
    linear_lora (CTA pairs, any alignment), 21 and 22 moe_glu (one kernel, any
    alignment)."""
    return lib().mbglu_last_variant()


def last_backward_path() -> int:
    """The second step of the calling thread's last glu_backward: 0 none, 1
    separate kernels, 2 one pass on the CUDA cores, 3 one pass on the tensor
    cores; of glu_gemm_backward: 4 the CTA-pair tcgen05 kernels, 5 the kernels
    for any alignment."""
    return lib().mbglu_last_backward_path()


PRODUCTS = ("glu_gemm", "grad_h", "grad_w", "glu_fp8", "matmul_fp8")


def block_plan(product, M, N, K):
    """How a product of the gated block (one of PRODUCTS) is laid out for operands
    that tensor copies take: (1 for the kernels of few rows or few tiles, tokens and
    outputs per tile, tiles done whole, tiles in ranges, ranges of each); see
    include/mbglu.h."""
    plan = (ctypes.c_int * 6)()
    st = lib().mbglu_block_plan(PRODUCTS.index(product), M, N, K, plan)
    if st != 0:
        raise MbgluError(st, "mbglu_block_plan")
    return tuple(plan)


def read_device_error() -> int:
    """Synchronises the current device, returns and clears its error word."""
    w = ctypes.c_int(0)
    st = lib().mbglu_read_device_error(ctypes.byref(w))
    if st != 0:
        raise MbgluError(st, "mbglu_read_device_error")
    return w.value


def set_launch_policy(policy: int) -> None:
    """0 serial, 1 programmatic dependent launch, 2 PDL + weight prefetch
    before the dependency wait (default; see include/mbglu.h for the contract)."""
    st = lib().mbglu_set_launch_policy(int(policy))
    if st != 0:
        raise MbgluError(st, "mbglu_set_launch_policy")


def get_launch_policy() -> int:
    return lib().mbglu_get_launch_policy()
