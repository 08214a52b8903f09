// bind_torch.cpp -- the common case of the binding's wide and e4m3 calls, and of
// those whose rows choose weights of their own: tensors of the right type, shape
// and device, on the current device's current stream.  Marshalling only, as
// binding.py, whose argument checks take longer than a decode step's kernels.  A
// call that is not the common case returns None and binding.py does it, with its
// own checks and errors.
//
// Each function returns what the Python function returns, None (not the common
// case: nothing was launched), or a non-zero status as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mbglu.h"

namespace {

using at::ScalarType;

decltype(&::glu_gemm) f_gemm = nullptr;
decltype(&::glu_gemm_backward) f_gemm_backward = nullptr;
decltype(&::glu_gemm_backward_workspace_bytes) f_gemm_backward_ws = nullptr;
decltype(&::add_rmsnorm_fp8) f_norm = nullptr;
decltype(&::glu_fp8) f_glu = nullptr;
decltype(&::matmul_fp8) f_matmul = nullptr;
decltype(&::matmul_fp8_workspace_bytes) f_matmul_ws = nullptr;
decltype(&::glu_lora) f_glu_lora = nullptr;
decltype(&::glu_lora_workspace_bytes) f_glu_lora_ws = nullptr;
decltype(&::linear_lora) f_linear_lora = nullptr;
decltype(&::linear_lora_workspace_bytes) f_linear_lora_ws = nullptr;
decltype(&::moe_glu) f_moe = nullptr;

constexpr ScalarType kBf16 = ScalarType::BFloat16, kE4m3 = ScalarType::Float8_e4m3fn, kF32 = ScalarType::Float;

struct Operand {
    void *p = nullptr;
    int64_t ld = 0;
};

// A 2-D CUDA tensor of type `type`: its sizes and device, or false.
bool first(PyObject *o, ScalarType type, int64_t &rows, int64_t &cols, int &device)
{
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() != 2 || t.scalar_type() != type) return false;
    rows = t.size(0);
    cols = t.size(1);
    device = t.get_device();
    return rows <= INT32_MAX && cols <= INT32_MAX / 2 && device == c10::cuda::current_device();
}

bool operand(const at::Tensor &t, ScalarType type, int64_t rows, int64_t cols, int device, Operand &out)
{
    if (!t.is_cuda() || t.get_device() != device || t.dim() != 2 || t.scalar_type() != type || t.size(0) != rows ||
        t.size(1) != cols || t.stride(1) != 1 || (rows > 1 && t.stride(0) < cols))
        return false;
    out.p = t.data_ptr();
    out.ld = rows > 1 ? t.stride(0) : cols;
    return true;
}

bool operand(PyObject *o, ScalarType type, int64_t rows, int64_t cols, int device, Operand &out)
{
    return THPVariable_Check(o) && operand(THPVariable_Unpack(o), type, rows, cols, device, out);
}

at::Tensor empty(int64_t rows, int64_t cols, ScalarType type, int device)
{
    return at::empty({rows, cols}, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
}

// e4m3 rows start on 16 bytes
at::Tensor empty_e4m3(int64_t rows, int64_t cols, int device)
{
    const int64_t wide = (cols + 15) / 16 * 16;
    at::Tensor t = empty(rows, wide, kE4m3, device);
    return wide == cols ? t : t.narrow(1, 0, cols);
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

cudaStream_t stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

PyObject *status(mbglu_status st) { return PyLong_FromLong(st); }

// The output at `given`, or a new one (kept alive in `made`).
bool output(PyObject *given, ScalarType type, int64_t rows, int64_t cols, int device, Operand &out, at::Tensor &made)
{
    if (given != Py_None) return operand(given, type, rows, cols, device, out);
    made = type == kE4m3 ? empty_e4m3(rows, cols, device) : empty(rows, cols, type, device);
    out.p = made.data_ptr();
    out.ld = rows > 1 ? made.stride(0) : cols;
    return true;
}

PyObject *result(PyObject *given, at::Tensor &made)
{
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(std::move(made));
}

PyObject *pair(PyObject *a, PyObject *b)
{
    PyObject *t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return t;
}

// No C++ exception leaves a function of the module.
template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
        return nullptr;
    }
}

// (h, gate_w, up_w, out, mode, gu)
PyObject *py_gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2;
        int dev, dev2;
        if (n != 6 || !first(a[0], kBf16, M, K, dev) || !first(a[1], kBf16, N, K2, dev2)) Py_RETURN_NONE;
        Operand h, g, u, o, gu;
        at::Tensor made;
        if (!operand(a[0], kBf16, M, K, dev, h) || !operand(a[1], kBf16, N, K, dev, g) || !operand(a[2], kBf16, N, K, dev, u) ||
            (a[5] != Py_None && !operand(a[5], kF32, M, 2 * N, dev, gu)) || !output(a[3], kBf16, M, N, dev, o, made))
            Py_RETURN_NONE;
        const long mode = PyLong_AsLong(a[4]);
        const mbglu_status st = f_gemm(static_cast<mbglu_bf16 *>(h.p), h.ld, static_cast<mbglu_bf16 *>(g.p), g.ld,
                                       static_cast<mbglu_bf16 *>(u.p), u.ld, static_cast<mbglu_bf16 *>(o.p), o.ld,
                                       static_cast<float *>(gu.p), gu.ld, static_cast<int>(M), static_cast<int>(N),
                                       static_cast<int>(K), static_cast<mbglu_mode>(mode), stream_of(dev));
        return st ? status(st) : result(a[3], made);
    });
}

// The autograd node of DualWeightGlu above the decode batch: forward keeps g and u
// in fp32, backward runs without the interpreter (a Python node costs the engine's
// thread two hand-overs of the interpreter lock).  A failing status becomes an
// exception, which autograd hands to the caller.
void must(mbglu_status st, const char *what)
{
    TORCH_CHECK(st == MBGLU_OK, what, ": status ", st);
}

struct WideGlu : torch::autograd::Function<WideGlu> {
    static at::Tensor forward(torch::autograd::AutogradContext *ctx, const at::Tensor &h, const at::Tensor &gate, const at::Tensor &up,
                              int64_t mode)
    {
        const int64_t M = h.size(0), K = h.size(1), N = gate.size(0);
        const int dev = h.get_device();
        Operand a, g, u;
        TORCH_CHECK(operand(h, kBf16, M, K, dev, a) && operand(gate, kBf16, N, K, dev, g) && operand(up, kBf16, N, K, dev, u),
                    "glu_gemm: operands");
        at::Tensor out = empty(M, N, kBf16, dev), gu = empty(M, 2 * N, kF32, dev);
        must(f_gemm(static_cast<mbglu_bf16 *>(a.p), a.ld, static_cast<mbglu_bf16 *>(g.p), g.ld, static_cast<mbglu_bf16 *>(u.p), u.ld,
                    static_cast<mbglu_bf16 *>(out.data_ptr()), N, static_cast<float *>(gu.data_ptr()), 2 * N, static_cast<int>(M),
                    static_cast<int>(N), static_cast<int>(K), static_cast<mbglu_mode>(mode), stream_of(dev)),
             "glu_gemm");
        ctx->save_for_backward({h, gate, up, gu});
        return out;
    }

    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, torch::autograd::variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const at::Tensor &h = saved[0], &gate = saved[1], &up = saved[2], &gu = saved[3];
        const int64_t M = h.size(0), K = h.size(1), N = gate.size(0);
        const int dev = h.get_device();
        torch::autograd::variable_list out(4);
        if (!grads[0].defined()) return out;
        at::Tensor d = grads[0].to(kBf16);
        // a broadcast gradient (of a sum) has stride 0; a single column may have any, and
        // counts as contiguous all the same: a copy has the strides of its shape
        if (d.stride(1) != 1 || d.stride(0) < N) d = d.clone(at::MemoryFormat::Contiguous);
        Operand a, g, u, dd, oh, og, ou;
        TORCH_CHECK(operand(h, kBf16, M, K, dev, a) && operand(gate, kBf16, N, K, dev, g) && operand(up, kBf16, N, K, dev, u) &&
                        operand(d, kBf16, M, N, dev, dd),
                    "glu_gemm_backward: operands");
        const bool want_w = ctx->needs_input_grad(1) || ctx->needs_input_grad(2);
        at::Tensor gh, gg, gw, ws;
        if (ctx->needs_input_grad(0)) output(Py_None, kBf16, M, K, dev, oh, gh);
        if (want_w) {
            output(Py_None, kBf16, N, K, dev, og, gg);
            output(Py_None, kBf16, N, K, dev, ou, gw);
        }
        const size_t need = f_gemm_backward_ws(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K));
        if (need) ws = empty(1, static_cast<int64_t>(need), ScalarType::Byte, dev);
        must(f_gemm_backward(static_cast<mbglu_bf16 *>(a.p), a.ld, static_cast<mbglu_bf16 *>(g.p), g.ld, static_cast<mbglu_bf16 *>(u.p),
                             u.ld, static_cast<mbglu_bf16 *>(dd.p), dd.ld, static_cast<float *>(gu.data_ptr()), 2 * N,
                             static_cast<mbglu_bf16 *>(oh.p), oh.ld, static_cast<mbglu_bf16 *>(og.p), og.ld,
                             static_cast<mbglu_bf16 *>(ou.p), ou.ld, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                             need ? ws.data_ptr() : nullptr, need, stream_of(dev)),
             "glu_gemm_backward");
        out[0] = gh;
        if (ctx->needs_input_grad(1)) out[1] = gg;
        if (ctx->needs_input_grad(2)) out[2] = gw;
        if (at::GradMode::is_enabled()) {   // create_graph: a second derivative is an error, not a zero
            for (at::Tensor &x : out)
                if (x.defined()) x.set_requires_grad(true);
            const auto error = std::make_shared<torch::autograd::DelayedError>(
                "DualWeightGlu has no second derivative: its backward is differentiable once", static_cast<int64_t>(out.size()));
            return (*error)(std::move(out));
        }
        return out;
    }
};

// (h, gate_w, up_w, mode): with an autograd node
PyObject *py_wide_glu(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2;
        int dev, dev2;
        if (n != 4 || !first(a[0], kBf16, M, K, dev) || !first(a[1], kBf16, N, K2, dev2) || M == 0 || N == 0 || K == 0)
            Py_RETURN_NONE;
        Operand o;
        for (int i = 0; i < 3; ++i)
            if (!operand(a[i], kBf16, i ? N : M, K, dev, o)) Py_RETURN_NONE;
        const long mode = PyLong_AsLong(a[3]);
        return THPVariable_Wrap(WideGlu::apply(THPVariable_Unpack(a[0]), THPVariable_Unpack(a[1]), THPVariable_Unpack(a[2]),
                                               static_cast<int64_t>(mode)));
    });
}

// (h, gate_w, up_w, dout, gu, want_h, want_w): new gradients and workspace
PyObject *py_gemm_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2;
        int dev, dev2;
        if (n != 7 || !first(a[0], kBf16, M, K, dev) || !first(a[1], kBf16, N, K2, dev2)) Py_RETURN_NONE;
        Operand h, g, u, d, gu, oh, og, ou;
        at::Tensor gh, gg, gw, ws;
        if (!operand(a[0], kBf16, M, K, dev, h) || !operand(a[1], kBf16, N, K, dev, g) || !operand(a[2], kBf16, N, K, dev, u) ||
            !operand(a[3], kBf16, M, N, dev, d) || (a[4] != Py_None && !operand(a[4], kF32, M, 2 * N, dev, gu)))
            Py_RETURN_NONE;
        if (a[5] == Py_True) output(Py_None, kBf16, M, K, dev, oh, gh);
        if (a[6] == Py_True) {
            output(Py_None, kBf16, N, K, dev, og, gg);
            output(Py_None, kBf16, N, K, dev, ou, gw);
        }
        const size_t need = f_gemm_backward_ws(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K));
        if (need) ws = empty(1, static_cast<int64_t>(need), ScalarType::Byte, dev);
        const mbglu_status st = f_gemm_backward(
            static_cast<mbglu_bf16 *>(h.p), h.ld, static_cast<mbglu_bf16 *>(g.p), g.ld, static_cast<mbglu_bf16 *>(u.p), u.ld,
            static_cast<mbglu_bf16 *>(d.p), d.ld, static_cast<float *>(gu.p), gu.ld, static_cast<mbglu_bf16 *>(oh.p), oh.ld,
            static_cast<mbglu_bf16 *>(og.p), og.ld, static_cast<mbglu_bf16 *>(ou.p), ou.ld, static_cast<int>(M),
            static_cast<int>(N), static_cast<int>(K), need ? ws.data_ptr() : nullptr, need, stream_of(dev));
        if (st) return status(st);
        PyObject *r[3] = {nullptr, nullptr, nullptr};
        at::Tensor *made[3] = {&gh, &gg, &gw};
        for (int i = 0; i < 3; ++i) {
            if (made[i]->defined()) {
                r[i] = THPVariable_Wrap(std::move(*made[i]));
            } else {
                Py_INCREF(Py_None);
                r[i] = Py_None;
            }
        }
        PyObject *t = r[0] && r[1] && r[2] ? PyTuple_Pack(3, r[0], r[1], r[2]) : nullptr;
        for (PyObject *x : r) Py_XDECREF(x);
        return t;
    });
}

// (x, residual, norm_w, eps, q, scale, residual_out)
PyObject *py_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K;
        int dev;
        if (n != 7 || !PyFloat_Check(a[3]) || !first(a[0], kBf16, M, K, dev) || !THPVariable_Check(a[2])) Py_RETURN_NONE;
        const at::Tensor &w = THPVariable_Unpack(a[2]);
        if (!w.is_cuda() || w.get_device() != dev || w.dim() != 1 || w.size(0) != K || w.scalar_type() != kBf16 ||
            !w.is_contiguous())
            Py_RETURN_NONE;
        Operand x, r, ro, q, s;
        at::Tensor mq, ms;
        if (!operand(a[0], kBf16, M, K, dev, x) || !operand(a[1], kBf16, M, K, dev, r) ||
            !operand(a[6] == Py_None ? a[1] : a[6], kBf16, M, K, dev, ro) || !output(a[4], kE4m3, M, K, dev, q, mq) ||
            !output(a[5], kF32, M, blocks(K), dev, s, ms))
            Py_RETURN_NONE;
        const mbglu_status st =
            f_norm(static_cast<mbglu_bf16 *>(x.p), x.ld, static_cast<mbglu_bf16 *>(r.p), r.ld, static_cast<mbglu_bf16 *>(ro.p),
                   ro.ld, static_cast<mbglu_bf16 *>(w.data_ptr()), static_cast<float>(PyFloat_AS_DOUBLE(a[3])),
                   static_cast<uint8_t *>(q.p), q.ld, static_cast<float *>(s.p), s.ld, static_cast<int>(M),
                   static_cast<int>(K), stream_of(dev));
        return st ? status(st) : pair(result(a[4], mq), result(a[5], ms));
    });
}

// (a, a_scale, gate_w, gate_scale, up_w, up_scale, out, out_scale, quant)
PyObject *py_glu(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2;
        int dev, dev2;
        if (n != 9 || !first(a[0], kE4m3, M, K, dev) || !first(a[2], kE4m3, N, K2, dev2)) Py_RETURN_NONE;
        const int64_t kb = blocks(K), nb = blocks(N);
        const bool quant = a[8] == Py_True;
        Operand x, xs, g, gs, u, us, o, os;
        at::Tensor mo, ms;
        if (!operand(a[0], kE4m3, M, K, dev, x) || !operand(a[1], kF32, M, kb, dev, xs) || !operand(a[2], kE4m3, N, K, dev, g) ||
            !operand(a[3], kF32, nb, kb, dev, gs) || !operand(a[4], kE4m3, N, K, dev, u) ||
            !operand(a[5], kF32, nb, kb, dev, us) || (!quant && a[7] != Py_None) ||
            !output(a[6], quant ? kE4m3 : kBf16, M, N, dev, o, mo) || (quant && !output(a[7], kF32, M, nb, dev, os, ms)))
            Py_RETURN_NONE;
        const mbglu_status st =
            f_glu(static_cast<uint8_t *>(x.p), x.ld, static_cast<float *>(xs.p), xs.ld, static_cast<uint8_t *>(g.p), g.ld,
                  static_cast<float *>(gs.p), gs.ld, static_cast<uint8_t *>(u.p), u.ld, static_cast<float *>(us.p), us.ld,
                  quant ? nullptr : static_cast<mbglu_bf16 *>(o.p), quant ? 0 : o.ld,
                  quant ? static_cast<uint8_t *>(o.p) : nullptr, quant ? o.ld : 0, static_cast<float *>(os.p), os.ld,
                  static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), stream_of(dev));
        if (st) return status(st);
        return quant ? pair(result(a[6], mo), result(a[7], ms)) : result(a[6], mo);
    });
}

// (a, a_scale, w, w_scale, out): a workspace of its own
PyObject *py_matmul(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2;
        int dev, dev2;
        if (n != 5 || !first(a[0], kE4m3, M, K, dev) || !first(a[2], kE4m3, N, K2, dev2)) Py_RETURN_NONE;
        const int64_t kb = blocks(K);
        Operand x, xs, w, ws, o;
        at::Tensor mo, scratch;
        if (!operand(a[0], kE4m3, M, K, dev, x) || !operand(a[1], kF32, M, kb, dev, xs) || !operand(a[2], kE4m3, N, K, dev, w) ||
            !operand(a[3], kF32, blocks(N), kb, dev, ws) || !output(a[4], kBf16, M, N, dev, o, mo))
            Py_RETURN_NONE;
        const size_t need = f_matmul_ws(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K));
        if (need) scratch = empty(1, static_cast<int64_t>(need), ScalarType::Byte, dev);
        const mbglu_status st =
            f_matmul(static_cast<uint8_t *>(x.p), x.ld, static_cast<float *>(xs.p), xs.ld, static_cast<uint8_t *>(w.p), w.ld,
                     static_cast<float *>(ws.p), ws.ld, static_cast<mbglu_bf16 *>(o.p), o.ld, static_cast<int>(M),
                     static_cast<int>(N), static_cast<int>(K), need ? scratch.data_ptr() : nullptr, need, stream_of(dev));
        return st ? status(st) : result(a[4], mo);
    });
}

// A 3-D bf16 tensor [count, rows, cols]: its address and strides.
bool stack(PyObject *o, int64_t count, int64_t rows, int64_t cols, int device, Operand &out, int64_t &outer)
{
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || t.dim() != 3 || t.scalar_type() != kBf16 || t.size(0) != count ||
        t.size(1) != rows || t.size(2) != cols || t.stride(2) != 1)
        return false;
    out.p = t.data_ptr();
    out.ld = rows > 1 ? t.stride(1) : cols;
    outer = count > 1 ? t.stride(0) : rows * out.ld;
    return true;
}

bool vector(PyObject *o, ScalarType type, int64_t n, int device, void *&p)
{
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || t.dim() != 1 || t.scalar_type() != type || t.size(0) != n || !t.is_contiguous())
        return false;
    p = t.data_ptr();
    return true;
}

// The workspace at `given`, or a new one of `need` bytes (kept alive in `made`).
bool workspace(PyObject *given, size_t need, int device, void *&p, size_t &bytes, at::Tensor &made)
{
    if (given == Py_None) {
        if (need) made = empty(1, static_cast<int64_t>(need), ScalarType::Byte, device);
        p = need ? made.data_ptr() : nullptr;
        bytes = need;
        return true;
    }
    if (!THPVariable_Check(given)) return false;
    const at::Tensor &t = THPVariable_Unpack(given);
    if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) return false;
    p = t.data_ptr();
    bytes = t.nbytes();
    return true;
}

// (count, R) of A [count, R, K]
bool ranks(PyObject *o, int64_t &count, int64_t &R)
{
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 3) return false;
    count = t.size(0);
    R = t.size(1);
    return count <= INT32_MAX - 511 && R <= MBGLU_LORA_MAX_RANK;
}

bool adapters(PyObject *a, PyObject *b, int64_t N, int64_t K, int64_t count, int64_t R, int device, mbglu_adapters &out)
{
    Operand x, y;
    if (!stack(a, count, R, K, device, x, out.a_adapter) || !stack(b, count, N, R, device, y, out.b_adapter)) return false;
    out.a = static_cast<mbglu_bf16 *>(x.p);
    out.lda = x.ld;
    out.b = static_cast<mbglu_bf16 *>(y.p);
    out.ldb = y.ld;
    return true;
}

// (h, gate_w, up_w, gate_a, gate_b, up_a, up_b, adapter, scale, out, mode, workspace)
PyObject *py_glu_lora(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2, count, R;
        int dev, dev2;
        if (n != 12 || !first(a[0], kBf16, M, K, dev) || !first(a[1], kBf16, N, K2, dev2) || !ranks(a[3], count, R)) Py_RETURN_NONE;
        Operand h, g, u, o;
        mbglu_adapters ga, ua;
        void *index = nullptr, *scale = nullptr, *ws = nullptr;
        size_t bytes = 0;
        at::Tensor made, scratch;
        if (!operand(a[0], kBf16, M, K, dev, h) || !operand(a[1], kBf16, N, K, dev, g) || !operand(a[2], kBf16, N, K, dev, u) ||
            !adapters(a[3], a[4], N, K, count, R, dev, ga) || !adapters(a[5], a[6], N, K, count, R, dev, ua) ||
            !vector(a[7], ScalarType::Int, M, dev, index) || (a[8] != Py_None && !vector(a[8], kF32, count, dev, scale)))
            Py_RETURN_NONE;
        const size_t need = a[11] == Py_None ? f_glu_lora_ws(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                                                            static_cast<int>(count), static_cast<int>(R))
                                             : 0;
        if (!workspace(a[11], need, dev, ws, bytes, scratch) || !output(a[9], kBf16, M, N, dev, o, made)) Py_RETURN_NONE;
        const long mode = PyLong_AsLong(a[10]);
        const mbglu_status st = f_glu_lora(
            static_cast<mbglu_bf16 *>(h.p), h.ld, static_cast<mbglu_bf16 *>(g.p), g.ld, static_cast<mbglu_bf16 *>(u.p), u.ld, &ga, &ua,
            static_cast<int32_t *>(index), static_cast<float *>(scale), static_cast<mbglu_bf16 *>(o.p), o.ld, static_cast<int>(M),
            static_cast<int>(N), static_cast<int>(K), static_cast<int>(count), static_cast<int>(R), static_cast<mbglu_mode>(mode), ws,
            bytes, stream_of(dev));
        return st ? status(st) : result(a[9], made);
    });
}

// (x, w, a, b, adapter, scale, out, workspace)
PyObject *py_linear_lora(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t M, K, N, K2, count, R;
        int dev, dev2;
        if (n != 8 || !first(a[0], kBf16, M, K, dev) || !first(a[1], kBf16, N, K2, dev2) || !ranks(a[2], count, R)) Py_RETURN_NONE;
        Operand x, w, o;
        mbglu_adapters ab;
        void *index = nullptr, *scale = nullptr, *ws = nullptr;
        size_t bytes = 0;
        at::Tensor made, scratch;
        if (!operand(a[0], kBf16, M, K, dev, x) || !operand(a[1], kBf16, N, K, dev, w) ||
            !adapters(a[2], a[3], N, K, count, R, dev, ab) || !vector(a[4], ScalarType::Int, M, dev, index) ||
            (a[5] != Py_None && !vector(a[5], kF32, count, dev, scale)))
            Py_RETURN_NONE;
        const size_t need = a[7] == Py_None ? f_linear_lora_ws(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                                                              static_cast<int>(count), static_cast<int>(R))
                                            : 0;
        if (!workspace(a[7], need, dev, ws, bytes, scratch) || !output(a[6], kBf16, M, N, dev, o, made)) Py_RETURN_NONE;
        const mbglu_status st =
            f_linear_lora(static_cast<mbglu_bf16 *>(x.p), x.ld, static_cast<mbglu_bf16 *>(w.p), w.ld, &ab, static_cast<int32_t *>(index),
                          static_cast<float *>(scale), static_cast<mbglu_bf16 *>(o.p), o.ld, static_cast<int>(M), static_cast<int>(N),
                          static_cast<int>(K), static_cast<int>(count), static_cast<int>(R), ws, bytes, stream_of(dev));
        return st ? status(st) : result(a[6], made);
    });
}

// (h, router_w, gate_w, up_w, down_w, top_k, renormalize, out, ids, weights, workspace): with a workspace
PyObject *py_moe(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        int64_t T, K, E, K2, N;
        int dev, dev2;
        if (n != 11 || a[10] == Py_None || !PyLong_CheckExact(a[5]) || !first(a[0], kBf16, T, K, dev) || !first(a[1], kBf16, E, K2, dev2) ||
            !THPVariable_Check(a[2]) || THPVariable_Unpack(a[2]).dim() != 3)
            Py_RETURN_NONE;
        N = THPVariable_Unpack(a[2]).size(1);
        const long k = PyLong_AsLong(a[5]);
        if (PyErr_Occurred()) {   // beyond a long: the checks in Python say so
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        if (T > MBGLU_MAX_M || E < 1 || E > MBGLU_MOE_MAX_EXPERTS || k < 1 || k > E || k > MBGLU_MOE_MAX_TOP_K || N > INT32_MAX - 511)
            Py_RETURN_NONE;
        Operand h, r, g, u, d, o, ids, w;
        int64_t ge, ue, de;
        void *ws = nullptr;
        size_t bytes = 0;
        at::Tensor made, made_ids, made_w, scratch;
        if (!operand(a[0], kBf16, T, K, dev, h) || !operand(a[1], kBf16, E, K, dev, r) || !stack(a[2], E, N, K, dev, g, ge) ||
            !stack(a[3], E, N, K, dev, u, ue) || !stack(a[4], E, K, N, dev, d, de) || !workspace(a[10], 0, dev, ws, bytes, scratch) ||
            !output(a[7], kBf16, T, K, dev, o, made) || !output(a[8], ScalarType::Int, T, k, dev, ids, made_ids) ||
            !output(a[9], kF32, T, k, dev, w, made_w) || ids.ld != k || w.ld != k)
            Py_RETURN_NONE;
        const mbglu_status st = f_moe(
            static_cast<mbglu_bf16 *>(h.p), h.ld, static_cast<mbglu_bf16 *>(r.p), r.ld, static_cast<mbglu_bf16 *>(g.p), ge, g.ld,
            static_cast<mbglu_bf16 *>(u.p), ue, u.ld, static_cast<mbglu_bf16 *>(d.p), de, d.ld, static_cast<mbglu_bf16 *>(o.p), o.ld,
            static_cast<int32_t *>(ids.p), static_cast<float *>(w.p), static_cast<int>(T), static_cast<int>(E), static_cast<int>(k),
            static_cast<int>(N), static_cast<int>(K), a[6] == Py_True, ws, bytes, stream_of(dev));
        if (st) return status(st);
        PyObject *x = result(a[7], made), *y = result(a[8], made_ids), *z = result(a[9], made_w);
        PyObject *t = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        Py_XDECREF(z);
        return t;
    });
}

// The addresses of the library's entry points, in this order.
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    constexpr int kEntries = 12;
    if (n != kEntries) {
        PyErr_SetString(PyExc_TypeError, "bind takes twelve addresses");
        return nullptr;
    }
    void *p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    f_gemm = reinterpret_cast<decltype(f_gemm)>(p[0]);
    f_gemm_backward = reinterpret_cast<decltype(f_gemm_backward)>(p[1]);
    f_gemm_backward_ws = reinterpret_cast<decltype(f_gemm_backward_ws)>(p[2]);
    f_norm = reinterpret_cast<decltype(f_norm)>(p[3]);
    f_glu = reinterpret_cast<decltype(f_glu)>(p[4]);
    f_matmul = reinterpret_cast<decltype(f_matmul)>(p[5]);
    f_matmul_ws = reinterpret_cast<decltype(f_matmul_ws)>(p[6]);
    f_glu_lora = reinterpret_cast<decltype(f_glu_lora)>(p[7]);
    f_glu_lora_ws = reinterpret_cast<decltype(f_glu_lora_ws)>(p[8]);
    f_linear_lora = reinterpret_cast<decltype(f_linear_lora)>(p[9]);
    f_linear_lora_ws = reinterpret_cast<decltype(f_linear_lora_ws)>(p[10]);
    f_moe = reinterpret_cast<decltype(f_moe)>(p[11]);
    Py_RETURN_NONE;
}

#define MBGLU_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    MBGLU_METHOD("bind", py_bind),         MBGLU_METHOD("glu_gemm", py_gemm),
    MBGLU_METHOD("wide_glu", py_wide_glu),
    MBGLU_METHOD("glu_gemm_backward", py_gemm_backward), MBGLU_METHOD("add_rmsnorm_fp8", py_norm),
    MBGLU_METHOD("glu_fp8", py_glu),       MBGLU_METHOD("matmul_fp8", py_matmul),
    MBGLU_METHOD("glu_lora", py_glu_lora), MBGLU_METHOD("linear_lora", py_linear_lora),
    MBGLU_METHOD("moe_glu", py_moe),
    {nullptr, nullptr, 0, nullptr}};

// MBGLU_BUILT_FOR: the torch and the Python whose headers this was compiled with
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mbglu_torch", MBGLU_BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mbglu_torch(void) { return PyModule_Create(&module); }
