// The common case of the operators' Python calls (bit_exact_xor_gb300/ops.py)
// without Python in between: tensors on the current device, laid out as the
// kernels want them, on the current stream.  Each function returns None where
// a call is not of that kind; ops.py then takes it, with every check and
// message spelled out.  A status other than DCR_OK comes back as an int.
// torch_version names the torch that it was built for (-DDCR_TORCH_VERSION).
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dcr_ops.h"

namespace {

using at::Tensor;

int code_of(at::ScalarType t)
{
    return t == at::kFloat ? DCR_F32 : t == at::kBFloat16 ? DCR_BF16 : t == at::kHalf ? DCR_F16 : DCR_NONE;
}
at::ScalarType type_of(long code) { return code == DCR_F32 ? at::kFloat : code == DCR_BF16 ? at::kBFloat16 : at::kHalf; }


// A two-dimensional CUDA matrix of one of the three types on the current
// device, contiguous in its last dimension.
struct Matrix {
    Tensor t;
    int64_t rows = 0, cols = 0, stride = 0;
    int type = DCR_NONE;
    bool set(PyObject* o)
    {
        if (!THPVariable_Check(o)) return false;
        t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.dim() != 2 || t.layout() != at::kStrided) return false;
        type = code_of(t.scalar_type());
        rows = t.size(0), cols = t.size(1), stride = rows > 1 ? t.stride(0) : cols;
        return type != DCR_NONE && t.get_device() == c10::cuda::current_device() && (cols <= 1 || t.stride(1) == 1) && stride >= cols;
    }
};

bool flat(PyObject* o, const Tensor& like, at::ScalarType type, int64_t n, void** p)
{
    if (!THPVariable_Check(o)) return false;
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || t.numel() != n || t.device() != like.device() || !t.is_contiguous()) return false;
    *p = t.data_ptr();
    return true;
}

Tensor make(at::IntArrayRef size, at::ScalarType type, const Tensor& like)
{
    return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// quantize(x, scale or None, per_row, values type code) -> (codes, scales, scale, values or None)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix x;
    if (n != 4 || !x.set(a[0]) || x.cols % 16 || x.t.numel() == 0) Py_RETURN_NONE;
    const int per_row = PyObject_IsTrue(a[2]);
    if (per_row < 0) return nullptr;
    const bool given = a[1] != Py_None;
    const long vt = PyLong_AsLong(a[3]);
    if (vt < DCR_F32 || vt > DCR_NONE) Py_RETURN_NONE;
    void* sp = nullptr;
    if (given && (per_row || !flat(a[1], x.t, at::kFloat, 1, &sp))) Py_RETURN_NONE;
    Tensor codes = make({x.rows, x.cols / 2}, at::kByte, x.t), scales = make({x.rows, x.cols / 16}, at::kByte, x.t), scale, work, values;
    if (!given) {
        scale = make({per_row ? x.rows : 1}, at::kFloat, x.t);
        sp = scale.data_ptr();
        if (!per_row) work = make({int64_t(DCR_QUANT_PARTIALS)}, at::kFloat, x.t);
    }
    if (vt != DCR_NONE) values = make({x.rows, x.cols}, type_of(vt), x.t);
    const int rc = dcr_nvfp4_quantize(x.t.data_ptr(), x.type, x.rows, x.cols, x.stride, given ? DCR_SCALE_GIVEN : per_row ? DCR_SCALE_ROW : DCR_SCALE_TENSOR,
                                      static_cast<float*>(sp), codes.data_ptr(), scales.data_ptr(), values.defined() ? values.data_ptr() : nullptr,
                                      uint32_t(vt), work.defined() ? work.data_ptr() : nullptr, stream_of(x.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    PyObject* s = given ? (Py_INCREF(a[1]), a[1]) : wrap(std::move(scale));
    PyObject* v = values.defined() ? wrap(std::move(values)) : (Py_INCREF(Py_None), Py_None);
    return Py_BuildValue("(NNNN)", wrap(std::move(codes)), wrap(std::move(scales)), s, v);
    END_HANDLE_TH_ERRORS
}

// linear(x, codes, scales, scale, offsets or None, type code) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix x;
    if (n != 6 || !x.set(a[0]) || !THPVariable_Check(a[1]) || !THPVariable_Check(a[2]) || !THPVariable_Check(a[3])) Py_RETURN_NONE;
    const Tensor &codes = THPVariable_Unpack(a[1]), &scales = THPVariable_Unpack(a[2]), &scale = THPVariable_Unpack(a[3]);
    const at::ScalarType st = scales.scalar_type();
    if (codes.scalar_type() != at::kByte || codes.dim() != 2 || !codes.is_contiguous() || codes.device() != x.t.device() ||
        codes.size(1) * 2 != x.cols || x.cols == 0 || x.cols % 32 || (st != at::kByte && st != at::kFloat8_e4m3fn) ||
        scales.numel() != codes.size(0) * (x.cols / 16) || !scales.is_contiguous() || scales.device() != x.t.device() ||
        scale.scalar_type() != at::kFloat || !scale.is_contiguous() || scale.device() != x.t.device())
        Py_RETURN_NONE;
    int64_t experts = 0;
    void* offsets = nullptr;
    if (a[4] != Py_None) {
        if (!THPVariable_Check(a[4])) Py_RETURN_NONE;
        experts = THPVariable_Unpack(a[4]).numel() - 1;
        if (experts < 1 || experts > int64_t(DCR_MAX_EXPERTS) || codes.size(0) % experts || !flat(a[4], x.t, at::kInt, experts + 1, &offsets))
            Py_RETURN_NONE;
    }
    const long t = PyLong_AsLong(a[5]);
    const int64_t rows = codes.size(0) / (experts ? experts : 1);
    Tensor y = make({x.rows, rows}, type_of(t), x.t), work = make({int64_t(DCR_LINEAR_WORKSPACE(x.rows, x.cols))}, at::kByte, x.t);
    const dcr_nvfp4 w = {codes.data_ptr(), scales.data_ptr(), scale.data_ptr<float>(), uint64_t(scale.numel())};
    const int rc = dcr_nvfp4_linear(x.t.data_ptr(), x.type, x.stride, &w, x.rows, rows, x.cols, static_cast<const int32_t*>(offsets),
                                    uint32_t(experts), y.data_ptr(), uint32_t(t), rows, work.data_ptr(), stream_of(x.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// loss(logits, tokens, old, advantages, weights, ref or None, clip_low, clip_high, kl, temperature, grad) -> (loss, logp, grad or None)
PyObject* loss(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix z;
    if (n != 11 || !z.set(a[0])) Py_RETURN_NONE;
    void *tokens, *old, *adv, *w, *ref = nullptr;
    if (!flat(a[1], z.t, at::kLong, z.rows, &tokens) || !flat(a[2], z.t, at::kFloat, z.rows, &old) ||
        !flat(a[3], z.t, at::kFloat, z.rows, &adv) || !flat(a[4], z.t, at::kFloat, z.rows, &w) ||
        (a[5] != Py_None && !flat(a[5], z.t, at::kFloat, z.rows, &ref)))
        Py_RETURN_NONE;
    dcr_policy_opts o;
    o.clip_low = float(PyFloat_AsDouble(a[6])), o.clip_high = float(PyFloat_AsDouble(a[7]));
    o.kl_coef = float(PyFloat_AsDouble(a[8])), o.temperature = float(PyFloat_AsDouble(a[9]));
    if (PyErr_Occurred()) return nullptr;
    const bool want = a[10] == Py_True;
    Tensor out = make({}, at::kFloat, z.t), logp = make({z.rows}, at::kFloat, z.t), rows = make({z.rows}, at::kFloat, z.t), grad;
    if (want) grad = make({z.rows, z.cols}, z.t.scalar_type(), z.t);
    const int rc = dcr_policy_loss(z.t.data_ptr(), z.type, z.rows, z.cols, z.stride, static_cast<const int64_t*>(tokens),
                                   static_cast<const float*>(old), static_cast<const float*>(ref), static_cast<const float*>(adv),
                                   static_cast<const float*>(w), &o, out.data_ptr<float>(), rows.data_ptr<float>(), logp.data_ptr<float>(),
                                   want ? grad.data_ptr() : nullptr, z.cols, stream_of(z.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    PyObject* g = want ? wrap(std::move(grad)) : (Py_INCREF(Py_None), Py_None);
    return Py_BuildValue("(NNN)", wrap(std::move(out)), wrap(std::move(logp)), g);
    END_HANDLE_TH_ERRORS
}

// logprobs(logits, tokens, temperature) -> logp
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix z;
    void* tokens;
    if (n != 3 || !z.set(a[0]) || !flat(a[1], z.t, at::kLong, z.rows, &tokens)) Py_RETURN_NONE;
    const double temperature = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) return nullptr;
    Tensor logp = make({z.rows}, at::kFloat, z.t);
    const int rc = dcr_token_logprobs(z.t.data_ptr(), z.type, z.rows, z.cols, z.stride, static_cast<const int64_t*>(tokens),
                                      float(temperature), logp.data_ptr<float>(), stream_of(z.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return wrap(std::move(logp));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"loss", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(loss)), METH_FASTCALL, nullptr},
    {"logprobs", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(logprobs)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", DCR_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
