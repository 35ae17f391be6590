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

#include <vector>

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

// A number from a Python float or int; false with no error set where it is neither.
bool number(PyObject* o, double* v)
{
    if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
    *v = PyFloat_AsDouble(o);
    if (!PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
bool whole(PyObject* o, uint64_t most, uint64_t* v)
{
    if (!PyLong_Check(o)) return false;
    *v = PyLong_AsUnsignedLongLong(o);
    if (!PyErr_Occurred()) return *v <= most;
    PyErr_Clear();
    return false;
}
// A contiguous tensor of such a shape, or None where that is allowed.
bool slots(PyObject* o, const Tensor& like, at::ScalarType type, int64_t tokens, int64_t k, void** p)
{
    return flat(o, like, type, tokens * k, p) && THPVariable_Unpack(o).dim() == 2 && THPVariable_Unpack(o).size(1) == k;
}
PyObject* none() { return Py_INCREF(Py_None), Py_None; }

// scores(logits, tokens, top, temperature) -> (logp, entropy, top_logp or None, top_tokens or None, stats)
PyObject* scores(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix z;
    void* tokens;
    uint64_t top;
    double temperature;
    if (n != 4 || !z.set(a[0]) || !flat(a[1], z.t, at::kLong, z.rows, &tokens) || !whole(a[2], DCR_MAX_TOP, &top) || !number(a[3], &temperature) ||
        int64_t(top) > z.cols)
        Py_RETURN_NONE;
    Tensor logp = make({z.rows}, at::kFloat, z.t), entropy = make({z.rows}, at::kFloat, z.t), stats = make({z.rows, 3}, at::kFloat, z.t), tl, tt;
    if (top) tl = make({z.rows, int64_t(top)}, at::kFloat, z.t), tt = make({z.rows, int64_t(top)}, at::kLong, z.t);
    const int rc = dcr_token_scores(z.t.data_ptr(), z.type, z.rows, z.cols, z.stride, static_cast<const int64_t*>(tokens), float(temperature),
                                    uint32_t(top), logp.data_ptr<float>(), entropy.data_ptr<float>(), top ? tl.data_ptr<float>() : nullptr,
                                    top ? tt.data_ptr<int64_t>() : nullptr, stats.data_ptr<float>(), stream_of(z.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    PyObject *l = top ? wrap(std::move(tl)) : none(), *t = top ? wrap(std::move(tt)) : none();
    return Py_BuildValue("(NNNNN)", wrap(std::move(logp)), wrap(std::move(entropy)), l, t, wrap(std::move(stats)));
    END_HANDLE_TH_ERRORS
}

// scores_grad(logits, tokens, stats, grad_logp or None, grad_entropy or None, temperature) -> grad
PyObject* scores_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix z;
    void *tokens, *stats, *gl = nullptr, *ge = nullptr;
    double temperature;
    if (n != 6 || !z.set(a[0]) || !flat(a[1], z.t, at::kLong, z.rows, &tokens) || !flat(a[2], z.t, at::kFloat, z.rows * 3, &stats) ||
        (a[3] != Py_None && !flat(a[3], z.t, at::kFloat, z.rows, &gl)) || (a[4] != Py_None && !flat(a[4], z.t, at::kFloat, z.rows, &ge)) ||
        !number(a[5], &temperature))
        Py_RETURN_NONE;
    Tensor grad = make({z.rows, z.cols}, z.t.scalar_type(), z.t);
    const int rc = dcr_token_scores_grad(z.t.data_ptr(), z.type, z.rows, z.cols, z.stride, static_cast<const int64_t*>(tokens),
                                         static_cast<const float*>(stats), static_cast<const float*>(gl), static_cast<const float*>(ge),
                                         float(temperature), grad.data_ptr(), z.cols, stream_of(z.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return wrap(std::move(grad));
    END_HANDLE_TH_ERRORS
}

bool route_opts(PyObject* scoring, uint64_t k, PyObject* renormalise, PyObject* scale, dcr_route_opts* o)
{
    uint64_t s;
    double f;
    const int r = PyObject_IsTrue(renormalise);
    if (r < 0) PyErr_Clear();
    if (r < 0 || !whole(scoring, 1, &s) || !number(scale, &f)) return false;
    *o = {uint32_t(s), uint32_t(k), 1, 1, 1, uint32_t(r), float(f)};
    return true;
}

// route(logits, k, scoring code, bias or None, groups, group_top, group_by, renormalise, scale, mask or None)
// -> (experts, weights, offsets, order, positions)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix z;
    uint64_t k, groups, group_top, group_by;
    dcr_route_opts o;
    void *bias = nullptr, *mask = nullptr;
    if (n != 10 || !z.set(a[0]) || !whole(a[1], DCR_MAX_CHOSEN, &k) || k == 0 || int64_t(k) > z.cols || z.cols > int64_t(DCR_MAX_EXPERTS) ||
        !route_opts(a[2], k, a[7], a[8], &o) || (a[3] != Py_None && !flat(a[3], z.t, at::kFloat, z.cols, &bias)) || !whole(a[4], 1 << 20, &groups) ||
        !whole(a[5], 1 << 20, &group_top) || !whole(a[6], 1 << 20, &group_by) ||
        (a[9] != Py_None && !flat(a[9], z.t, at::kBool, z.rows, &mask) && !flat(a[9], z.t, at::kByte, z.rows, &mask)))
        Py_RETURN_NONE;
    o.groups = uint32_t(groups), o.group_top = uint32_t(group_top), o.group_by = uint32_t(group_by);
    const int64_t kk = int64_t(k);
    Tensor experts = make({z.rows, kk}, at::kInt, z.t), weights = make({z.rows, kk}, at::kFloat, z.t), offsets = make({z.cols + 1}, at::kInt, z.t),
           order = make({z.rows * kk}, at::kInt, z.t), positions = make({z.rows, kk}, at::kInt, z.t),
           work = make({int64_t(DCR_ROUTE_WORKSPACE(z.cols))}, at::kByte, z.t);
    const int rc = dcr_route(z.t.data_ptr(), z.type, z.rows, uint32_t(z.cols), z.stride, static_cast<const float*>(bias),
                             static_cast<const uint8_t*>(mask), &o, experts.data_ptr<int32_t>(), weights.data_ptr<float>(),
                             offsets.data_ptr<int32_t>(), order.data_ptr<int32_t>(), positions.data_ptr<int32_t>(), work.data_ptr(), stream_of(z.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("(NNNNN)", wrap(std::move(experts)), wrap(std::move(weights)), wrap(std::move(offsets)), wrap(std::move(order)),
                         wrap(std::move(positions)));
    END_HANDLE_TH_ERRORS
}

// route_grad(logits, experts, grad_weights, scoring code, renormalise, scale) -> grad
PyObject* route_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix z;
    void *chosen, *gw;
    dcr_route_opts o;
    if (n != 6 || !z.set(a[0]) || !THPVariable_Check(a[1]) || THPVariable_Unpack(a[1]).dim() != 2) Py_RETURN_NONE;
    const int64_t k = THPVariable_Unpack(a[1]).size(1);
    if (k < 1 || k > int64_t(DCR_MAX_CHOSEN) || !slots(a[1], z.t, at::kInt, z.rows, k, &chosen) || !slots(a[2], z.t, at::kFloat, z.rows, k, &gw) ||
        !route_opts(a[3], k, a[4], a[5], &o))
        Py_RETURN_NONE;
    Tensor grad = make({z.rows, z.cols}, z.t.scalar_type(), z.t);
    const int rc = dcr_route_grad(z.t.data_ptr(), z.type, z.rows, uint32_t(z.cols), z.stride, static_cast<const int32_t*>(chosen),
                                  static_cast<const float*>(gw), &o, grad.data_ptr(), z.cols, stream_of(z.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return wrap(std::move(grad));
    END_HANDLE_TH_ERRORS
}

// A Route's positions and, if asked for, weights.
struct Slots {
    int64_t tokens = 0, k = 0;
    void *positions = nullptr, *weights = nullptr;
    bool set(PyObject* pos, PyObject* w, const Tensor& like)
    {
        if (!THPVariable_Check(pos) || THPVariable_Unpack(pos).dim() != 2) return false;
        tokens = THPVariable_Unpack(pos).size(0), k = THPVariable_Unpack(pos).size(1);
        return k >= 1 && k <= int64_t(DCR_MAX_CHOSEN) && slots(pos, like, at::kInt, tokens, k, &positions) &&
               (w == Py_None || slots(w, like, at::kFloat, tokens, k, &weights));
    }
};

// A new matrix, or the one that is given if it is of that shape (and type, if t is one): its tensor, row stride and type code.
bool output(PyObject* o, int64_t rows, int64_t cols, int type, const Tensor& like, Matrix* m)
{
    if (o == Py_None) {
        m->t = make({rows, cols}, type_of(type), like);
        m->rows = rows, m->cols = cols, m->stride = cols, m->type = type;
        return true;
    }
    return m->set(o) && m->rows == rows && m->cols == cols && m->t.device() == like.device();
}

// gather(x, positions, weights or None, type code, out or None) -> rows
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix x, y;
    Slots s;
    uint64_t type;
    if (n != 5 || !x.set(a[0]) || !s.set(a[1], a[2], x.t) || s.tokens != x.rows || !whole(a[3], DCR_F16, &type) ||
        !output(a[4], s.tokens * s.k, x.cols, int(type), x.t, &y))
        Py_RETURN_NONE;
    const int rc = dcr_experts_gather(x.t.data_ptr(), x.type, x.rows, x.cols, x.stride, static_cast<const int32_t*>(s.positions), uint32_t(s.k),
                                      static_cast<const float*>(s.weights), y.t.data_ptr(), y.type, y.rows, y.stride, stream_of(x.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return a[4] == Py_None ? wrap(std::move(y.t)) : (Py_INCREF(a[4]), a[4]);
    END_HANDLE_TH_ERRORS
}

// combine(y, positions, weights or None, type code, out or None) -> sums
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix y, out;
    Slots s;
    uint64_t type;
    if (n != 5 || !y.set(a[0]) || !s.set(a[1], a[2], y.t) || s.tokens * s.k != y.rows || !whole(a[3], DCR_F16, &type) ||
        !output(a[4], s.tokens, y.cols, int(type), y.t, &out))
        Py_RETURN_NONE;
    const int rc = dcr_experts_combine(y.t.data_ptr(), y.type, y.rows, y.cols, y.stride, static_cast<const int32_t*>(s.positions),
                                       static_cast<const float*>(s.weights), s.tokens, uint32_t(s.k), out.t.data_ptr(), out.type, out.stride,
                                       stream_of(y.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return a[4] == Py_None ? wrap(std::move(out.t)) : (Py_INCREF(a[4]), a[4]);
    END_HANDLE_TH_ERRORS
}

// combine_grad(y, positions, weights, grad, out or None) -> (gradient by y, by the weights)
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Matrix y, g, out;
    Slots s;
    if (n != 5 || a[2] == Py_None || !y.set(a[0]) || !s.set(a[1], a[2], y.t) || s.tokens * s.k != y.rows || !g.set(a[3]) || g.rows != s.tokens ||
        g.cols != y.cols || !output(a[4], y.rows, y.cols, y.type, y.t, &out) || out.type != y.type)
        Py_RETURN_NONE;
    Tensor gw = make({s.tokens, s.k}, at::kFloat, y.t);
    const int rc = dcr_experts_combine_grad(y.t.data_ptr(), y.type, y.rows, y.cols, y.stride, static_cast<const int32_t*>(s.positions),
                                            static_cast<const float*>(s.weights), s.tokens, uint32_t(s.k), g.t.data_ptr(), g.type, g.stride,
                                            out.t.data_ptr(), out.stride, gw.data_ptr<float>(), stream_of(y.t));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    PyObject* first = a[4] == Py_None ? wrap(std::move(out.t)) : (Py_INCREF(a[4]), a[4]);
    return Py_BuildValue("(NN)", first, wrap(std::move(gw)));
    END_HANDLE_TH_ERRORS
}

// Contiguous tensors of one type code on the current device.
struct Tensors {
    std::vector<const Tensor*> t;
    int type = DCR_NONE;
    bool set(PyObject* list)
    {
        if (!PyList_Check(list) || PyList_GET_SIZE(list) == 0) return false;
        const Py_ssize_t n = PyList_GET_SIZE(list);
        t.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject* o = PyList_GET_ITEM(list, i);
            if (!THPVariable_Check(o)) return false;
            const Tensor& x = THPVariable_Unpack(o);
            if (!x.is_cuda() || x.layout() != at::kStrided || !x.is_contiguous() || x.get_device() != c10::cuda::current_device()) return false;
            const int c = code_of(x.scalar_type());
            if (c == DCR_NONE || (i && c != type)) return false;
            type = c;
            t.push_back(&x);
        }
        return true;
    }
};

// norm(list of gradients) -> norm
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Tensors g;
    if (n != 1 || !g.set(a[0])) Py_RETURN_NONE;
    std::vector<dcr_grad> table;
    table.reserve(g.t.size());
    for (const Tensor* x : g.t) table.push_back({x->data_ptr(), uint64_t(x->numel())});
    const Tensor& like = *g.t[0];
    Tensor work = make({int64_t(DCR_NORM_WORKSPACE)}, at::kByte, like), out = make({}, at::kFloat, like);
    const int rc = dcr_grad_norm(table.data(), uint32_t(table.size()), g.type, work.data_ptr(), out.data_ptr<float>(), stream_of(like));
    if (rc != DCR_OK) return PyLong_FromLong(rc);
    return wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// adamw(weights, grads, states (all of one kind), bits, copies or None, norm or None, step, lr, beta1, beta2, eps, weight_decay,
// max_norm, grad_scale, seed) -> DCR_OK
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Tensors w, g, c;
    if (n != 15 || !w.set(a[0]) || !g.set(a[1]) || g.t.size() != w.t.size() || !PyList_Check(a[2]) ||
        size_t(PyList_GET_SIZE(a[2])) != w.t.size() || (a[4] != Py_None && (!c.set(a[4]) || c.t.size() != w.t.size())))
        Py_RETURN_NONE;
    const Tensor& like = *w.t[0];
    uint64_t bits, step, seed;
    dcr_adamw_opts o{};
    void* np = nullptr;
    if (!whole(a[3], 32, &bits) || (bits != 8 && bits != 32) || (a[5] != Py_None && !flat(a[5], like, at::kFloat, 1, &np)) || !whole(a[6], ~0ull, &step) ||
        !number(a[7], &o.lr) || !number(a[8], &o.beta1) || !number(a[9], &o.beta2) || !number(a[10], &o.eps) || !number(a[11], &o.weight_decay) ||
        !number(a[12], &o.max_norm) || !number(a[13], &o.grad_scale) || !whole(a[14], 0xFFFFFFFFull, &seed))
        Py_RETURN_NONE;
    o.step = step, o.norm = static_cast<const float*>(np), o.seed = uint32_t(seed), o.state_bits = uint32_t(bits);
    std::vector<dcr_adamw_tensor> table;
    table.reserve(w.t.size());
    PyTypeObject* kind = Py_TYPE(PyList_GET_ITEM(a[2], 0));
    const Py_ssize_t parts = bits == 8 ? 4 : 2;
    for (size_t i = 0; i < w.t.size(); ++i) {
        PyObject* s = PyList_GET_ITEM(a[2], i);
        const int64_t size = w.t[i]->numel();
        if (Py_TYPE(s) != kind || !PyTuple_Check(s) || PyTuple_GET_SIZE(s) != parts || g.t[i]->numel() != size ||
            (a[4] != Py_None && c.t[i]->numel() != size))
            Py_RETURN_NONE;
        dcr_adamw_tensor t{};
        void *m, *v, *ms = nullptr, *vs = nullptr;
        if (bits == 32) {
            if (!flat(PyTuple_GET_ITEM(s, 0), like, at::kFloat, size, &m) || !flat(PyTuple_GET_ITEM(s, 1), like, at::kFloat, size, &v)) Py_RETURN_NONE;
        } else {
            const int64_t blocks = (size + DCR_ADAMW_BLOCK - 1) / DCR_ADAMW_BLOCK;
            auto codes = [&](PyObject* x, void** p) { return flat(x, like, at::kByte, size, p) || flat(x, like, at::kFloat8_e4m3fn, size, p); };
            if (!codes(PyTuple_GET_ITEM(s, 0), &m) || !codes(PyTuple_GET_ITEM(s, 2), &v) ||
                !flat(PyTuple_GET_ITEM(s, 1), like, at::kFloat, blocks, &ms) || !flat(PyTuple_GET_ITEM(s, 3), like, at::kFloat, blocks, &vs))
                Py_RETURN_NONE;
        }
        t.w = w.t[i]->data_ptr(), t.grad = g.t[i]->data_ptr(), t.m = m, t.v = v, t.m_scale = static_cast<float*>(ms);
        t.v_scale = static_cast<float*>(vs), t.copy = a[4] == Py_None ? nullptr : c.t[i]->data_ptr(), t.n = uint64_t(size);
        table.push_back(t);
    }
    return PyLong_FromLong(dcr_adamw(table.data(), uint32_t(table.size()), w.type, g.type, a[4] == Py_None ? int(DCR_NONE) : c.type, &o, stream_of(like)));
    END_HANDLE_TH_ERRORS
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    CALL(quantize), CALL(linear), CALL(loss),   CALL(logprobs), CALL(scores),       CALL(scores_grad), CALL(route),
    CALL(route_grad), CALL(gather), CALL(combine), CALL(combine_grad), CALL(norm), CALL(adamw),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", DCR_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
