// Python binding of the calls around dispatch and combine: checks of torch
// tensors, output allocation on the current stream, and the C entry points of
// include/ep_api.h.  Marshalling only.  A binding in C++ because a one-token
// call is a few microseconds on the GPU: through ctypes the host took 10 to
// 14 us a call.
//
// Every function takes its arguments by position and runs on the tensors'
// device and its current stream; moe.py gives names, defaults and streams.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <mutex>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/ep_api.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {       // becomes a ValueError
    using std::runtime_error::runtime_error;
};
struct PythonError {};                      // a Python error is set already
struct Failed {                             // becomes an EpError
    ep_status_t status;
    const char *what;
};

PyObject *ep_error_class = nullptr;

[[noreturn]] void refuse(const std::string &why) { throw Refused(why); }

void check(ep_status_t s, const char *what) {
    if (s != EP_SUCCESS) throw Failed{s, what};
}

// ------------------------------------------------------------- arguments

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const Tensor *optional(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}
int64_t whole(PyObject *o) {
    PyObject *i = PyNumber_Index(o);
    if (!i) throw PythonError{};
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v != 0;
}
// The place of a name among `names`.
int choice(PyObject *o, const char *what, std::initializer_list<const char *> names) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    int i = 0;
    for (const char *name : names) {
        if (s && !std::strcmp(s, name)) return i;
        ++i;
    }
    if (PyErr_Occurred()) throw PythonError{};
    std::string all;
    for (const char *name : names) all += std::string(all.empty() ? "" : ", ") + name;
    refuse(std::string(what) + ": one of " + all);
}

std::string shape_text(at::IntArrayRef shape) {
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

void on_device(const Tensor &t, c10::DeviceIndex index, const char *name) {
    if (!t.is_cuda() || t.get_device() != index)
        refuse(std::string(name) + " must be on cuda:" + std::to_string((int)index));
}
void dense(const Tensor &t, at::ScalarType type, at::IntArrayRef shape, const char *name) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        refuse(std::string(name) + " must be contiguous " + c10::toString(type) + " " + shape_text(shape));
}

// The tensors' device made current, its index and current stream.
struct Here {
    c10::DeviceIndex index;
    c10::cuda::OptionalCUDAGuard guard;
    explicit Here(const Tensor &t, const char *name) {
        if (!t.is_cuda()) refuse(std::string(name) + " must be on a CUDA device");
        index = t.get_device();
        guard.set_index(index);
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(index).stream(); }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        // at::empty fills under deterministic algorithms, if torch is told to
        if (at::globalContext().deterministicAlgorithms())
            return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, index)));
        // past the dispatcher, 0.4 us sooner; made on the current stream like any other
        return Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, index), std::nullopt));
    }
    // Bytes that no caller sees.
    Tensor scratch(size_t bytes) const {
        return Tensor(at::detail::empty_cuda({(int64_t)bytes}, at::kByte, c10::Device(c10::kCUDA, index), std::nullopt));
    }
};

// A device's error word, kept for the life of the process.
std::mutex word_lock;
Tensor *words[64];

const Tensor &error_word(c10::DeviceIndex index) {
    if (index < 0 || index >= 64) refuse("device index");
    std::lock_guard<std::mutex> hold(word_lock);
    if (!words[index]) {
        c10::cuda::CUDAGuard guard(index);
        Tensor t = at::detail::empty_cuda({1}, at::kInt, c10::Device(c10::kCUDA, index), std::nullopt);
        t.zero_();
        c10::cuda::getCurrentCUDAStream(index).synchronize();       // zero for every stream
        words[index] = new Tensor(t);
    }
    return *words[index];
}
uint32_t *error_ptr(c10::DeviceIndex index) { return static_cast<uint32_t *>(error_word(index).data_ptr()); }

template <typename... T> PyObject *pack(T &&...t) {
    PyObject *r = PyTuple_New(sizeof...(t));
    if (!r) throw PythonError{};
    Py_ssize_t i = 0;
    auto put = [&](const Tensor &x) {
        PyObject *o = nullptr;
        if (x.defined()) {
            o = THPVariable_Wrap(x);
        } else {
            o = Py_None;
            Py_INCREF(o);
        }
        if (!o) {
            Py_DECREF(r);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(r, i++, o);
    };
    (put(t), ...);
    return r;
}

// --------------------------------------------------------------- routing

struct Routing {
    ep_route_desc_t d{};
    int32_t counts[EP_MAX_WORLD];
    std::vector<int64_t> choices;        // shape of weights and indices
};

// [T][E] or [W][T][E] logits.
Routing routing(const Tensor &x, int64_t topk, PyObject *num_tokens, int score, bool renormalize, double scale,
                double balance_coef, double z_coef) {
    Routing r;
    const auto shape = x.sizes(), strides = x.strides();
    const auto type = x.scalar_type();
    if ((shape.size() != 2 && shape.size() != 3) ||
        (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat))
        refuse("logits must be bf16, fp16 or fp32 [T][E] or [W][T][E]");
    const size_t n = shape.size();
    const int64_t W = n == 3 ? shape[0] : 1, T = shape[n - 2], E = shape[n - 1];
    if (E < 1 || E > EP_MAX_ROUTE_EXPERTS)
        refuse("1 to " + std::to_string(EP_MAX_ROUTE_EXPERTS) + " experts, not " + std::to_string(E));
    if (W < 1 || W > EP_MAX_WORLD)
        refuse("1 to " + std::to_string(EP_MAX_WORLD) + " ranks, not " + std::to_string(W));
    const int64_t most = E < EP_MAX_TOPK ? E : EP_MAX_TOPK;
    if (topk < 1 || topk > most) refuse("topk must be 1 to " + std::to_string(most) + ", not " + std::to_string(topk));
    if ((strides[n - 1] != 1 && E > 1) || (strides[n - 2] < E && T > 1))
        refuse("the rows of logits must be contiguous and must not overlap");
    if (T > (int64_t)1 << 30) refuse("too many tokens");
    if (num_tokens == Py_None) {
        for (int64_t s = 0; s < W; ++s) r.counts[s] = (int32_t)T;
    } else {
        PyObject *seq = PySequence_Fast(num_tokens, "num_tokens must be a sequence of counts");
        if (!seq) throw PythonError{};
        bool fits = PySequence_Fast_GET_SIZE(seq) == W;
        try {
            for (int64_t s = 0; fits && s < W; ++s) {
                const int64_t c = whole(PySequence_Fast_GET_ITEM(seq, s));
                fits = c >= 0 && c <= T;
                r.counts[s] = (int32_t)c;
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
        Py_DECREF(seq);
        if (!fits) refuse("num_tokens must be " + std::to_string(W) + " counts of 0 to " + std::to_string(T));
    }
    r.d.world_size = (int32_t)W;
    r.d.tokens = (int32_t)T;
    r.d.num_experts = (int32_t)E;
    r.d.topk = (int32_t)topk;
    r.d.dtype = type == at::kBFloat16 ? EP_DT_BF16 : type == at::kHalf ? EP_DT_FP16 : EP_DT_FP32;
    r.d.score = score;
    r.d.renormalize = renormalize;
    r.d.scale = (float)scale;
    r.d.balance_coef = (float)balance_coef;
    r.d.z_coef = (float)z_coef;
    r.d.row_stride = strides[n - 2] > E ? strides[n - 2] : E;
    r.d.rank_stride = W > 1 ? strides[0] : 0;
    r.choices.assign(shape.begin(), shape.end() - 1);
    r.choices.push_back(topk);
    return r;
}

int score_of(PyObject *o) { return choice(o, "score", {"softmax", "sigmoid"}); }

// (logits, topk, score, renormalize, scale, bias, num_tokens)
PyObject *route(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "logits");
    Here here(x, "logits");
    Routing r = routing(x, whole(a[1]), a[6], score_of(a[2]), truth(a[3]), number(a[4]), 0, 0);
    const Tensor *bias = optional(a[5], "bias");
    if (bias) {
        on_device(*bias, here.index, "bias");
        dense(*bias, at::kFloat, {r.d.num_experts}, "bias");
    }
    Tensor w = here.empty(r.choices, at::kFloat), idx = here.empty(r.choices, at::kInt);
    if (r.d.tokens)
        check(ep_route(&r.d, x.data_ptr(), bias ? static_cast<const float *>(bias->data_ptr()) : nullptr, r.counts,
                       static_cast<float *>(w.data_ptr()), static_cast<int32_t *>(idx.data_ptr()), here.stream()),
              "ep_route");
    return pack(w, idx);
}

// (logits, topk, grad_weights, indices, grad_loss, counts, num_tokens, score,
// renormalize, scale, balance_coef, z_coef)
PyObject *route_backward(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "logits");
    Here here(x, "logits");
    Routing r = routing(x, whole(a[1]), a[6], score_of(a[7]), truth(a[8]), number(a[9]), number(a[10]), number(a[11]));
    const Tensor *gw = optional(a[2], "grad_weights"), *idx = optional(a[3], "indices");
    const Tensor *gl = optional(a[4], "grad_loss"), *counts = optional(a[5], "counts");
    if (gw) {
        if (!idx) refuse("grad_weights needs indices");
        on_device(*gw, here.index, "grad_weights");
        on_device(*idx, here.index, "indices");
        dense(*gw, at::kFloat, r.choices, "grad_weights");
        dense(*idx, at::kInt, r.choices, "indices");
    }
    if (gl) {
        if (!counts) refuse("grad_loss needs the counts of balance_loss");
        on_device(*gl, here.index, "grad_loss");
        on_device(*counts, here.index, "counts");
        if (gl->scalar_type() != at::kFloat || gl->numel() != 1)
            refuse("grad_loss must be one fp32 value on the device");
        dense(*counts, at::kInt, {r.d.num_experts}, "counts");
    }
    if (!gw && !gl) refuse("nothing to differentiate");
    Tensor out = here.empty(x.sizes(), x.scalar_type());
    if (r.d.tokens)
        check(ep_route_backward(&r.d, x.data_ptr(), gw ? static_cast<const float *>(gw->data_ptr()) : nullptr,
                                gw ? static_cast<const int32_t *>(idx->data_ptr()) : nullptr,
                                gl ? static_cast<const float *>(gl->data_ptr()) : nullptr,
                                gl ? static_cast<const int32_t *>(counts->data_ptr()) : nullptr, r.counts,
                                out.data_ptr(), error_ptr(here.index), here.stream()),
              "ep_route_backward");
    return THPVariable_Wrap(out);
}

// (logits, indices, balance_coef, z_coef, num_tokens)
PyObject *balance_loss(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "logits"), &idx = tensor(a[1], "indices");
    Here here(x, "logits");
    if (idx.dim() < 1) refuse("indices must be [...][topk]");
    Routing r = routing(x, idx.size(-1), a[4], 0, true, 1.0, number(a[2]), number(a[3]));
    on_device(idx, here.index, "indices");
    dense(idx, at::kInt, r.choices, "indices");
    const int64_t E = r.d.num_experts;
    Tensor loss = here.empty({3}, at::kFloat), counts = here.empty({E}, at::kInt), probs = here.empty({E}, at::kFloat);
    if (r.d.tokens) {
        size_t need = 0;
        check(ep_balance_loss_workspace(&r.d, &need), "ep_balance_loss_workspace");
        Tensor scratch = here.scratch(need);
        check(ep_balance_loss(&r.d, x.data_ptr(), static_cast<const int32_t *>(idx.data_ptr()), r.counts,
                              static_cast<float *>(loss.data_ptr()), static_cast<int32_t *>(counts.data_ptr()),
                              static_cast<float *>(probs.data_ptr()), scratch.data_ptr(), need,
                              error_ptr(here.index), here.stream()),
              "ep_balance_loss");
    } else {
        loss.zero_();
        counts.zero_();
        probs.zero_();
    }
    return pack(loss, counts, probs);
}

// -------------------------------------------------------------- products

struct Product {
    ep_product_desc_t d{};
    int64_t rows, wide, G;
    std::vector<int64_t> y, pre;         // shapes
};

// A tensor's rows as the kernels can read them.
ep_rows_t rows_of(const Tensor &t, const char *name) {
    const auto shape = t.sizes(), strides = t.strides();
    const size_t n = shape.size();
    const bool many = n == 3 && shape[0] > 1;
    const int64_t width = shape[n - 1];
    const int64_t rank = many ? strides[0] : 0, row = shape[n - 2] > 1 ? strides[n - 2] : (width + 7) / 8 * 8;
    if (strides[n - 1] != 1 || row < width || (row | rank) % 8 != 0 || (many && rank <= 0) ||
        reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0)
        refuse(std::string(name) + ": contiguous rows, 16-byte aligned, with strides of a multiple of 8 elements");
    return ep_rows_t{t.data_ptr(), rank, row};
}
// The same of a given tensor of a given type and shape.
ep_rows_t rows_as(const Tensor &t, c10::DeviceIndex index, at::ScalarType type, at::IntArrayRef shape,
                  const char *name) {
    on_device(t, index, name);
    if (t.scalar_type() != type || t.sizes() != shape)
        refuse(std::string(name) + " must be " + c10::toString(type) + " " + shape_text(shape));
    return t.numel() ? rows_of(t, name) : ep_rows_t{nullptr, 0, 0};
}
// And of a tensor just made.
ep_rows_t rows_new(const Tensor &t, int64_t rows, int64_t width) { return ep_rows_t{t.data_ptr(), rows * width, width}; }

Product product(const Here &here, const Tensor &x, const Tensor &weight, const Tensor *count, const Tensor *offset,
                PyObject *activation) {
    Product p;
    const auto shape = x.sizes();
    const auto type = x.scalar_type();
    if ((type != at::kBFloat16 && type != at::kHalf) || (shape.size() != 2 && shape.size() != 3))
        refuse("x must be bf16 or fp16 [rows][K] or [R][rows][K]");
    const size_t n = shape.size();
    const int64_t R = n == 3 ? shape[0] : 1, K = shape[n - 1];
    p.rows = shape[n - 2];
    const int act = choice(activation, "activation", {"none", "relu", "gelu", "silu", "swiglu"});
    if (weight.scalar_type() != type || weight.dim() != 3 || weight.size(2) != K)
        refuse("weight must be " + std::string(c10::toString(type)) + " [groups][features][" + std::to_string(K) + "]");
    on_device(weight, here.index, "weight");
    p.G = weight.size(0);
    p.wide = weight.size(1);
    const bool gated = act == EP_ACT_SWIGLU;
    const int64_t N = gated ? p.wide / 2 : p.wide;
    if (K % 8 || K == 0 || N % 8 || N == 0 || (gated && p.wide % 2) || K > 1 << 24 || N > 1 << 24)
        refuse("feature counts must be multiples of 8");
    if (R < 1 || p.G == 0 || p.G % R) refuse(std::to_string(p.G) + " groups do not divide over " + std::to_string(R) + " ranks");
    if (p.rows > (int64_t)1 << 30 || p.G > 65535) refuse("too many rows or groups");
    if (!count != !offset) refuse("count and offset come together");
    if (!count && p.G != R) refuse("without count and offset there is one group per rank");
    if (count) {
        for (const Tensor *t : {count, offset}) {
            on_device(*t, here.index, "count and offset");
            if (t->scalar_type() != at::kInt || t->numel() != p.G || !t->is_contiguous())
                refuse("count and offset must be contiguous int32 of " + std::to_string(p.G) + " groups");
        }
        p.d.d_count = static_cast<const int32_t *>(count->data_ptr());
        p.d.d_offset = static_cast<const int32_t *>(offset->data_ptr());
    }
    p.d.ranks = (int32_t)R;
    p.d.groups = (int32_t)(p.G / R);
    p.d.rows = (int32_t)p.rows;
    p.d.in_features = (int32_t)K;
    p.d.out_features = (int32_t)N;
    p.d.dtype = type == at::kBFloat16 ? EP_DT_BF16 : EP_DT_FP16;
    p.d.activation = act;
    p.d.weight = rows_of(weight, "weight");
    p.d.x = p.rows ? rows_of(x, "x") : ep_rows_t{nullptr, 0, 0};
    p.y.assign(shape.begin(), shape.end() - 1);
    p.pre = p.y;
    p.y.push_back(N);
    p.pre.push_back(p.wide);
    return p;
}

// (x, weight, count, offset, bias, activation, residual, save_pre, out)
PyObject *expert_product(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    Here here(x, "x");
    Product p = product(here, x, weight, optional(a[2], "count"), optional(a[3], "offset"), a[5]);
    const auto type = x.scalar_type();
    const Tensor *bias = optional(a[4], "bias"), *residual = optional(a[6], "residual"), *out = optional(a[8], "out");
    if (bias) {
        on_device(*bias, here.index, "bias");
        dense(*bias, type, {p.G, p.wide}, "bias");
    }
    ep_rows_t res{}, y{}, pre{};
    if (residual) res = rows_as(*residual, here.index, type, p.y, "residual");
    if (out) y = rows_as(*out, here.index, type, p.y, "out");
    Tensor made, saved;
    if (!out) {
        made = here.empty(p.y, type);
        y = rows_new(made, p.rows, p.d.out_features);
    }
    if (truth(a[7])) {
        saved = here.empty(p.pre, type);
        pre = rows_new(saved, p.rows, p.wide);
    }
    if (p.rows)
        check(ep_expert_product(&p.d, bias ? bias->data_ptr() : nullptr, &res, &y, &pre, error_ptr(here.index),
                                here.stream()),
              "ep_expert_product");
    PyObject *result = nullptr;
    if (out) {
        if (!out->is_inference()) out->unsafeGetTensorImpl()->bump_version();     // whoever saved it sees the change
        result = a[8];
        Py_INCREF(result);
    } else {
        result = THPVariable_Wrap(made);
    }
    if (!result || !saved.defined()) return result;
    PyObject *second = THPVariable_Wrap(saved), *both = second ? PyTuple_Pack(2, result, second) : nullptr;
    Py_DECREF(result);
    Py_XDECREF(second);
    return both;
}

// Rows of codes and their blocks' scales, [...][width] and [...][ceil(width / 128)].
void codes_of(const Tensor &codes, const Tensor &scales, c10::DeviceIndex index, at::IntArrayRef shape, ep_rows_t *q,
              ep_rows_t *s) {
    on_device(codes, index, "codes");
    on_device(scales, index, "scales");
    const size_t n = shape.size();
    std::vector<int64_t> blocks(shape.begin(), shape.end());
    blocks[n - 1] = (blocks[n - 1] + 127) / 128;
    if ((codes.scalar_type() != at::kFloat8_e4m3fn && codes.scalar_type() != at::kByte) || codes.sizes() != shape)
        refuse("codes must be float8_e4m3fn or uint8 " + shape_text(shape));
    if (scales.scalar_type() != at::kFloat || scales.sizes() != at::IntArrayRef(blocks))
        refuse("scales must be fp32 " + shape_text(blocks));
    if (!codes.numel()) return;
    const bool many = n == 3 && shape[0] > 1, rows = shape[n - 2] > 1;
    const auto cs = codes.strides(), ss = scales.strides();
    *q = ep_rows_t{codes.data_ptr(), many ? cs[0] : 0, rows ? cs[n - 2] : (shape[n - 1] + 7) / 8 * 8};
    *s = ep_rows_t{scales.data_ptr(), many ? ss[0] : 0, rows ? ss[n - 2] : blocks[n - 1]};
    if (cs[n - 1] != 1 || q->row_stride < shape[n - 1] || (q->row_stride | q->rank_stride) % 8 != 0 ||
        (many && q->rank_stride <= 0) || reinterpret_cast<uintptr_t>(q->ptr) % 8 != 0)
        refuse("codes: contiguous rows, 8-byte aligned, with strides of a multiple of 8");
    if ((ss[n - 1] != 1 && blocks[n - 1] > 1) || s->row_stride < blocks[n - 1] || (many && s->rank_stride <= 0))
        refuse("scales: contiguous rows that do not overlap");
}

// (grad, x, weight, count, offset, pre, activation, bias_grad, pre_scales)
PyObject *expert_product_backward(PyObject *const *a) {
    const Tensor &grad = tensor(a[0], "grad"), &x = tensor(a[1], "x"), &weight = tensor(a[2], "weight");
    Here here(x, "x");
    Product p = product(here, x, weight, optional(a[3], "count"), optional(a[4], "offset"), a[6]);
    const auto type = x.scalar_type();
    const Tensor *saved = optional(a[5], "pre");
    if (!saved && p.d.activation != EP_ACT_NONE) refuse("the gradient of this activation needs pre");
    const Tensor *saved_scales = optional(a[8], "pre_scales");
    if (saved_scales && !saved) refuse("pre_scales needs pre's codes");
    ep_rows_t g = rows_as(grad, here.index, type, p.y, "grad"), pre{}, scales{};
    if (saved_scales) codes_of(*saved, *saved_scales, here.index, p.pre, &pre, &scales);
    else if (saved) pre = rows_as(*saved, here.index, type, p.pre, "pre");
    const int64_t K = p.d.in_features;
    Tensor dx = here.empty(x.sizes(), type), dw = here.empty({p.G, p.wide, K}, type), db;
    if (truth(a[7])) db = here.empty({p.G, p.wide}, type);
    size_t need = 0;
    check(ep_expert_product_workspace(&p.d, &need), "ep_expert_product_workspace");
    Tensor scratch = here.scratch(need);
    const ep_rows_t gx = rows_new(dx, p.rows, K);
    void *bias = db.defined() ? db.data_ptr() : nullptr;
    if (saved_scales)
        check(ep_expert_product_backward_checkpoint(&p.d, &g, &pre, &scales, &gx, dw.data_ptr(), bias, scratch.data_ptr(),
                                                    need, error_ptr(here.index), here.stream()),
              "ep_expert_product_backward_checkpoint");
    else
        check(ep_expert_product_backward(&p.d, &g, &pre, &gx, dw.data_ptr(), bias, scratch.data_ptr(), need,
                                         error_ptr(here.index), here.stream()),
              "ep_expert_product_backward");
    return pack(dx, dw, db);
}

// ----------------------------------------------------------- checkpoints

ep_checkpoint_desc_t checkpoint_desc(const Here &here, at::IntArrayRef shape, const Tensor *count, const Tensor *offset,
                                     int dtype, int act) {
    ep_checkpoint_desc_t d{};
    if (shape.size() != 2 && shape.size() != 3) refuse("rows must be [rows][features] or [R][rows][features]");
    const size_t n = shape.size();
    const int64_t R = n == 3 ? shape[0] : 1, rows = shape[n - 2], F = shape[n - 1];
    if (F < 8 || F % 8 || F > 1 << 24) refuse("features must be a multiple of 8");
    if (!count != !offset) refuse("count and offset come together");
    int64_t G = R;
    if (count) {
        G = count->numel();
        for (const Tensor *t : {count, offset}) {
            on_device(*t, here.index, "count and offset");
            if (t->scalar_type() != at::kInt || t->numel() != G || !t->is_contiguous())
                refuse("count and offset must be contiguous int32 of the same number of groups");
        }
        d.d_count = static_cast<const int32_t *>(count->data_ptr());
        d.d_offset = static_cast<const int32_t *>(offset->data_ptr());
    }
    if (R < 1 || G < 1 || G % R) refuse(std::to_string(G) + " groups do not divide over " + std::to_string(R) + " ranks");
    if (rows > (int64_t)1 << 30 || G > 65535) refuse("too many rows or groups");
    d.ranks = (int32_t)R;
    d.groups = (int32_t)(G / R);
    d.rows = (int32_t)rows;
    d.features = (int32_t)F;
    d.dtype = dtype;
    d.activation = act;
    return d;
}

// (x, count, offset)
PyObject *checkpoint(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    Here here(x, "x");
    if (x.scalar_type() != at::kBFloat16 && x.scalar_type() != at::kHalf) refuse("x must be bf16 or fp16");
    const ep_checkpoint_desc_t d =
        checkpoint_desc(here, x.sizes(), optional(a[1], "count"), optional(a[2], "offset"),
                        x.scalar_type() == at::kBFloat16 ? EP_DT_BF16 : EP_DT_FP16, EP_ACT_NONE);
    std::vector<int64_t> blocks(x.sizes().begin(), x.sizes().end());
    const int64_t nb = ((int64_t)d.features + 127) / 128;
    blocks.back() = nb;
    Tensor codes = here.empty(x.sizes(), at::kFloat8_e4m3fn), scales = here.empty(blocks, at::kFloat);
    if (d.rows) {
        const ep_rows_t from = rows_of(x, "x"), q = rows_new(codes, d.rows, d.features), s = rows_new(scales, d.rows, nb);
        check(ep_checkpoint_save(&d, &from, &q, &s, here.stream()), "ep_checkpoint_save");
    }
    return pack(codes, scales);
}

// (codes, scales, count, offset, activation, dtype code)
PyObject *checkpoint_restore(PyObject *const *a) {
    const Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
    Here here(codes, "codes");
    const int act = choice(a[4], "activation", {"none", "relu", "gelu", "silu", "swiglu"});
    const int64_t dtype = whole(a[5]);
    const ep_checkpoint_desc_t d = checkpoint_desc(here, codes.sizes(), optional(a[2], "count"), optional(a[3], "offset"),
                                                   (int)dtype, act);
    if (act == EP_ACT_SWIGLU && d.features % 16) refuse("swiglu needs a multiple of 16 features");
    ep_rows_t q{}, s{};
    codes_of(codes, scales, here.index, codes.sizes(), &q, &s);
    std::vector<int64_t> shape(codes.sizes().begin(), codes.sizes().end());
    if (act == EP_ACT_SWIGLU) shape.back() /= 2;
    Tensor y = here.empty(shape, dtype == EP_DT_BF16 ? at::kBFloat16 : at::kHalf);
    if (d.rows) {
        const ep_rows_t to = rows_new(y, d.rows, shape.back());
        check(ep_checkpoint_restore(&d, &q, &s, &to, here.stream()), "ep_checkpoint_restore");
    }
    return THPVariable_Wrap(y);
}

// ------------------------------------------------------------------ norm

// Rows of a norm: [H], [rows][H] or [R][rows][H] with any strides, or dense of
// any shape.
struct Norm {
    ep_norm_desc_t d{};
    bool flat;                           // one rank of dense rows
};
ep_rows_t norm_rows(const Norm &n, const Tensor &t, const char *name) {
    const int64_t H = n.d.width;
    if (n.flat) {
        if (!t.is_contiguous()) refuse(std::string(name) + ": rows of such a shape must be dense");
        return ep_rows_t{t.data_ptr(), 0, H};
    }
    const auto shape = t.sizes(), strides = t.strides();
    const size_t k = shape.size();
    const bool many = n.d.ranks > 1;
    const ep_rows_t r{t.data_ptr(), many ? strides[0] : 0, n.d.rows > 1 ? strides[k - 2] : H};
    if ((strides[k - 1] != 1 && H > 1) || r.row_stride < H || (many && r.rank_stride <= 0))
        refuse(std::string(name) + ": rows must be contiguous and must not overlap");
    return r;
}
ep_rows_t norm_rows_as(const Norm &n, const Tensor &t, const Tensor &like, c10::DeviceIndex index, const char *name) {
    on_device(t, index, name);
    if (t.scalar_type() != like.scalar_type() || t.sizes() != like.sizes())
        refuse(std::string(name) + " must be " + c10::toString(like.scalar_type()) + " " + shape_text(like.sizes()));
    return t.numel() ? norm_rows(n, t, name) : ep_rows_t{nullptr, 0, 0};
}
Norm norm_of(const Here &here, const Tensor &x, const char *name, const Tensor &weight, double eps) {
    Norm n;
    const auto shape = x.sizes();
    const auto type = x.scalar_type(), wt = weight.scalar_type();
    if (shape.empty() || (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat))
        refuse(std::string(name) + " must be bf16, fp16 or fp32 [...][H]");
    const int64_t H = shape.back();
    if (H < 1 || H > EP_MAX_NORM_WIDTH) refuse("rows of 1 to " + std::to_string(EP_MAX_NORM_WIDTH) + " values, not " + std::to_string(H));
    on_device(weight, here.index, "weight");
    if ((wt != type && wt != at::kFloat) || weight.dim() != 1 || weight.size(0) != H || !weight.is_contiguous())
        refuse("weight must be contiguous [" + std::to_string(H) + "] of the rows' type or fp32");
    if (!(eps >= 0.0) || eps > 3e38) refuse("eps must be 0 or more");
    const int64_t rows = x.numel() / H;
    if (rows > (int64_t)1 << 30) refuse("too many rows");
    n.flat = shape.size() > 3 || (shape.size() == 3 && shape[0] > 65535) || shape.size() == 1;
    const bool many = !n.flat && shape.size() == 3 && rows;
    n.d.ranks = many ? (int32_t)shape[0] : 1;
    n.d.rows = (int32_t)(rows / n.d.ranks);
    n.d.width = (int32_t)H;
    n.d.dtype = type == at::kBFloat16 ? EP_DT_BF16 : type == at::kHalf ? EP_DT_FP16 : EP_DT_FP32;
    n.d.weight_dtype = wt == type ? n.d.dtype : EP_DT_FP32;
    n.d.eps = (float)eps;
    n.d.weight = weight.data_ptr();
    if (rows) n.d.x = norm_rows(n, x, name);
    return n;
}

// (x, weight, residual, eps, quantize)
PyObject *rms_norm(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    Here here(x, "x");
    const Norm n = norm_of(here, x, "x", weight, number(a[3]));
    const Tensor *residual = optional(a[2], "residual");
    const bool eight = truth(a[4]);
    const int64_t H = n.d.width;
    if (eight && H % 128) refuse("8-bit rows need a multiple of 128 values, not " + std::to_string(H));
    ep_rows_t res{}, total{}, scales{};
    Tensor sum, sc, y = here.empty(x.sizes(), eight ? at::kFloat8_e4m3fn : x.scalar_type());
    const ep_rows_t to{y.data_ptr(), n.d.rows * H, H};
    if (residual) {
        res = norm_rows_as(n, *residual, x, here.index, "residual");
        sum = here.empty(x.sizes(), x.scalar_type());
        total = ep_rows_t{sum.data_ptr(), n.d.rows * H, H};
    }
    if (eight) {
        std::vector<int64_t> blocks(x.sizes().begin(), x.sizes().end());
        blocks.back() = H / 128;
        sc = here.empty(blocks, at::kFloat);
        scales = ep_rows_t{sc.data_ptr(), n.d.rows * (H / 128), H / 128};
    }
    if (n.d.rows) check(ep_rms_norm(&n.d, &res, &total, &to, &scales, here.stream()), "ep_rms_norm");
    if (eight && residual) return pack(y, sc, sum);
    if (eight) return pack(y, sc);
    if (residual) return pack(y, sum);
    return THPVariable_Wrap(y);
}

// (grad, total, weight, grad_total, eps)
PyObject *rms_norm_backward(PyObject *const *a) {
    const Tensor &grad = tensor(a[0], "grad"), &total = tensor(a[1], "total"), &weight = tensor(a[2], "weight");
    Here here(total, "total");
    const Norm n = norm_of(here, total, "total", weight, number(a[4]));
    const Tensor *more = optional(a[3], "grad_total");
    const ep_rows_t g = norm_rows_as(n, grad, total, here.index, "grad");
    const ep_rows_t gt = more ? norm_rows_as(n, *more, total, here.index, "grad_total") : ep_rows_t{nullptr, 0, 0};
    const int64_t H = n.d.width;
    Tensor dx = here.empty(total.sizes(), total.scalar_type()), dw = here.empty({H}, weight.scalar_type());
    size_t need = 0;
    check(ep_rms_norm_workspace(&n.d, &need), "ep_rms_norm_workspace");
    Tensor scratch = here.scratch(need);
    const ep_rows_t to{dx.data_ptr(), n.d.rows * H, H};
    check(ep_rms_norm_backward(&n.d, &g, &gt, &to, dw.data_ptr(), scratch.data_ptr(), need,
                               error_ptr(here.index), here.stream()),
          "ep_rms_norm_backward");
    return pack(dx, dw);
}

// ------------------------------------------------------------ a few tokens

// (x, weights, indices, up, down, activation, up_bias, down_bias, residual)
PyObject *moe_few_tokens(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weights"), &idx = tensor(a[2], "indices");
    const Tensor &up = tensor(a[3], "up"), &down = tensor(a[4], "down");
    Here here(x, "x");
    const auto shape = x.sizes();
    const auto type = x.scalar_type();
    if ((type != at::kBFloat16 && type != at::kHalf) || (shape.size() != 2 && shape.size() != 3))
        refuse("x must be bf16 or fp16 [T][H] or [W][T][H]");
    const int64_t H = shape.back(), T = shape.size() == 3 ? shape[0] * shape[1] : shape[0];
    if (T > EP_MAX_FEW_TOKENS)
        refuse("at most " + std::to_string(EP_MAX_FEW_TOKENS) + " tokens, not " + std::to_string(T) +
               ": more of them go through dispatch and expert_product");
    const int act = choice(a[5], "activation", {"none", "relu", "gelu", "silu", "swiglu"});
    if (idx.dim() != x.dim()) refuse("indices must be [...][topk]");
    const int64_t k = idx.size(-1);
    if (k < 1 || k > EP_MAX_TOPK) refuse("topk must be 1 to " + std::to_string(EP_MAX_TOPK) + ", not " + std::to_string(k));
    std::vector<int64_t> choices(shape.begin(), shape.end() - 1);
    choices.push_back(k);
    on_device(w, here.index, "weights");
    on_device(idx, here.index, "indices");
    dense(w, at::kFloat, choices, "weights");
    dense(idx, at::kInt, choices, "indices");
    on_device(up, here.index, "up");
    on_device(down, here.index, "down");
    if (up.scalar_type() != type || up.dim() != 3 || up.size(2) != H)
        refuse("up must be " + std::string(c10::toString(type)) + " [experts][features][" + std::to_string(H) + "]");
    const int64_t E = up.size(0), wide = up.size(1), F = act == EP_ACT_SWIGLU ? wide / 2 : wide;
    if (E < 1 || E > EP_MAX_ROUTE_EXPERTS)
        refuse("1 to " + std::to_string(EP_MAX_ROUTE_EXPERTS) + " experts, not " + std::to_string(E));
    if (H < 8 || H % 8 || H > 1 << 20 || F < 8 || F % 8 || F > 1 << 20 || (act == EP_ACT_SWIGLU && wide % 2))
        refuse("feature counts must be multiples of 8");
    if (down.scalar_type() != type || down.sizes() != at::IntArrayRef({E, H, F}))
        refuse("down must be " + std::string(c10::toString(type)) + " " + shape_text({E, H, F}));
    const Tensor *up_bias = optional(a[6], "up_bias"), *down_bias = optional(a[7], "down_bias");
    const Tensor *residual = optional(a[8], "residual");
    if (up_bias) {
        on_device(*up_bias, here.index, "up_bias");
        dense(*up_bias, type, {E, wide}, "up_bias");
    }
    if (down_bias) {
        on_device(*down_bias, here.index, "down_bias");
        dense(*down_bias, type, {E, H}, "down_bias");
    }
    ep_few_desc_t d{};
    d.tokens = (int32_t)T;
    d.experts = (int32_t)E;
    d.topk = (int32_t)k;
    d.hidden = (int32_t)H;
    d.inner = (int32_t)F;
    d.dtype = type == at::kBFloat16 ? EP_DT_BF16 : EP_DT_FP16;
    d.activation = act;
    d.up = rows_of(up, "up");
    d.down = rows_of(down, "down");
    d.up_bias = up_bias ? up_bias->data_ptr() : nullptr;
    d.down_bias = down_bias ? down_bias->data_ptr() : nullptr;
    // the tokens of all ranks as one list
    auto tokens = [&](const Tensor &t, const char *name) {
        on_device(t, here.index, name);
        if (t.scalar_type() != type || t.sizes() != shape)
            refuse(std::string(name) + " must be " + c10::toString(type) + " " + shape_text(shape));
        if (!T) return ep_rows_t{nullptr, 0, 0};
        ep_rows_t r = rows_of(t, name);
        if (shape.size() == 3 && shape[0] > 1) {
            if (shape[1] == 1) r.row_stride = r.rank_stride;
            else if (r.rank_stride != shape[1] * r.row_stride)
                refuse(std::string(name) + ": the ranks' rows must follow each other");
            if (r.row_stride < H) refuse(std::string(name) + ": rows must not overlap");
        }
        return r;
    };
    const ep_rows_t from = tokens(x, "x"), res = residual ? tokens(*residual, "residual") : ep_rows_t{nullptr, 0, 0};
    Tensor out = here.empty(shape, type);
    if (T) {
        size_t need = 0;
        check(ep_moe_few_workspace(&d, &need), "ep_moe_few_workspace");
        Tensor scratch = here.scratch(need);
        const ep_rows_t to{out.data_ptr(), 0, H};
        check(ep_moe_few(&d, &from, static_cast<const float *>(w.data_ptr()), static_cast<const int32_t *>(idx.data_ptr()),
                         &res, &to, scratch.data_ptr(), need, error_ptr(here.index), here.stream()),
              "ep_moe_few");
    }
    return THPVariable_Wrap(out);
}

// ------------------------------------------------------------------ module

// (device index) -> the error word
PyObject *error_word_py(PyObject *const *a) { return THPVariable_Wrap(error_word((c10::DeviceIndex)whole(a[0]))); }

// (class) that is raised, with (status, what), for a refused or failed C call
PyObject *set_error_class(PyObject *const *a) {
    Py_INCREF(a[0]);
    Py_XSETREF(ep_error_class, a[0]);
    Py_RETURN_NONE;
}

// No C++ exception leaves a call.
template <PyObject *(*CALL)(PyObject *const *), Py_ssize_t ARGS>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != ARGS) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", ARGS, n);
        return nullptr;
    }
    try {
        return CALL(args);
    } catch (const PythonError &) {
    } catch (const Failed &f) {
        PyObject *e = ep_error_class ? PyObject_CallFunction(ep_error_class, "is", (int)f.status, f.what) : nullptr;
        if (e) {
            PyErr_SetObject(ep_error_class, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, f.what);
        }
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *kind = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (kind) PyErr_SetString(kind, e.what());
        Py_XDECREF(kind);
        Py_XDECREF(torch);
    } catch (const std::bad_alloc &) {
        PyErr_NoMemory();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

#define ENTRY(name, call, args) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<call, args>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    ENTRY("route", route, 7),
    ENTRY("route_backward", route_backward, 12),
    ENTRY("balance_loss", balance_loss, 5),
    ENTRY("expert_product", expert_product, 9),
    ENTRY("expert_product_backward", expert_product_backward, 9),
    ENTRY("checkpoint", checkpoint, 3),
    ENTRY("checkpoint_restore", checkpoint_restore, 6),
    ENTRY("rms_norm", rms_norm, 5),
    ENTRY("rms_norm_backward", rms_norm_backward, 5),
    ENTRY("moe_few_tokens", moe_few_tokens, 9),
    ENTRY("error_word", error_word_py, 1),
    ENTRY("set_error_class", set_error_class, 1),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe() { return PyModule_Create(&module); }
