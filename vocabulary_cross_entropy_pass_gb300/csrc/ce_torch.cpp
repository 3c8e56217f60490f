// ce_torch.cpp -- torch tensors into the C ABI for the operators around the
// cross-entropy pass (embedding, norm, logits, log-probabilities, distillation): a CPython module of fast calls.
//
// These operators run at every decoding step, where a call through ctypes took
// two to four times as long on the host (16 us for a norm) as its kernel on the
// GPU.  The module checks its arguments, allocates the outputs that are not given
// and enqueues; it holds no arithmetic.  Argument lists, semantics and documentation
// are those of the functions of the same names in vocab_ops.py and logprob_ops.py, which call
// these with every argument by position.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "../../include/ce.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // the package's CEError

// A refusal: becomes the Python exception of that type.
struct Refused {
    PyObject* type;
    std::string what;
};
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
struct PythonError {};  // one is set already

// No C++ exception leaves the module.
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

void done(int status, const char* what) {
    if (status == CE_OK) return;
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", status, what) : nullptr;
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, what);
    }
    throw PythonError{};
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
Tensor maybe(PyObject* o, const char* name) { return o == Py_None ? Tensor() : tensor(o, name); }
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return static_cast<float>(v);
}
void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("wrong number of arguments");
}

int dtype_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return CE_F32;
        case at::kBFloat16: return CE_BF16;
        case at::kHalf: return CE_F16;
        default: return -1;
    }
}
// The dtype code of the tensor an operator goes by, on the GPU.
ce_dtype cuda(const Tensor& t, const char* name) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
    const int c = dtype_code(t.scalar_type());
    if (c < 0) type_error(std::string("unsupported ") + name + " dtype " + c10::toString(t.scalar_type()));
    return static_cast<ce_dtype>(c);
}
void beside(const Tensor& t, const Tensor& like, const char* name) {
    if (t.defined() && t.device() != like.device())
        value_error(std::string(name) + " must be on " + like.device().str() + " (there is no CPU path)");
}
void matches(const Tensor& t, const Tensor& like, const char* name) {
    if (!t.defined()) return;
    beside(t, like, name);
    if (t.scalar_type() != like.scalar_type() || !t.sizes().equals(like.sizes()))
        value_error(std::string(name) + " must match in shape and dtype");
}
// A workspace is one run of memory: its bytes are counted from its elements.
void workspace(const Tensor& t, const Tensor& like) {
    beside(t, like, "workspace");
    if (t.defined() && !t.is_contiguous()) value_error("workspace must be contiguous");
}
size_t bytes(const Tensor& t) { return t.defined() ? t.numel() * t.element_size() : 0; }
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// (rows, stride between them) of a (..., H) tensor.
std::pair<int64_t, int64_t> rows(const Tensor& t, int64_t H, const char* name) {
    const auto n = t.sizes(), s = t.strides();
    if (n.empty() || n.back() != H)
        value_error(std::string(name) + " must have rows of " + std::to_string(H) + " elements");
    const int64_t N = H ? t.numel() / H : 0;
    if (t.is_contiguous() || N == 0) return {N, H};
    if (H > 1 && s.back() != 1)
        value_error(std::string("the last dimension of ") + name + " must be contiguous (call .contiguous())");
    int64_t step = -1, size = 1;
    for (int64_t d = (int64_t)n.size() - 2; d >= 0; --d) {
        if (n[d] == 1) continue;
        if (step < 0) step = s[d];
        else if (s[d] != step * size)
            value_error(std::string("the rows of ") + name + " must be evenly spaced (call .contiguous())");
        size *= n[d];
    }
    return {N, step < 0 ? H : step};
}
int64_t stride(const Tensor& t, int64_t H, const char* name) { return t.defined() ? rows(t, H, name).second : 0; }

// Where a call runs: the stream handed in (an object with a cuda_stream) or the
// current one, on the tensors' device.  A stream handed in is the current one for
// as long as the call lasts: what is allocated here comes from its memory and goes
// back there, behind the kernels that use it, and a copy of the tokens is made on it.
class Launch {
  public:
    Launch(PyObject* given, const Tensor& like)
        : on_(like.device()), before_(c10::cuda::getCurrentCUDAStream(like.device().index())),
          stream(before_.stream()) {
        if (given == Py_None) return;
        PyObject* h = PyObject_GetAttrString(given, "cuda_stream");
        if (!h) throw PythonError{};
        const unsigned long long v = PyLong_AsUnsignedLongLong(h);
        Py_DECREF(h);
        if (PyErr_Occurred()) throw PythonError{};
        stream = reinterpret_cast<void*>(static_cast<uintptr_t>(v));
        if (stream == before_.stream()) return;
        // the legacy default stream by its other name
        const auto raw = stream == cudaStreamLegacy ? nullptr : static_cast<cudaStream_t>(stream);
        other_.reset_stream(c10::cuda::getStreamFromExternal(raw, like.device().index()));
    }
    Tensor empty(at::IntArrayRef sizes, at::ScalarType t, const Tensor& like) const {
        return at::empty(sizes, like.options().dtype(t));
    }
    // Of the other stream's memory too, but for the caller: not used again there
    // before what the caller's own stream then does with it.
    Tensor output(at::IntArrayRef sizes, at::ScalarType t, const Tensor& like) const {
        Tensor r = empty(sizes, t, like);
        if (other_.current_stream()) r.record_stream(before_.unwrap());
        return r;
    }

  private:
    c10::cuda::CUDAGuard on_;
    c10::cuda::CUDAStream before_;
    c10::cuda::OptionalCUDAStreamGuard other_;

  public:
    void* stream;
};

struct Tokens {
    Tensor t;
    int64_t d0, d1, s[2];
};
Tokens tokens_of(const Tensor& t, const Tensor& like) {
    beside(t, like, "tokens");
    if (t.scalar_type() != at::kLong) type_error("tokens must be int64");
    if (t.is_contiguous()) return {t, 1, t.numel(), {0, 1}};
    if (t.dim() == 2) return {t, t.size(0), t.size(1), {t.stride(0), t.stride(1)}};
    const Tensor f = t.reshape({-1});
    return {f, 1, f.numel(), {0, f.stride(0)}};
}

// ce_embed_fwd(tokens, weight, scale, ignore_idx, out, workspace, stream)
PyObject* embed_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 7);
        const Tensor& tokens = tensor(a[0], "tokens");
        const Tensor& weight = tensor(a[1], "weight");
        Tensor out = maybe(a[4], "out");
        const Tensor ws = maybe(a[5], "workspace");
        const ce_dtype dt = cuda(weight, "weight");
        if (weight.dim() != 2) value_error("weight must be (V, H)");
        const int64_t V = weight.size(0), H = weight.size(1);
        const Launch on(a[6], weight);
        const Tokens t = tokens_of(tokens, weight);
        workspace(ws, weight);
        at::DimVector shape(tokens.sizes());
        shape.push_back(H);
        if (!out.defined()) {
            out = on.output(shape, weight.scalar_type(), weight);
        } else {
            beside(out, weight, "out");
            if (out.scalar_type() != weight.scalar_type() || !out.sizes().equals(shape))
                value_error("out must be (*tokens.shape, H) in the weight's dtype");
        }
        done(ce_embed_fwd(t.t.const_data_ptr<int64_t>(), t.d0, t.d1, t.s, weight.data_ptr(), dt, V, H,
                          stride(weight, H, "weight"), number(a[2]), integer(a[3]), out.data_ptr(),
                          stride(out, H, "out"), ptr(ws), bytes(ws), on.stream),
             "ce_embed_fwd");
        return THPVariable_Wrap(out);
    });
}

// ce_embed_bwd(grad_out, tokens, num_embeddings, scale, ignore_idx, grad_weight, accumulate, grad_dtype (code),
//              workspace, stream)
PyObject* embed_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 10);
        const Tensor& g = tensor(a[0], "grad_out");
        const Tensor& tokens = tensor(a[1], "tokens");
        const int64_t V = integer(a[2]);
        Tensor dw = maybe(a[5], "grad_weight"), ws = maybe(a[8], "workspace");
        const int accumulate = PyObject_IsTrue(a[6]);
        const ce_dtype dt = cuda(g, "grad_out");
        const int64_t nd = g.dim();
        if (nd == 0 || !g.sizes().slice(0, nd - 1).equals(tokens.sizes()))
            value_error("grad_out must be (*tokens.shape, H)");
        const int64_t H = g.size(nd - 1);
        const Launch on(a[9], g);
        const Tokens t = tokens_of(tokens, g);
        if (!dw.defined()) {
            if (accumulate) value_error("accumulate needs the grad_weight to add to");
            const int64_t code = integer(a[7]);
            if (code != CE_F32 && code != dt) type_error("grad_dtype must be float32 or grad_out's dtype");
            dw = on.output({V, H}, code == CE_F32 ? at::kFloat : g.scalar_type(), g);
        } else {
            beside(dw, g, "grad_weight");
            if (dw.dim() != 2 || dw.size(0) != V || dw.size(1) != H)
                value_error("grad_weight must be (num_embeddings, H)");
        }
        const int wdt = dtype_code(dw.scalar_type());
        if (wdt < 0 || (wdt != CE_F32 && wdt != dt)) type_error("grad_weight must be float32 or of grad_out's dtype");
        if (accumulate && wdt != CE_F32) type_error("grad_weight accumulates in float32");
        if (!ws.defined())
            ws = on.empty({(int64_t)ce_embed_bwd_workspace_bytes(t.d0 * t.d1, H, V)}, at::kByte, g);
        else
            workspace(ws, g);
        done(ce_embed_bwd(g.data_ptr(), dt, stride(g, H, "grad_out"), t.t.const_data_ptr<int64_t>(), t.d0, t.d1, t.s,
                          V, H, number(a[3]), integer(a[4]), dw.data_ptr(), (ce_dtype)wdt,
                          stride(dw, H, "grad_weight"), accumulate, ws.data_ptr(), bytes(ws), on.stream),
             "ce_embed_bwd");
        return THPVariable_Wrap(dw);
    });
}

ce_dtype weight_code(const Tensor& w, const Tensor& like, int64_t H, ce_dtype dt) {
    beside(w, like, "weight");
    const int wdt = dtype_code(w.scalar_type());
    if (wdt != dt && wdt != CE_F32) type_error("weight must be of the rows' dtype or float32");
    if (w.dim() != 1 || w.size(0) != H || !w.is_contiguous())
        value_error("weight must be a contiguous vector of H elements");
    return (ce_dtype)wdt;
}

// ce_rmsnorm_fwd(x, weight, residual, eps, out, residual_out, quant (code), group_size, scales_out, stream)
PyObject* rmsnorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 10);
        const Tensor& x = tensor(a[0], "x");
        const Tensor& w = tensor(a[1], "weight");
        const Tensor res = maybe(a[2], "residual");
        Tensor out = maybe(a[4], "out"), h = maybe(a[5], "residual_out"), scales = maybe(a[8], "scales_out");
        const ce_quant quant = (ce_quant)integer(a[6]);
        const int64_t group = integer(a[7]);
        const ce_dtype dt = cuda(x, "x");
        if (x.dim() == 0) value_error("x must be (..., H)");
        const int64_t H = x.size(-1);
        const auto [N, xs] = rows(x, H, "x");
        const ce_dtype wdt = weight_code(w, x, H, dt);
        matches(res, x, "residual");
        const Launch on(a[9], x);
        if (res.defined() && !h.defined()) h = on.output(x.sizes(), x.scalar_type(), x);
        matches(h, x, "residual_out");
        at::ScalarType ot = x.scalar_type();
        if (quant == CE_QUANT_NONE) {
            if (group || scales.defined()) value_error("group_size and scales_out go with quant");
        } else {
            ot = quant == CE_QUANT_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
            if (group != 0 && group != 32 && group != 64 && group != 128)
                value_error("group_size must be 0, 32, 64 or 128");
            const int64_t G = group == 0 ? 1 : (H + group - 1) / group;
            if (!scales.defined()) {
                scales = on.output({N, G}, at::kFloat, x);
            } else {
                beside(scales, x, "scales_out");
                if (scales.scalar_type() != at::kFloat || scales.numel() != N * G || !scales.is_contiguous())
                    value_error("scales_out must be contiguous float32 (rows, groups)");
            }
        }
        if (!out.defined()) {
            out = on.output(x.sizes(), ot, x);
        } else {
            beside(out, x, "out");
            if (out.scalar_type() != ot || !out.sizes().equals(x.sizes()))
                value_error("out must match x in shape, in x's dtype or quant's");
        }
        done(ce_rmsnorm_fwd(x.data_ptr(), ptr(res), w.data_ptr(), dt, wdt, N, H, xs, stride(res, H, "residual"),
                            number(a[3]), out.data_ptr(), stride(out, H, "out"), quant, (int)group,
                            static_cast<float*>(ptr(scales)), ptr(h), stride(h, H, "residual_out"),
                            on.stream),
             "ce_rmsnorm_fwd");
        PyObject* r = PyTuple_New(3);
        if (!r) throw PythonError{};
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(h.defined() ? h : x));
        if (scales.defined()) {
            PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(scales));
        } else {
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(r, 2, Py_None);
        }
        return r;
    });
}

// ce_rmsnorm_bwd(grad_out, h, weight, eps, grad_h, grad_x, grad_weight (True, None or tensor), workspace, stream)
PyObject* rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 9);
        const Tensor& g = tensor(a[0], "grad_out");
        const Tensor& h = tensor(a[1], "h");
        const Tensor& w = tensor(a[2], "weight");
        const Tensor dh = maybe(a[4], "grad_h");
        Tensor dx = maybe(a[5], "grad_x"), ws = maybe(a[7], "workspace"), dw;
        const ce_dtype dt = cuda(h, "h");
        if (h.dim() == 0) value_error("h must be (..., H)");
        const int64_t H = h.size(-1);
        const auto [N, hs] = rows(h, H, "h");
        const ce_dtype wdt = weight_code(w, h, H, dt);
        matches(g, h, "grad_out");
        matches(dh, h, "grad_h");
        matches(dx, h, "grad_x");
        const Launch on(a[8], h);
        if (!dx.defined()) dx = on.output(h.sizes(), h.scalar_type(), h);
        if (a[6] == Py_True) {
            dw = on.output({H}, at::kFloat, h);
        } else if (a[6] != Py_None && a[6] != Py_False) {
            dw = tensor(a[6], "grad_weight");
            beside(dw, h, "grad_weight");
            if (dw.scalar_type() != at::kFloat || dw.dim() != 1 || dw.size(0) != H || !dw.is_contiguous())
                type_error("grad_weight must be a contiguous float32 vector of H elements");
        }
        workspace(ws, h);
        if (dw.defined() && !ws.defined()) ws = on.empty({(int64_t)ce_rmsnorm_bwd_workspace_bytes(N, H)}, at::kByte, h);
        done(ce_rmsnorm_bwd(g.data_ptr(), h.data_ptr(), w.data_ptr(), ptr(dh), dt, wdt, N, H, stride(g, H, "grad_out"),
                            hs, stride(dh, H, "grad_h"), number(a[3]), dx.data_ptr(), stride(dx, H, "grad_x"),
                            static_cast<float*>(ptr(dw)), ptr(ws), bytes(ws), on.stream),
             "ce_rmsnorm_bwd");
        PyObject* r = PyTuple_New(2);
        if (!r) throw PythonError{};
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(dx));
        if (dw.defined()) {
            PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(dw));
        } else {
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(r, 1, Py_None);
        }
        return r;
    });
}

struct Dims {
    int64_t d0, d1, V, s[3];
};
Dims logits_dims(const Tensor& t, const char* name) {
    const auto n = t.sizes(), s = t.strides();
    if (n.size() != 2 && n.size() != 3) value_error(std::string(name) + " must be (dim0, dim1, V) or (N, V)");
    if (s.back() != 1 && n.back() > 1)
        value_error(std::string("the vocabulary dimension of ") + name + " must be contiguous (call .contiguous())");
    if (n.size() == 2) return {1, n[0], n[1], {n[0] * s[0], s[0], 1}};
    return {n[0], n[1], n[2], {s[0], s[1], 1}};
}

// The parameters by name, their keys kept as interned strings.
enum Param { kHistory, kHistoryLengths, kPromptLengths, kRepetition, kFrequency, kPresence, kBiasTokens, kBiasValues,
             kMask, kTemperature, kMaskValue, kParams };
const char* const kNames[kParams] = {"history", "history_lengths", "prompt_lengths", "repetition_penalty",
                                     "frequency_penalty", "presence_penalty", "bias_tokens", "bias_values", "mask",
                                     "temperature", "mask_value"};
PyObject* g_keys[kParams];

ce_logits_params logits_params(PyObject* given, int64_t N, int64_t V, const Tensor& like) {
    ce_logits_params p = {};
    p.mask_value = -INFINITY;
    PyObject* got[kParams];
    Py_ssize_t known = 0;
    for (int k = 0; k < kParams; ++k) {
        got[k] = PyDict_GetItemWithError(given, g_keys[k]);
        if (!got[k] && PyErr_Occurred()) throw PythonError{};
        if (got[k]) ++known;
        if (got[k] == Py_None) got[k] = nullptr;
    }
    if (known != PyDict_Size(given)) {
        std::string s = "unknown parameter; known are:";
        for (const char* k : kNames) s += std::string(" ") + k;
        type_error(s);
    }
    auto per_row = [&](int k, at::ScalarType want) -> const void* {
        if (!got[k]) return nullptr;
        const Tensor& t = tensor(got[k], kNames[k]);
        if (t.scalar_type() != want || t.device() != like.device() || t.numel() != N || !t.is_contiguous())
            type_error(std::string(kNames[k]) + " must be a contiguous " + c10::toString(want) +
                       " CUDA tensor with one value per row");
        return t.data_ptr();
    };
    auto list = [&](int k, at::ScalarType want, int64_t* step, int64_t* entries) -> const void* {
        const Tensor& t = tensor(got[k], kNames[k]);
        if (t.scalar_type() != want || t.device() != like.device() || t.dim() != 2 || t.size(0) != N)
            type_error(std::string(kNames[k]) + " must be " + c10::toString(want) +
                       " on the logits' device, one row of entries per row of logits");
        if (t.size(1) > 1 && t.stride(1) != 1)
            value_error(std::string("the entries of ") + kNames[k] + " must be contiguous (call .contiguous())");
        *entries = t.size(1);
        *step = t.is_contiguous() ? t.size(1) : t.stride(0);
        return t.data_ptr();
    };
    p.history_lengths = static_cast<const int64_t*>(per_row(kHistoryLengths, at::kLong));
    p.prompt_lengths = static_cast<const int64_t*>(per_row(kPromptLengths, at::kLong));
    p.repetition_penalty = static_cast<const float*>(per_row(kRepetition, at::kFloat));
    p.frequency_penalty = static_cast<const float*>(per_row(kFrequency, at::kFloat));
    p.presence_penalty = static_cast<const float*>(per_row(kPresence, at::kFloat));
    p.temperature = static_cast<const float*>(per_row(kTemperature, at::kFloat));
    if (got[kHistory])
        p.history = static_cast<const int64_t*>(list(kHistory, at::kLong, &p.history_stride, &p.history_max));
    else if (got[kHistoryLengths] || got[kPromptLengths] || got[kRepetition] || got[kFrequency] || got[kPresence])
        value_error("the penalties and lengths need a history");
    if (!got[kBiasTokens] != !got[kBiasValues]) value_error("bias_tokens and bias_values go together");
    if (got[kBiasTokens]) {
        int64_t m = 0;
        p.bias_tokens = static_cast<const int64_t*>(list(kBiasTokens, at::kLong, &p.bias_tokens_stride, &p.bias_max));
        p.bias_values = static_cast<const float*>(list(kBiasValues, at::kFloat, &p.bias_values_stride, &m));
        if (m != p.bias_max) value_error("bias_tokens and bias_values must have the same shape");
    }
    if (got[kMask]) {
        const Tensor& m = tensor(got[kMask], "mask");
        const int64_t words = (V + 31) / 32;
        if (m.scalar_type() != at::kInt || m.device() != like.device() || m.dim() < 1 || m.size(-1) != words)
            type_error("mask must be int32 on the logits' device with " + std::to_string(words) + " words per row");
        if (m.dim() > 2 || (m.dim() == 2 && m.size(0) != 1 && m.size(0) != N) || (words > 1 && m.stride(-1) != 1))
            value_error("mask must be (words,) for all rows or (N, words), its words contiguous");
        p.mask = static_cast<const int32_t*>(m.data_ptr());
        p.mask_stride = m.dim() == 2 && m.size(0) == N && N > 1 ? m.stride(0) : 0;
    }
    if (got[kMaskValue]) p.mask_value = number(got[kMaskValue]);
    return p;
}

Tensor logits_workspace(const Launch& on, const Tensor& given, const ce_logits_params& p, const Dims& d, ce_dtype dt,
                        const Tensor& like) {
    if (given.defined()) {
        workspace(given, like);
        return given;
    }
    const size_t need =
        p.history_max || p.bias_max ? ce_logits_workspace_bytes(d.d0 * d.d1, d.V, dt, p.history_max, p.bias_max) : 0;
    return need ? on.empty({(int64_t)need}, at::kByte, like) : Tensor();
}

// ce_logits_process(logits, out, workspace, stream, params)
PyObject* logits_process(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 5);
        const Tensor& x = tensor(a[0], "logits");
        Tensor out = maybe(a[1], "out");
        const ce_dtype dt = cuda(x, "logits");
        const Dims d = logits_dims(x, "logits");
        const Launch on(a[3], x);
        const ce_logits_params p = logits_params(a[4], d.d0 * d.d1, d.V, x);
        matches(out, x, "out");
        if (!out.defined()) out = on.output(x.sizes(), x.scalar_type(), x);
        const Dims o = logits_dims(out, "out");
        const Tensor ws = logits_workspace(on, maybe(a[2], "workspace"), p, d, dt, x);
        done(ce_logits_process(x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, &p, out.data_ptr(), o.s, ptr(ws), bytes(ws),
                               on.stream),
             "ce_logits_process");
        return THPVariable_Wrap(out);
    });
}

// ce_logits_process_bwd(grad_out, logits, grad, workspace, stream, params)
PyObject* logits_process_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 6);
        const Tensor& g = tensor(a[0], "grad_out");
        const Tensor& x = tensor(a[1], "logits");
        Tensor out = maybe(a[2], "grad");
        const ce_dtype dt = cuda(x, "logits");
        const Dims d = logits_dims(x, "logits");
        matches(g, x, "grad_out");
        const Dims gd = logits_dims(g, "grad_out");
        const Launch on(a[4], x);
        const ce_logits_params p = logits_params(a[5], d.d0 * d.d1, d.V, x);
        matches(out, x, "grad");
        if (!out.defined()) out = on.output(x.sizes(), x.scalar_type(), x);
        const Dims o = logits_dims(out, "grad");
        const Tensor ws = logits_workspace(on, maybe(a[3], "workspace"), p, d, dt, x);
        done(ce_logits_process_bwd(g.data_ptr(), gd.s, x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, &p, out.data_ptr(), o.s,
                                   ptr(ws), bytes(ws), on.stream),
             "ce_logits_process_bwd");
        return THPVariable_Wrap(out);
    });
}

// A list of tokens for each row of logits: (rows), one token each, or (rows, n).
struct Listed {
    Tensor t;
    int64_t n = 0, s[3] = {0, 0, 0};
};
Listed listed_of(const Tensor& t, const Tensor& logits, const char* name) {
    Listed l;
    if (!t.defined()) return l;
    beside(t, logits, name);
    const int64_t lead = logits.dim() - 1;
    if ((t.dim() != lead && t.dim() != lead + 1) || !t.sizes().slice(0, lead).equals(logits.sizes().slice(0, lead)))
        value_error(std::string(name) + " must be one value, or a list of them, for each row of logits");
    l.t = t;
    const auto st = t.strides();
    l.n = t.dim() == lead ? 1 : t.size(lead);
    l.s[2] = t.dim() == lead ? 0 : st[lead];
    l.s[1] = st[lead - 1];
    l.s[0] = lead == 2 ? st[0] : 0;
    return l;
}
const int64_t* token_ptr(const Listed& l) {
    if (!l.t.defined()) return nullptr;
    if (l.t.scalar_type() != at::kLong) type_error("tokens must be int64");
    return l.t.const_data_ptr<int64_t>();
}
// A float32 tensor of `numel` values, in order.
float* floats(const Tensor& t, const Tensor& like, int64_t numel, const char* name) {
    if (!t.defined()) return nullptr;
    beside(t, like, name);
    if (t.scalar_type() != at::kFloat || t.numel() != numel || !t.is_contiguous())
        type_error(std::string(name) + " must be contiguous float32 with " + std::to_string(numel) + " values");
    return static_cast<float*>(t.data_ptr());
}
int64_t* count_ptr(const Tensor& t, const Tensor& like, const char* name) {
    if (!t.defined()) return nullptr;
    beside(t, like, name);
    if (t.scalar_type() != at::kLong || t.numel() != 1) type_error(std::string(name) + " must be one int64");
    return static_cast<int64_t*>(t.data_ptr());
}
void put(PyObject* tuple, int k, const Tensor& t) {
    PyObject* o = Py_None;
    if (t.defined()) {
        o = THPVariable_Wrap(t);
        if (!o) throw PythonError{};
    } else {
        Py_INCREF(o);
    }
    PyTuple_SET_ITEM(tuple, k, o);
}
struct Tuple {  // released where it was not handed out
    PyObject* o;
    explicit Tuple(Py_ssize_t n) : o(PyTuple_New(n)) {
        if (!o) throw PythonError{};
    }
    ~Tuple() { Py_XDECREF(o); }
    PyObject* out() {
        PyObject* r = o;
        o = nullptr;
        return r;
    }
};
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v != 0;
}

// ce_logprobs_fwd(logits, tokens, top_k, entropy, stats, ignore_idx, workspace, stream)
PyObject* logprobs_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 8);
        const Tensor& x = tensor(a[0], "logits");
        const ce_dtype dt = cuda(x, "logits");
        const Dims d = logits_dims(x, "logits");
        const Listed l = listed_of(maybe(a[1], "tokens"), x, "tokens");
        const int64_t* tokens = token_ptr(l);
        const int64_t top_k = integer(a[2]), N = d.d0 * d.d1;
        const bool want_entropy = truth(a[3]), want_stats = truth(a[4]);
        Tensor ws = maybe(a[6], "workspace");
        workspace(ws, x);
        if (top_k < 0 || top_k > 256 || top_k > d.V) value_error("top_k must be between 0 and min(256, V)");
        if (l.n == 0 && top_k == 0 && !want_entropy && !want_stats)
            value_error("nothing asked for: tokens, top_k, entropy or stats");
        const Launch on(a[7], x);
        Tensor lp, ent, top, top_lp, stats;
        at::DimVector shape(x.sizes().slice(0, x.dim() - 1));
        if (l.t.defined()) lp = on.output(l.t.sizes(), at::kFloat, x);
        if (want_entropy) ent = on.output(shape, at::kFloat, x);
        if (want_stats) stats = on.output({N, 4}, at::kFloat, x);
        if (top_k) {
            shape.push_back(top_k);
            top = on.output(shape, at::kLong, x);
            top_lp = on.output(shape, at::kFloat, x);
        }
        if (!ws.defined()) ws = on.empty({(int64_t)ce_logprobs_workspace_bytes(N, d.V, dt, (int)top_k)}, at::kByte, x);
        done(ce_logprobs_fwd(x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, tokens, l.s, l.n, integer(a[5]),
                             static_cast<float*>(ptr(lp)), static_cast<float*>(ptr(ent)), (int)top_k,
                             static_cast<int64_t*>(ptr(top)), static_cast<float*>(ptr(top_lp)),
                             static_cast<float*>(ptr(stats)), ptr(ws), bytes(ws), on.stream),
             "ce_logprobs_fwd");
        Tuple r(5);
        put(r.o, 0, lp);
        put(r.o, 1, ent);
        put(r.o, 2, top);
        put(r.o, 3, top_lp);
        put(r.o, 4, stats);
        return r.out();
    });
}

// The gradient's tensor, allocated when none is given.
Tensor grad_of(const Tensor& given, const Tensor& x, const Launch& on) {
    matches(given, x, "grad");
    return given.defined() ? given : on.output(x.sizes(), x.scalar_type(), x);
}

// ce_logprobs_bwd(logits, stats, tokens, grad_logprobs, grad_entropy, ignore_idx, grad, stream)
PyObject* logprobs_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 8);
        const Tensor& x = tensor(a[0], "logits");
        const ce_dtype dt = cuda(x, "logits");
        const Dims d = logits_dims(x, "logits");
        const int64_t N = d.d0 * d.d1;
        const Tensor stats = tensor(a[1], "stats");
        const Listed l = listed_of(maybe(a[2], "tokens"), x, "tokens");
        const int64_t* tokens = token_ptr(l);
        const Tensor gl = maybe(a[3], "grad_logprobs"), ge = maybe(a[4], "grad_entropy");
        if (gl.defined() && l.n == 0) value_error("grad_logprobs goes with tokens");
        const float* st = floats(stats, x, N * 4, "stats");
        const float* g = floats(gl, x, N * l.n, "grad_logprobs");
        const float* h = floats(ge, x, N, "grad_entropy");
        const Launch on(a[7], x);
        const Tensor grad = grad_of(maybe(a[6], "grad"), x, on);
        const Dims o = logits_dims(grad, "grad");
        done(ce_logprobs_bwd(x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, tokens, l.s, l.n, integer(a[5]), st, g, h,
                             grad.data_ptr(), o.s, on.stream),
             "ce_logprobs_bwd");
        return THPVariable_Wrap(grad);
    });
}

// The teacher's tokens and logits.
struct Taught {
    Listed tokens, logits;
    const int64_t* t;
    ce_dtype dt;
};
Taught taught(PyObject* tokens, PyObject* logits, const Tensor& x) {
    Taught r;
    r.tokens = listed_of(tensor(tokens, "teacher_tokens"), x, "teacher_tokens");
    r.logits = listed_of(tensor(logits, "teacher_logits"), x, "teacher_logits");
    r.t = token_ptr(r.tokens);
    r.dt = cuda(r.logits.t, "teacher_logits");
    if (!r.tokens.t.sizes().equals(r.logits.t.sizes()))
        value_error("teacher_tokens and teacher_logits must have the same shape");
    return r;
}

// ce_distill_fwd(_bwd)(logits, teacher_tokens, teacher_logits, temperature, normalize, ignore_idx, reduce_loss, dloss,
//                      grad (False: forward only, None, or a tensor), stats, loss_out, n_non_ignore_out, workspace,
//                      stream)
PyObject* distill_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 14);
        const Tensor& x = tensor(a[0], "logits");
        const ce_dtype dt = cuda(x, "logits");
        const Dims d = logits_dims(x, "logits");
        const int64_t N = d.d0 * d.d1, ignore = integer(a[5]);
        const Taught t = taught(a[1], a[2], x);
        const float tau = number(a[3]);
        const int normalize = truth(a[4]), reduce = truth(a[6]);
        const bool backward = a[8] != Py_False, want_stats = truth(a[9]);
        Tensor loss = maybe(a[10], "loss_out"), ws = maybe(a[12], "workspace"), grad, stats;
        const Tensor dloss = maybe(a[7], "dloss");
        const float* g = floats(dloss, x, reduce ? 1 : N, "dloss");
        floats(loss, x, reduce ? 1 : N, "loss_out");
        int64_t* count = count_ptr(maybe(a[11], "n_non_ignore_out"), x, "n_non_ignore_out");
        workspace(ws, x);
        const Launch on(a[13], x);
        if (!loss.defined()) loss = on.output({reduce ? 1 : N}, at::kFloat, x);
        if (!ws.defined()) ws = on.empty({(int64_t)ce_distill_workspace_bytes(N, d.V, dt)}, at::kByte, x);
        int status;
        if (backward) {
            grad = grad_of(maybe(a[8], "grad"), x, on);
            const Dims o = logits_dims(grad, "grad");
            status = ce_distill_fwd_bwd(x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, t.t, t.tokens.s, t.logits.t.data_ptr(),
                                        t.dt, t.logits.s, t.tokens.n, tau, normalize, ignore, reduce, g,
                                        static_cast<float*>(loss.data_ptr()), grad.data_ptr(), o.s, count, ptr(ws),
                                        bytes(ws), on.stream);
        } else {
            if (want_stats) stats = on.output({N, 4}, at::kFloat, x);
            status = ce_distill_fwd(x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, t.t, t.tokens.s, t.logits.t.data_ptr(),
                                    t.dt, t.logits.s, t.tokens.n, tau, normalize, ignore, reduce,
                                    static_cast<float*>(loss.data_ptr()), static_cast<float*>(ptr(stats)), count,
                                    ptr(ws), bytes(ws), on.stream);
        }
        done(status, backward ? "ce_distill_fwd_bwd" : "ce_distill_fwd");
        Tuple r(2);
        put(r.o, 0, loss);
        put(r.o, 1, backward ? grad : stats);
        return r.out();
    });
}

// ce_distill_bwd(logits, teacher_tokens, teacher_logits, stats, temperature, normalize, ignore_idx, reduce_loss, dloss,
//                n_non_ignore, grad, stream)
PyObject* distill_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 12);
        const Tensor& x = tensor(a[0], "logits");
        const ce_dtype dt = cuda(x, "logits");
        const Dims d = logits_dims(x, "logits");
        const int64_t N = d.d0 * d.d1;
        const Taught t = taught(a[1], a[2], x);
        const float* stats = floats(tensor(a[3], "stats"), x, N * 4, "stats");
        const int reduce = truth(a[7]);
        const Tensor dloss = maybe(a[8], "dloss");
        const float* g = floats(dloss, x, reduce ? 1 : N, "dloss");
        const int64_t* count = count_ptr(maybe(a[9], "n_non_ignore"), x, "n_non_ignore");
        if (reduce && !count) value_error("reduce_loss needs the forward's n_non_ignore");
        const Launch on(a[11], x);
        const Tensor grad = grad_of(maybe(a[10], "grad"), x, on);
        const Dims o = logits_dims(grad, "grad");
        done(ce_distill_bwd(x.data_ptr(), dt, d.d0, d.d1, d.V, d.s, t.t, t.tokens.s, t.logits.t.data_ptr(), t.dt,
                            t.logits.s, t.tokens.n, number(a[4]), truth(a[5]), integer(a[6]), reduce, stats, g, count,
                            grad.data_ptr(), o.s, on.stream),
             "ce_distill_bwd");
        return THPVariable_Wrap(grad);
    });
}

// row_stride(t): the stride between a tensor's rows, ValueError where they are not evenly spaced.
PyObject* row_stride(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arity(n, 1);
        const Tensor& t = tensor(a[0], "tensor");
        if (t.dim() == 0) value_error("tensor must have rows");
        return PyLong_FromLongLong(rows(t, t.size(-1), "tensor").second);
    });
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"embed_fwd", FAST(embed_fwd), "ce_embed_fwd"},
                         {"embed_bwd", FAST(embed_bwd), "ce_embed_bwd"},
                         {"rmsnorm_fwd", FAST(rmsnorm_fwd), "ce_rmsnorm_fwd"},
                         {"rmsnorm_bwd", FAST(rmsnorm_bwd), "ce_rmsnorm_bwd"},
                         {"logits_process", FAST(logits_process), "ce_logits_process"},
                         {"logits_process_bwd", FAST(logits_process_bwd), "ce_logits_process_bwd"},
                         {"logprobs_fwd", FAST(logprobs_fwd), "ce_logprobs_fwd"},
                         {"logprobs_bwd", FAST(logprobs_bwd), "ce_logprobs_bwd"},
                         {"distill_fwd", FAST(distill_fwd), "ce_distill_fwd and ce_distill_fwd_bwd"},
                         {"distill_bwd", FAST(distill_bwd), "ce_distill_bwd"},
                         {"row_stride", FAST(row_stride), "stride between a tensor's rows"},
                         {"set_error", set_error, METH_O, "the class of library errors"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gbce_torch", "torch tensors into libgbce", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gbce_torch() {
    for (int k = 0; k < kParams; ++k)
        if (!(g_keys[k] = PyUnicode_InternFromString(kNames[k]))) return nullptr;
    return PyModule_Create(&module);
}
