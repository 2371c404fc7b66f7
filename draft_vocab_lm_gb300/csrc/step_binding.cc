// Python entry points of the drafting step's operators: the module _step.
//
// A step of a few rows takes 2 to 8 us on the GPU, so what the host spends on
// a call counts as much as the kernel.  Checking the tensors and marshalling
// the arguments in Python took 3 to 9 us of it (7.2 us per call for the norm
// of one row, 12.8 for a small reordering); reading the tensors' fields here
// takes a few hundred nanoseconds.  The module checks and marshals only:
// every step of the computation runs behind the C ABI.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>
#include <vector>

#include "dvl.h"

// Weak: a stand-in for the library that lacks them still links with this module.
// (The package asks its own library for every entry point before it loads this, so
// one that lacks them is refused there.)
extern "C" {
__attribute__((weak)) dvl_status dvl_qk_norm_rope(const dvl_qk *args, void *stream);
__attribute__((weak)) dvl_status dvl_cache_keep(const dvl_kv_cache *, const int32_t *, int64_t, int32_t,
                                                const int32_t *, const int32_t *, const int32_t *, int64_t,
                                                const int32_t *, int32_t, int32_t, int32_t *, void *);
}

namespace {

using at::Tensor;

// A refusal of an argument: a Python ValueError.
struct Refused {
    std::string what;
};
// A Python exception is set.
struct Raised {};

void need(bool ok, const char *what)
{
    if (!ok)
        throw Refused{what};
}

// ---- arguments ----------------------------------------------------------

constexpr int kMost = 16;

struct Signature {
    const char *name;
    int positional;  // the first ones may be given by position
    int count;
    const char *names[kMost];
    PyObject *interned[kMost];
};

void intern(Signature &s)
{
    for (int i = 0; i < s.count; ++i)
        s.interned[i] = PyUnicode_InternFromString(s.names[i]);
}

// Values by the signature's order, nullptr for absent ones and None.
struct Args {
    PyObject *v[kMost] = {};

    Args(const Signature &s, PyObject *const *args, Py_ssize_t n, PyObject *kw)
    {
        if (n > s.positional) {
            PyErr_Format(PyExc_TypeError, "%s() takes %d positional arguments but %zd were given",
                         s.name, s.positional, n);
            throw Raised{};
        }
        for (Py_ssize_t i = 0; i < n; ++i)
            v[i] = args[i];
        const Py_ssize_t nk = kw ? PyTuple_GET_SIZE(kw) : 0;
        for (Py_ssize_t k = 0; k < nk; ++k) {
            PyObject *key = PyTuple_GET_ITEM(kw, k);
            int at = -1;
            for (int i = 0; i < s.count && at < 0; ++i)
                if (key == s.interned[i])
                    at = i;
            for (int i = 0; i < s.count && at < 0; ++i)
                if (PyUnicode_Compare(key, s.interned[i]) == 0)
                    at = i;
            if (at < 0 || v[at]) {
                PyErr_Format(PyExc_TypeError,
                             at < 0 ? "%s() got an unexpected keyword argument '%U'"
                                    : "%s() got multiple values for argument '%U'",
                             s.name, key);
                throw Raised{};
            }
            v[at] = args[n + k];
        }
        for (PyObject *&x : v)
            if (x == Py_None)
                x = nullptr;
    }

    const Tensor *tensor(int i, const char *what) const
    {
        if (!v[i])
            return nullptr;
        if (!THPVariable_Check(v[i]))
            throw Refused{std::string(what) + " must be a tensor"};
        return &THPVariable_Unpack(v[i]);
    }
    const Tensor &required(int i, const char *what) const
    {
        const Tensor *t = tensor(i, what);
        if (!t)
            throw Refused{std::string(what) + " must be a tensor"};
        return *t;
    }
    int64_t integer(int i, int64_t absent) const
    {
        if (!v[i])
            return absent;
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred())
            throw Raised{};
        return x;
    }
    double number(int i, double absent) const
    {
        if (!v[i])
            return absent;
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred())
            throw Raised{};
        return x;
    }
    // An absent truth value keeps its default; None counts as absent.
    bool truth(int i, bool absent) const
    {
        const int x = v[i] ? PyObject_IsTrue(v[i]) : absent;
        if (x < 0)
            throw Raised{};
        return x != 0;
    }
};

// ---- tensors ------------------------------------------------------------

int cuda_device(const Tensor &t) { return t.is_cuda() ? (int)t.get_device() : -1; }

// The tensors' device as the current one for a call's duration: the library's
// kernels, grids and default stream are the current device's.  (Asking for the
// current device takes 0.1 us of a call's 2.7, so where there is only one it
// is not asked.)
class OnDevice {
    const int was_, dev_;

    static int enter(int dev)
    {
        static const bool several = c10::cuda::device_count() > 1;
        return several ? c10::cuda::ExchangeDevice((c10::DeviceIndex)dev) : dev;
    }

public:
    explicit OnDevice(int dev) : was_(enter(dev)), dev_(dev) {}
    ~OnDevice()
    {
        if (was_ != dev_)
            (void)c10::cuda::SetDevice((c10::DeviceIndex)was_);
    }
    OnDevice(const OnDevice &) = delete;
    OnDevice &operator=(const OnDevice &) = delete;
};

// The stream's handle: a torch stream, or an integer handle.
cudaStream_t handle_of(PyObject *stream)
{
    PyObject *handle = PyObject_GetAttrString(stream, "cuda_stream");
    if (!handle) {
        PyErr_Clear();
        handle = Py_NewRef(stream);
    }
    void *p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (PyErr_Occurred())
        throw Raised{};
    return static_cast<cudaStream_t>(p);
}

// Where a call runs: its tensors' device, and the given stream or the device's
// current one.  What the call makes for itself on another stream than the
// current one is that stream's, so that its memory comes from and returns to
// work in that stream's order; results are known to the current stream too,
// where the caller's next use of them is, and outlive it.
class Place {
    const OnDevice on_;
    const c10::cuda::CUDAStream current_;
    const cudaStream_t stream_;
    const bool foreign_;

public:
    Place(PyObject *stream, int dev)
        : on_(dev), current_(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev)),
          stream_(stream ? handle_of(stream) : current_.stream()),
          foreign_(stream && stream_ != current_.stream())
    {
    }
    void *stream() const { return stream_; }
    Tensor make(at::IntArrayRef shape, at::ScalarType type, const Tensor &like) const
    {
        const auto options = at::TensorOptions().dtype(type).device(like.device());
        if (!foreign_)
            return at::empty(shape, options);
        struct Back {
            const c10::cuda::CUDAStream &to;
            ~Back() { c10::cuda::setCurrentCUDAStream(to); }
        } back{current_};
        c10::cuda::setCurrentCUDAStream(
            c10::cuda::getStreamFromExternal(stream_, current_.device_index()));
        Tensor t = at::empty(shape, options);
        t.record_stream(current_.unwrap());
        return t;
    }
};

std::string shape_text(at::IntArrayRef shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i)
        s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

// Data pointer of a contiguous tensor of this shape and type on this device.
void *flat(const Tensor &t, at::IntArrayRef shape, at::ScalarType type, int dev, const char *name)
{
    if (cuda_device(t) != dev || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        throw Refused{std::string(name) + " must be a contiguous CUDA " + at::toString(type) +
                      " tensor of shape " + shape_text(shape) + " on the inputs' device"};
    return t.data_ptr();
}

struct Rows {
    void *p = nullptr;
    int64_t stride = 0;
};
// A 2-D tensor of this shape whose rows are contiguous.
Rows rows_of(const Tensor &t, at::IntArrayRef shape, bool type_ok, int dev, const char *name)
{
    if (cuda_device(t) != dev || !type_ok || t.sizes() != shape ||
        (t.stride(1) != 1 && shape[1] != 1))
        throw Refused{std::string(name) + " has another type or shape than x's " +
                      shape_text(shape) + ", rows that are not contiguous, or another device"};
    return {t.data_ptr(), t.stride(0)};
}

PyObject *wrap(const Tensor *given, PyObject *object, const Tensor &made)
{
    return given ? Py_NewRef(object) : THPVariable_Wrap(made);
}

// ---- results ------------------------------------------------------------

// The package's own check() raises its DvlError.
void check(const char *fn, dvl_status st)
{
    if (st == DVL_OK)
        return;
    PyObject *m = PyImport_ImportModule("draft_vocab_lm_gb300._native");
    PyObject *r = m ? PyObject_CallMethod(m, "check", "si", fn, (int)st) : nullptr;
    Py_XDECREF(r);
    Py_XDECREF(m);
    throw Raised{};
}

template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// What a KVCache object holds (step.py): the address of its C struct and its
// device.
const dvl_kv_cache *cache_of(PyObject *cache, int *dev)
{
    static PyObject *address = PyUnicode_InternFromString("_address"),
                    *device = PyUnicode_InternFromString("_dev");
    PyObject *a = PyObject_GetAttr(cache, address), *d = a ? PyObject_GetAttr(cache, device) : nullptr;
    const dvl_kv_cache *c =
        d ? static_cast<const dvl_kv_cache *>(PyLong_AsVoidPtr(a)) : nullptr;
    if (d)
        *dev = (int)PyLong_AsLong(d);
    Py_XDECREF(a);
    Py_XDECREF(d);
    if (!c || PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{"cache must be a KVCache"};
    }
    return c;
}

// A workspace made by the package's own function.
PyObject *new_workspace(const char *fn, PyObject *args, PyObject *stream)
{
    PyObject *m = PyImport_ImportModule("draft_vocab_lm_gb300.step");
    PyObject *f = m ? PyObject_GetAttrString(m, fn) : nullptr;
    PyObject *kw = f ? Py_BuildValue("{s:O}", "stream", stream ? stream : Py_None) : nullptr;
    PyObject *ws = kw && args ? PyObject_Call(f, args, kw) : nullptr;
    Py_XDECREF(kw);
    Py_XDECREF(f);
    Py_XDECREF(m);
    Py_XDECREF(args);
    if (!ws)
        throw Raised{};
    return ws;
}

struct Workspace {
    PyObject *owned = nullptr;
    void *p = nullptr;
    size_t bytes = 0;
    void set(const Tensor &t, int dev)
    {
        need(cuda_device(t) == dev && t.is_contiguous(), "ws must be a contiguous tensor on the inputs' device");
        p = t.data_ptr();
        bytes = t.numel() * t.element_size();
    }
    ~Workspace() { Py_XDECREF(owned); }
};

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

// ---- add_rmsnorm --------------------------------------------------------

Signature norm_sig = {"add_rmsnorm", 3, 11,
                      {"x", "weight", "residual", "eps", "bf16", "fp8_group", "out", "residual_out",
                       "codes", "scales", "stream"},
                      {}};

PyObject *add_rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw)
{
    return guarded([&]() -> PyObject * {
        const Args a(norm_sig, args, n, kw);
        const Tensor &x = a.required(0, "x"), &weight = a.required(1, "weight");
        const int dev = cuda_device(x);
        need(dev >= 0 && x.dim() == 2 && weight.dim() == 1, "x must be a CUDA [rows][K] tensor, weight [K]");
        const Place on(a.v[10], dev);
        const int64_t shape[2] = {x.size(0), x.size(1)};
        const int64_t K = shape[1];
        dvl_norm p = {};
        need(K <= INT32_MAX, "x is too wide");
        p.rows = shape[0];
        p.K = (int32_t)K;
        p.eps = (float)a.number(3, 1e-6);
        Rows r = rows_of(x, shape, x.scalar_type() == kBf16, dev, "x");
        p.x = r.p;
        p.x_stride = r.stride;
        p.weight = flat(weight, {K}, kBf16, dev, "weight");

        const Tensor *residual = a.tensor(2, "residual"), *residual_out = a.tensor(7, "residual_out");
        const Tensor *out = a.tensor(6, "out"), *codes = a.tensor(8, "codes"),
                     *scales = a.tensor(9, "scales");
        Tensor new_residual, new_out, new_codes, new_scales;
        p.residual_dtype = DVL_BF16;
        if (residual) {
            const auto type = residual->scalar_type();
            r = rows_of(*residual, shape, type == kBf16 || type == kF32, dev, "residual");
            p.residual = r.p;
            p.residual_stride = r.stride;
            p.residual_dtype = type == kF32 ? DVL_F32 : DVL_BF16;
            if (!residual_out)
                new_residual = on.make(shape, type, x);
            const Tensor &to = residual_out ? *residual_out : new_residual;
            r = rows_of(to, shape, to.scalar_type() == type, dev, "residual_out");
            p.residual_out = r.p;
            p.residual_out_stride = r.stride;
        } else {
            need(!residual_out, "residual_out goes with a residual");
        }
        const bool bf16 = a.truth(4, true);
        if (bf16) {
            if (!out)
                new_out = on.make(shape, kBf16, x);
            const Tensor &to = out ? *out : new_out;
            r = rows_of(to, shape, to.scalar_type() == kBf16, dev, "out");
            p.out = r.p;
            p.out_stride = r.stride;
        } else {
            need(!out, "out goes with bf16=True");
        }
        const bool fp8 = a.v[5] != nullptr;
        if (fp8) {
            const int64_t group = a.integer(5, 0);
            need(group == 0 || group == 16 || group == 32 || group == 64 || group == 128 || group == 256,
                 "fp8_group must be 0, 16, 32, 64, 128 or 256");
            p.group = (int32_t)group;
            const int64_t groups[2] = {shape[0], group ? (K + group - 1) / group : 1};
            if (!codes)
                new_codes = on.make(shape, at::kFloat8_e4m3fn, x);
            if (!scales)
                new_scales = on.make(groups, kF32, x);
            const Tensor &to = codes ? *codes : new_codes;
            r = rows_of(to, shape,
                        to.scalar_type() == at::kFloat8_e4m3fn || to.scalar_type() == at::kByte, dev,
                        "codes");
            p.codes = static_cast<uint8_t *>(r.p);
            p.codes_stride = r.stride;
            p.scales =
                static_cast<float *>(flat(scales ? *scales : new_scales, groups, kF32, dev, "scales"));
        } else {
            need(!codes && !scales, "codes and scales go with fp8_group");
        }
        need(bf16 || fp8, "no output asked for");
        if (shape[0] > 0)
            check("dvl_add_rmsnorm", dvl_add_rmsnorm(&p, on.stream()));
        PyObject *t = PyTuple_New(4);
        PyTuple_SET_ITEM(t, 0, bf16 ? wrap(out, a.v[6], new_out) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(t, 1, residual ? wrap(residual_out, a.v[7], new_residual) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(t, 2, fp8 ? wrap(codes, a.v[8], new_codes) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(t, 3, fp8 ? wrap(scales, a.v[9], new_scales) : Py_NewRef(Py_None));
        return t;
    });
}

// ---- paged_attention ----------------------------------------------------

Signature attention_sig = {"paged_attention", 4, 10,
                           {"cache", "q", "table", "lengths", "scale", "out", "lse", "want_lse", "ws",
                            "stream"},
                           {}};

PyObject *paged_attention(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw)
{
    return guarded([&]() -> PyObject * {
        const Args a(attention_sig, args, n, kw);
        need(a.v[0] != nullptr, "cache must be a KVCache");
        int dev = -1;
        const dvl_kv_cache *cache = cache_of(a.v[0], &dev);
        const Place on(a.v[9], dev);
        const Tensor &q = a.required(1, "q"), &table = a.required(2, "table"),
                     &lengths = a.required(3, "lengths");
        const int64_t dim = q.dim();
        need(dim == 3 || dim == 4, "q must be [B][T][Hq][D] or [B][Hq][D]");
        const at::IntArrayRef shape = q.sizes();
        const int64_t B = shape[0], T = dim == 4 ? shape[1] : 1, Hq = shape[dim - 2], D = shape[dim - 1];
        need(cuda_device(q) == dev && q.scalar_type() == kBf16 && D == cache->D && q.stride(dim - 1) == 1,
             "q must be bf16 on the cache's device, its last axis the cache's D, contiguous");
        need(cuda_device(table) == dev && table.scalar_type() == kI32 && table.dim() == 2 &&
                 table.size(0) == B && (table.stride(1) == 1 || table.size(1) == 1),
             "table must be a CUDA int32 [B][width] tensor with contiguous rows");
        need(B <= INT32_MAX && T <= INT32_MAX && Hq <= INT32_MAX && table.size(1) <= INT32_MAX,
             "sizes past 2^31");
        const auto *pl = static_cast<const int32_t *>(flat(lengths, {B}, kI32, dev, "lengths"));
        const Tensor *out = a.tensor(5, "out"), *lse = a.tensor(6, "lse");
        const bool want_lse = lse || a.truth(7, true);
        const at::IntArrayRef rows = shape.slice(0, dim - 1);
        Tensor new_out, new_lse;
        if (!out)
            new_out = on.make(shape, kBf16, q);
        if (!lse && want_lse)
            new_lse = on.make(rows, kF32, q);
        void *po = flat(out ? *out : new_out, shape, kBf16, dev, "out");
        float *pe = want_lse ? static_cast<float *>(flat(lse ? *lse : new_lse, rows, kF32, dev, "lse"))
                             : nullptr;
        Workspace ws;
        if (const Tensor *t = a.tensor(8, "ws")) {
            ws.set(*t, dev);
        } else if (B > 0) {
            ws.owned = new_workspace("attention_workspace",
                                     Py_BuildValue("(OLLL)", a.v[0], (long long)B, (long long)T,
                                                   (long long)Hq),
                                     a.v[9]);
            ws.set(THPVariable_Unpack(ws.owned), dev);
        }
        const float scale = (float)a.number(4, 1.0 / std::sqrt((double)D));
        if (B > 0)
            check("dvl_paged_attention",
                  dvl_paged_attention(cache, q.data_ptr(), B > 1 ? q.stride(0) : 0,
                                      dim == 4 && T > 1 ? q.stride(1) : 0,
                                      Hq > 1 ? q.stride(dim - 2) : 0, (int32_t)B, (int32_t)T,
                                      (int32_t)Hq, static_cast<const int32_t *>(table.data_ptr()),
                                      B > 1 ? table.stride(0) : 0, (int32_t)table.size(1), pl, scale,
                                      po, pe, ws.p, ws.bytes, on.stream()));
        PyObject *t = PyTuple_New(2);
        PyTuple_SET_ITEM(t, 0, wrap(out, a.v[5], new_out));
        PyTuple_SET_ITEM(t, 1, want_lse ? wrap(lse, a.v[6], new_lse) : Py_NewRef(Py_None));
        return t;
    });
}

// ---- beam_select --------------------------------------------------------

Signature select_sig = {"beam_select", 3, 9,
                        {"logits", "scores", "k", "d2t", "out_scores", "parents", "tokens", "ws", "stream"},
                        {}};

PyObject *beam_select(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw)
{
    return guarded([&]() -> PyObject * {
        const Args a(select_sig, args, n, kw);
        const Tensor &logits = a.required(0, "logits"), &scores = a.required(1, "scores");
        const int dev = cuda_device(logits);
        need(dev >= 0 && logits.dim() == 3 && (logits.stride(2) == 1 || logits.size(2) == 1),
             "logits must be a CUDA [batch][beams][N] tensor with contiguous rows");
        const Place on(a.v[8], dev);
        const auto type = logits.scalar_type();
        need(type == kF32 || type == kBf16, "logits must be bf16 or fp32");
        const int64_t batch = logits.size(0), beams = logits.size(1), N = logits.size(2);
        need(batch <= INT32_MAX && beams <= INT32_MAX && N <= INT32_MAX, "sizes past 2^31");
        need(a.v[2] != nullptr, "k is missing");
        const int64_t k = a.integer(2, 0);
        need(k >= 1 && k <= DVL_MAX_BEAMS && beams >= 1 && beams <= DVL_MAX_BEAMS && N >= 1,
             "k or beams outside 1 .. 32, or no logits");
        const auto *p_in = static_cast<const float *>(flat(scores, {batch, beams}, kF32, dev, "scores"));
        const Tensor *d2t = a.tensor(3, "d2t");
        const auto *pd =
            d2t ? static_cast<const int32_t *>(flat(*d2t, {N}, kI32, dev, "d2t")) : nullptr;
        const Tensor *given[3] = {a.tensor(4, "out_scores"), a.tensor(5, "parents"), a.tensor(6, "tokens")};
        const char *names[3] = {"out_scores", "parents", "tokens"};
        const int64_t got[2] = {batch, k};
        Tensor made[3];
        void *p[3];
        for (int i = 0; i < 3; ++i) {
            const auto t = i == 0 ? kF32 : kI32;
            if (!given[i])
                made[i] = on.make(got, t, logits);
            p[i] = flat(given[i] ? *given[i] : made[i], got, t, dev, names[i]);
        }
        Workspace ws;
        if (const Tensor *t = a.tensor(7, "ws")) {
            ws.set(*t, dev);
        } else if (batch > 0) {
            ws.owned = new_workspace("_beam_workspace_on",
                                     Py_BuildValue("(LLLi)", (long long)batch, (long long)beams,
                                                   (long long)N, dev),
                                     a.v[8]);
            ws.set(THPVariable_Unpack(ws.owned), dev);
        }
        if (batch > 0)
            check("dvl_beam_select",
                  dvl_beam_select(logits.data_ptr(), type == kF32 ? DVL_F32 : DVL_BF16, logits.stride(0),
                                  logits.stride(1), p_in, (int32_t)batch, (int32_t)beams, (int32_t)N,
                                  (int32_t)k, pd, static_cast<float *>(p[0]), static_cast<int32_t *>(p[1]),
                                  static_cast<int32_t *>(p[2]), ws.p, ws.bytes, on.stream()));
        PyObject *t = PyTuple_New(3);
        for (int i = 0; i < 3; ++i)
            PyTuple_SET_ITEM(t, i, wrap(given[i], a.v[4 + i], made[i]));
        return t;
    });
}

// ---- beam_reorder -------------------------------------------------------

Signature reorder_sig = {"beam_reorder", 2, 10,
                         {"parents", "states", "states_out", "cache", "table", "table_out", "lengths",
                          "lengths_out", "spare", "stream"},
                         {}};

// A list or tuple of tensors; its items stay borrowed from it.
std::vector<PyObject *> items_of(PyObject *seq, const char *what)
{
    std::vector<PyObject *> v;
    if (!seq)
        return v;
    if (!PyList_Check(seq) && !PyTuple_Check(seq))
        throw Refused{std::string(what) + " must be a list or tuple of tensors"};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *x = PySequence_Fast_GET_ITEM(seq, i);
        if (!THPVariable_Check(x))
            throw Refused{std::string(what) + " must hold tensors"};
        v.push_back(x);
    }
    return v;
}

PyObject *beam_reorder(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw)
{
    return guarded([&]() -> PyObject * {
        const Args a(reorder_sig, args, n, kw);
        const Tensor &parents = a.required(0, "parents");
        const int dev = cuda_device(parents);
        need(dev >= 0 && parents.dim() == 2, "parents must be a CUDA int32 [batch][k] tensor");
        const Place on(a.v[9], dev);
        const int64_t batch = parents.size(0), k = parents.size(1);
        const auto *pp =
            static_cast<const int32_t *>(flat(parents, {batch, k}, kI32, dev, "parents"));
        const auto states = items_of(a.v[1], "states");
        auto outs = items_of(a.v[2], "states_out");
        const int count = (int)states.size();
        need(states.size() <= DVL_MAX_STATES, "at most 8 states");
        need(count > 0 || a.v[3], "nothing to reorder");
        const Tensor *table = a.tensor(4, "table"), *lengths = a.tensor(6, "lengths"),
                     *spare = a.tensor(8, "spare");
        if (a.v[3])
            need(table && table->dim() == 3 && lengths && spare,
                 "a cache goes with table, lengths and spare");
        else
            need(!table && !lengths && !spare, "table, lengths and spare go with a cache");
        need(count == 0 || THPVariable_Unpack(states[0]).dim() >= 2, "a state must be [batch][beams][...]");
        const int64_t beams = count ? THPVariable_Unpack(states[0]).size(1) : table->size(1);
        need(batch <= INT32_MAX && beams <= INT32_MAX && k <= INT32_MAX, "sizes past 2^31");

        need(!a.v[2] || (int)outs.size() == count, "states_out must match states");
        std::vector<Tensor> made(a.v[2] ? 0 : count);
        dvl_state st[DVL_MAX_STATES];
        for (int i = 0; i < count; ++i) {
            const Tensor &s = THPVariable_Unpack(states[i]);
            std::vector<int64_t> in(s.sizes().begin(), s.sizes().end());
            need(in.size() >= 2, "a state must be [batch][beams][...]");
            std::vector<int64_t> to = in;
            in[0] = to[0] = batch;
            in[1] = beams;
            to[1] = k;
            int64_t bytes = s.element_size();
            for (size_t j = 2; j < in.size(); ++j)
                bytes *= in[j];
            need(bytes > 0, "a state's rows must not be empty");
            st[i].src = flat(s, in, s.scalar_type(), dev, "a state");
            if (!a.v[2])
                made[i] = on.make(to, s.scalar_type(), s);
            st[i].dst = flat(a.v[2] ? THPVariable_Unpack(outs[i]) : made[i], to, s.scalar_type(), dev,
                             "a state's output");
            st[i].row_bytes = st[i].src_stride = st[i].dst_stride = bytes;
        }
        const dvl_kv_cache *cache = nullptr;
        dvl_beam_pages pages = {};
        const Tensor *table_out = a.tensor(5, "table_out"), *lengths_out = a.tensor(7, "lengths_out");
        Tensor new_table, new_lengths;
        if (a.v[3]) {
            int cache_dev = -1;
            cache = cache_of(a.v[3], &cache_dev);
            need(cache_dev == dev, "the cache must be on the parents' device");
            const int64_t width = table->size(2);
            need(width <= INT32_MAX, "sizes past 2^31");
            if (!table_out)
                new_table = on.make({batch, k, width}, kI32, parents);
            if (!lengths_out)
                new_lengths = on.make({batch, k}, kI32, parents);
            auto ints = [&](const Tensor &t, at::IntArrayRef shape, const char *name) {
                return static_cast<int32_t *>(flat(t, shape, kI32, dev, name));
            };
            pages.table = ints(*table, {batch, beams, width}, "table");
            pages.table_out = ints(table_out ? *table_out : new_table, {batch, k, width}, "table_out");
            pages.lengths = ints(*lengths, {batch, beams}, "lengths");
            pages.lengths_out = ints(lengths_out ? *lengths_out : new_lengths, {batch, k}, "lengths_out");
            pages.spare = ints(*spare, {batch, k}, "spare");
            pages.width = (int32_t)width;
        }
        if (batch > 0)
            check("dvl_beam_reorder",
                  dvl_beam_reorder(st, count, cache ? &pages : nullptr, cache, pp, (int32_t)batch,
                                   (int32_t)beams, (int32_t)k, on.stream()));
        PyObject *list = PyList_New(count);
        for (int i = 0; i < count; ++i)
            PyList_SET_ITEM(list, i, a.v[2] ? Py_NewRef(outs[i]) : THPVariable_Wrap(made[i]));
        PyObject *t = PyTuple_New(3);
        PyTuple_SET_ITEM(t, 0, list);
        PyTuple_SET_ITEM(t, 1, cache ? wrap(table_out, a.v[5], new_table) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(t, 2, cache ? wrap(lengths_out, a.v[7], new_lengths) : Py_NewRef(Py_None));
        return t;
    });
}

// ---- qk_norm_rope -------------------------------------------------------

Signature qk_sig = {"qk_norm_rope", 3, 15,
                    {"q", "k", "v", "rope", "q_weight", "k_weight", "eps", "positions", "cache", "table",
                     "lengths", "starts", "q_out", "k_out", "stream"},
                    {}};

// A tensor [rows][heads][D] whose values of a head are contiguous, or the same
// with the rows as [B][T], which must lie evenly.
struct HeadRows {
    const void *p = nullptr;
    int64_t stride = 0, head_stride = 0;
};
HeadRows heads_of(const Tensor &t, at::IntArrayRef shape, int dev, const char *name)
{
    const int64_t n = (int64_t)shape.size();
    bool ok = cuda_device(t) == dev && t.scalar_type() == kBf16 && t.sizes() == shape &&
              (t.stride(n - 1) == 1 || t.numel() == 0);
    if (ok && n == 4 && shape[0] > 1 && shape[1] > 1)
        ok = t.stride(0) == shape[1] * t.stride(1);
    if (!ok)
        throw Refused{std::string(name) + " must be a bf16 tensor of shape " + shape_text(shape) +
                      " on q's device, the values of a head contiguous and the rows evenly spaced"};
    const int64_t rows = n == 4 ? shape[0] * shape[1] : shape[0];
    HeadRows r;
    r.p = t.data_ptr();
    r.stride = rows > 1 ? (n == 4 && shape[1] == 1 ? t.stride(0) : t.stride(n - 3)) : 0;
    r.head_stride = shape[n - 2] > 1 ? t.stride(n - 2) : 0;
    return r;
}

// What a Rope object holds (step.py).
struct RopeOf {
    const Tensor *freq = nullptr;
    int dim = 0;
    bool interleaved = false;
    PyObject *held = nullptr;  // keeps freq alive

    RopeOf(PyObject *rope, int dev)
    {
        if (!rope)
            return;
        static PyObject *names[3] = {PyUnicode_InternFromString("freq"), PyUnicode_InternFromString("dim"),
                                     PyUnicode_InternFromString("interleaved")};
        held = PyObject_GetAttr(rope, names[0]);
        PyObject *d = held ? PyObject_GetAttr(rope, names[1]) : nullptr;
        PyObject *i = d ? PyObject_GetAttr(rope, names[2]) : nullptr;
        const bool ok = i && THPVariable_Check(held);
        if (ok) {
            freq = &THPVariable_Unpack(held);
            dim = (int)PyLong_AsLong(d);
            interleaved = PyObject_IsTrue(i) == 1;
        }
        Py_XDECREF(d);
        Py_XDECREF(i);
        if (!ok || PyErr_Occurred()) {
            PyErr_Clear();
            Py_XDECREF(held);
            throw Refused{"rope must be a Rope"};
        }
        if (cuda_device(*freq) != dev) {
            Py_XDECREF(held);
            throw Refused{"the Rope must be on q's device"};
        }
    }
    ~RopeOf() { Py_XDECREF(held); }
    RopeOf(const RopeOf &) = delete;
    RopeOf &operator=(const RopeOf &) = delete;
};

PyObject *qk_norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw)
{
    return guarded([&]() -> PyObject * {
        const Args a(qk_sig, args, n, kw);
        const Tensor &q = a.required(0, "q"), &k = a.required(1, "k");
        const int dev = cuda_device(q);
        const int64_t dim = q.dim();
        need(dev >= 0 && (dim == 3 || dim == 4) && k.dim() == dim,
             "q and k must be CUDA [rows][heads][D] or [B][T][heads][D] tensors");
        const Place on(a.v[14], dev);
        const at::IntArrayRef shape = q.sizes();
        const int64_t rows = dim == 4 ? shape[0] * shape[1] : shape[0];
        need(rows <= INT32_MAX && shape[dim - 1] <= INT32_MAX && shape[dim - 2] <= INT32_MAX &&
                 k.size(dim - 2) <= INT32_MAX,
             "sizes past 2^31");
        std::vector<int64_t> kshape(shape.begin(), shape.end());
        kshape[dim - 2] = k.size(dim - 2);
        const int64_t D = shape[dim - 1];
        dvl_qk p = {};
        p.rows = rows;
        p.Hq = (int32_t)shape[dim - 2];
        p.H = (int32_t)kshape[dim - 2];
        p.D = (int32_t)D;
        p.eps = (float)a.number(6, 1e-6);
        HeadRows r = heads_of(q, shape, dev, "q");
        p.q = r.p, p.q_stride = r.stride, p.q_head_stride = r.head_stride;
        r = heads_of(k, kshape, dev, "k");
        p.k = r.p, p.k_stride = r.stride, p.k_head_stride = r.head_stride;
        const Tensor *v = a.tensor(2, "v");
        if (v) {
            r = heads_of(*v, kshape, dev, "v");
            p.v = r.p, p.v_stride = r.stride, p.v_head_stride = r.head_stride;
        }
        const RopeOf rope(a.v[3], dev);
        if (rope.freq) {
            need(rope.dim <= D, "the Rope rotates more values than a head has");
            p.rot = rope.dim;
            p.interleaved = rope.interleaved;
            p.freq = static_cast<const uint64_t *>(flat(*rope.freq, {rope.dim / 2}, at::kLong, dev, "the Rope's freq"));
        }
        const Tensor *wq = a.tensor(4, "q_weight"), *wk = a.tensor(5, "k_weight");
        if (wq)
            p.q_weight = flat(*wq, {D}, kBf16, dev, "q_weight");
        if (wk)
            p.k_weight = flat(*wk, {D}, kBf16, dev, "k_weight");
        if (const Tensor *positions = a.tensor(7, "positions")) {
            if (dim == 4 && positions->dim() == 2)
                p.positions = static_cast<const int32_t *>(flat(*positions, shape.slice(0, 2), kI32, dev, "positions"));
            else
                p.positions = static_cast<const int32_t *>(flat(*positions, {rows}, kI32, dev, "positions"));
        }
        const Tensor *table = a.tensor(9, "table"), *lengths = a.tensor(10, "lengths"),
                     *starts = a.tensor(11, "starts");
        if (a.v[8]) {
            int cache_dev = -1;
            p.cache = cache_of(a.v[8], &cache_dev);
            need(cache_dev == dev, "the cache must be on q's device");
            need(v && table && lengths, "a cache goes with v, table and lengths");
            need(cuda_device(*table) == dev && table->scalar_type() == kI32 && table->dim() == 2 &&
                     (table->stride(1) == 1 || table->size(1) == 1),
                 "table must be a CUDA int32 [B][width] tensor with contiguous rows");
            const int64_t B = table->size(0);
            need(B <= INT32_MAX && table->size(1) <= INT32_MAX, "sizes past 2^31");
            need(!starts || dim == 3, "starts goes with q as [rows][heads][D]");
            need(dim == 3 || shape[0] == B, "q's first axis must be table's");
            need(starts || (B > 0 ? rows % B == 0 : rows == 0), "rows without starts must be as many for each sequence");
            p.table = static_cast<const int32_t *>(table->data_ptr());
            p.table_stride = B > 1 ? table->stride(0) : 0;
            p.table_width = (int32_t)table->size(1);
            p.B = (int32_t)B;
            p.lengths = static_cast<const int32_t *>(flat(*lengths, {B}, kI32, dev, "lengths"));
            if (starts)
                p.starts = static_cast<const int32_t *>(flat(*starts, {B + 1}, kI32, dev, "starts"));
        } else {
            need(!v && !table && !lengths && !starts, "v, table, lengths and starts go with a cache");
            need(!rope.freq || p.positions, "without a cache a Rope goes with positions");
        }
        const Tensor *q_out = a.tensor(12, "q_out"), *k_out = a.tensor(13, "k_out");
        const bool want_k = k_out || !a.v[8];
        Tensor new_q, new_k;
        if (!q_out)
            new_q = on.make(shape, kBf16, q);
        r = heads_of(q_out ? *q_out : new_q, shape, dev, "q_out");
        p.q_out = const_cast<void *>(r.p), p.q_out_stride = r.stride, p.q_out_head_stride = r.head_stride;
        if (want_k) {
            if (!k_out)
                new_k = on.make(kshape, kBf16, q);
            r = heads_of(k_out ? *k_out : new_k, kshape, dev, "k_out");
            p.k_out = const_cast<void *>(r.p), p.k_out_stride = r.stride, p.k_out_head_stride = r.head_stride;
        }
        if (rows > 0) {
            need(dvl_qk_norm_rope != nullptr, "this build has no qk_norm_rope");
            check("dvl_qk_norm_rope", dvl_qk_norm_rope(&p, on.stream()));
        }
        PyObject *t = PyTuple_New(2);
        PyTuple_SET_ITEM(t, 0, wrap(q_out, a.v[12], new_q));
        PyTuple_SET_ITEM(t, 1, want_k ? wrap(k_out, a.v[13], new_k) : Py_NewRef(Py_None));
        return t;
    });
}

// ---- cache_keep ---------------------------------------------------------

Signature keep_sig = {"cache_keep", 6, 8,
                      {"cache", "table", "lengths", "first", "keep", "counts", "lengths_out", "stream"},
                      {}};

PyObject *cache_keep(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw)
{
    return guarded([&]() -> PyObject * {
        const Args a(keep_sig, args, n, kw);
        need(a.v[0] != nullptr, "cache must be a KVCache");
        int dev = -1;
        const dvl_kv_cache *cache = cache_of(a.v[0], &dev);
        const Place on(a.v[7], dev);
        const Tensor &table = a.required(1, "table"), &lengths = a.required(2, "lengths"),
                     &first = a.required(3, "first"), &keep = a.required(4, "keep"),
                     &counts = a.required(5, "counts");
        auto rows = [&](const Tensor &t) {
            return cuda_device(t) == dev && t.scalar_type() == kI32 && t.dim() == 2 &&
                   (t.stride(1) == 1 || t.size(1) <= 1) && t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX;
        };
        need(rows(table), "table must be a CUDA int32 [B][width] tensor with contiguous rows");
        need(rows(keep) && keep.size(0) == table.size(0),
             "keep must be a CUDA int32 [B][M] tensor with contiguous rows");
        const int64_t B = table.size(0);
        auto ints = [&](const Tensor &t, const char *name) {
            return static_cast<int32_t *>(flat(t, {B}, kI32, dev, name));
        };
        const int32_t *pl = ints(lengths, "lengths"), *pf = ints(first, "first"), *pc = ints(counts, "counts");
        const Tensor *out = a.tensor(6, "lengths_out");
        Tensor made;
        if (!out)
            made = on.make({B}, kI32, lengths);
        int32_t *po = ints(out ? *out : made, "lengths_out");
        if (B > 0) {
            need(dvl_cache_keep != nullptr, "this build has no cache_keep");
            check("dvl_cache_keep",
                  dvl_cache_keep(cache, static_cast<const int32_t *>(table.data_ptr()),
                                 B > 1 ? table.stride(0) : 0, (int32_t)table.size(1), pl, pf,
                                 static_cast<const int32_t *>(keep.data_ptr()), B > 1 ? keep.stride(0) : 0, pc,
                                 (int32_t)B, (int32_t)keep.size(1), po, on.stream()));
        }
        return wrap(out, a.v[6], made);
    });
}

// ---- module -------------------------------------------------------------

#define DVL_METHOD(name, doc)                                                           \
    {                                                                                   \
        #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)),       \
            METH_FASTCALL | METH_KEYWORDS, doc                                          \
    }

PyMethodDef methods[] = {
    DVL_METHOD(add_rmsnorm,
               "add_rmsnorm(x, weight, residual=None, *, eps=1e-6, bf16=True, fp8_group=None, out=None,\n"
               "            residual_out=None, codes=None, scales=None, stream=None)\n--\n\n"
               "u = x + residual; y = u * weight / sqrt(mean(u^2) + eps), per row.\n\n"
               "x:         CUDA bf16 [rows][K] (rows may be strided).\n"
               "residual:  bf16 or fp32 [rows][K], or None (u = x).\n"
               "bf16:      whether y is wanted in bf16.\n"
               "fp8_group: None, or the number of values per scale of E4M3 codes of y\n"
               "           (16, 32, 64, 128, 256; 0: one scale per row).\n"
               "Returns (out, residual_out, codes, scales) with None for what was not asked\n"
               "for; y ~ codes * scales.  residual_out (u in the residual's type) may be\n"
               "the residual itself; codes is float8_e4m3fn (a given one may be uint8)."),
    DVL_METHOD(paged_attention,
               "paged_attention(cache, q, table, lengths, *, scale=None, out=None, lse=None,\n"
               "                want_lse=True, ws=None, stream=None)\n--\n\n"
               "Attention of the T newest tokens of each sequence over its cached keys\n"
               "and values (its own included: lengths counts them).\n\n"
               "cache:   a KVCache.\n"
               "q:       bf16 [B][T][Hq][D], or [B][Hq][D] for one token.\n"
               "table:   int32 [B][width]: the page of each page_size tokens.\n"
               "lengths: int32 [B].\n"
               "scale:   of the scores; 1 / sqrt(D) by default.\n"
               "ws:      from attention_workspace (made for the call otherwise).\n"
               "Returns (out, lse): bf16 of q's shape and fp32 without the D axis (None\n"
               "without want_lse).  An empty sequence, and a token that sees no position,\n"
               "give 0 and -inf."),
    DVL_METHOD(beam_select,
               "beam_select(logits, scores, k, *, d2t=None, out_scores=None, parents=None,\n"
               "            tokens=None, ws=None, stream=None)\n--\n\n"
               "The k best next beams of each request, best first: score(j, n) =\n"
               "scores[j] + log_softmax(logits[j])[n].\n\n"
               "logits: CUDA bf16 or fp32 [batch][beams][N], rows contiguous.\n"
               "scores: fp32 [batch][beams]; -inf marks a dead beam.\n"
               "d2t:    int32 [N] full-vocabulary id of each row, or None (the row).\n"
               "ws:     from beam_workspace (made for the call otherwise).\n"
               "Returns (scores fp32, parents int32, tokens int32), each [batch][k]; places\n"
               "without a candidate hold (-inf, -1, -1)."),
    DVL_METHOD(beam_reorder,
               "beam_reorder(parents, states=(), *, states_out=None, cache=None, table=None,\n"
               "             table_out=None, lengths=None, lengths_out=None, spare=None, stream=None)\n--\n\n"
               "Give each new beam its parent's rows: state[b][parents[b][i]] for every\n"
               "state, zeros for a parent outside [0, beams).\n\n"
               "parents: int32 [batch][k].\n"
               "states:  CUDA tensors [batch][beams][...], contiguous, any type.\n"
               "With cache, table [batch][beams][width], lengths [batch][beams] and spare\n"
               "[batch][k] (int32): the page tables and lengths move the same way, and the\n"
               "new beam gets its spare page in place of the parent's partly filled last\n"
               "page, with that page's tokens copied (in the cache, in place).\n"
               "Outputs overlap neither inputs nor each other: nothing but the cache moves\n"
               "in place.\n"
               "Returns (states, table, lengths) as tensors [batch][k][...]; the last two\n"
               "None without a cache."),
    DVL_METHOD(qk_norm_rope,
               "qk_norm_rope(q, k, v=None, *, rope=None, q_weight=None, k_weight=None, eps=1e-6,\n"
               "             positions=None, cache=None, table=None, lengths=None, starts=None,\n"
               "             q_out=None, k_out=None, stream=None)\n--\n\n"
               "Norm of the new tokens' queries and keys for each head (with a weight),\n"
               "rotation by their position (with a Rope), and with a cache the new keys and\n"
               "values to their places there.\n\n"
               "q, k, v: CUDA bf16 [rows][heads][D] or [B][T][heads][D]; heads and rows may be\n"
               "         strided (views of one projection's output).\n"
               "q_weight, k_weight: bf16 [D]; None: no norm.\n"
               "cache, table [B][width], lengths [B] (int32): as in paged_attention; lengths\n"
               "         counts the new tokens, whose places are the last ones.\n"
               "starts:  int32 [B + 1], rising: sequence b's new tokens are rows starts[b] ..\n"
               "         starts[b + 1] - 1; rows past starts[B] are padding, left as they are.\n"
               "         None: as many for every sequence.\n"
               "positions: int32 [rows] to rotate by in place of the tokens' places (a tree's\n"
               "         depths); needed by a Rope without a cache.\n"
               "q_out, k_out: may be q and k themselves.\n"
               "Returns (q_out, k_out), bf16; k_out is None with a cache unless it is given."),
    DVL_METHOD(cache_keep,
               "cache_keep(cache, table, lengths, first, keep, counts, *, lengths_out=None,\n"
               "           stream=None)\n--\n\n"
               "Keep some of each sequence's newest tokens, without gaps: the token at place\n"
               "first[b] + keep[b][i] moves to place first[b] + i for i < counts[b], in the\n"
               "cache, in place.\n\n"
               "table:   int32 [B][width]; lengths, first, counts: int32 [B].\n"
               "keep:    int32 [B][M], strictly rising in each row.\n"
               "For a caller that verifies a tree by its own attention, or drops tokens of a\n"
               "long cache: what is accepted of a chain, as paged_attention masks it, lies\n"
               "without gaps already.\n"
               "Returns the new lengths, first + counts (int32 [B])."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", "The drafting step's operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step(void)
{
    intern(norm_sig);
    intern(attention_sig);
    intern(select_sig);
    intern(reorder_sig);
    intern(qk_sig);
    intern(keep_sig);
    return PyModule_Create(&module);
}
