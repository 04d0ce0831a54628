// marshal.cpp - argument marshalling of the softmax-attention serving calls,
// compiled: these run in decode loops, where a step's kernels take a few
// microseconds and the host's time is what counts.  Like the ctypes part of the
// binding it only checks device, type, shape and strides of torch tensors,
// allocates outputs that were not given, and passes pointers and the current
// stream to libgdn.so.  On the GB300's host a gdn_page_plan call takes 6.4 us this
// way (20.5 through ctypes), gdn_qk_norm_rope 4.1 (16), gdn_attention_paged 7.1
// (22), gdn_attention_varlen 4.3 (17).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <optional>
#include <string>
#include <vector>

#include "gdn.h"

namespace {

PyObject *g_error = nullptr;  // GdnError, set by init()

// Up to so many new tokens (8 MB) the six outputs of a plan share one allocation, which any one of them
// keeps alive: six allocations take longer than the rest of the call (64 requests: 9.7 us with six, 6.4
// with one; with 107781 new tokens a call among others 13.1 and 8.8).
constexpr int kSharedN = 1 << 20;

// Lets other Python threads run while it lives: allocations and launches may wait for the device, and what the
// device waits for (a host function in a stream) may need the interpreter.
class Unlocked {
    PyThreadState *state_ = PyEval_SaveThread();

public:
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    ~Unlocked() { PyEval_RestoreThread(state_); }
};

at::Tensor allocate(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    const Unlocked others;
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// A refusal with a gdn_status.
struct Refusal {
    int status;
    std::string message;
};
// A Python exception is set already.
struct Raised {};

const char *type_name(at::ScalarType t) {
    switch (t) {
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
    }
}

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
        throw Raised{};
    }
    return THPVariable_Unpack(o);
}

const at::Tensor &tensor_of(PyObject *o, const char *name, int dims) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != dims)
        throw Refusal{GDN_ERR_SHAPE, std::string(name) + " has " + std::to_string(t.dim()) + " dimensions, expected " +
                                         std::to_string(dims)};
    return t;
}

c10::Device cuda_device(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) throw Refusal{GDN_ERR_CUDA, std::string(name) + " must be a CUDA tensor"};
    return t.device();
}

void check(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
    if (t.device() != dev)
        throw Refusal{GDN_ERR_CUDA, std::string(name) + " is on " + t.device().str() + ", expected " + dev.str()};
    if (t.scalar_type() != type)
        throw Refusal{GDN_ERR_SHAPE, std::string(name) + " has dtype " + type_name(t.scalar_type()) + ", expected " + type_name(type)};
    if (t.sizes() != shape)
        throw Refusal{GDN_ERR_SHAPE, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape)};
}

// Pointer of a contiguous tensor (None: nullptr when optional).
void *at(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape, dev);
    if (!t.is_contiguous()) throw Refusal{GDN_ERR_SHAPE, std::string(name) + " must be contiguous"};
    return t.data_ptr();
}

// Pointer and token stride of rows that are contiguous but for the token stride.
void *rows(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev, int64_t &stride) {
    check(t, name, type, shape, dev);
    int64_t width = 1;
    for (size_t i = shape.size(); i-- > 1;) {
        if (shape[i] != 1 && t.stride(i) != width)
            throw Refusal{GDN_ERR_SHAPE, std::string(name) + " must be contiguous within a token"};
        width *= shape[i];
    }
    stride = shape[0] > 1 ? t.stride(0) : width;
    if (stride < width)
        throw Refusal{GDN_ERR_SHAPE, std::string(name) + " has token stride " + std::to_string(stride) +
                                         ", below its row width " + std::to_string(width)};
    return t.data_ptr();
}

// An output: the caller's tensor or a new one, its pointer, and a reference to return.
struct Out {
    PyObject *object = nullptr;
    void *ptr = nullptr;
    Out(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
        if (o == Py_None) {
            at::Tensor t = allocate(shape, type, dev);
            ptr = t.data_ptr();
            object = THPVariable_Wrap(std::move(t));
            if (!object) throw Raised{};
        } else {
            ptr = at(o, name, type, shape, dev);
            Py_INCREF(o);
            object = o;
        }
    }
    // A new output of n values inside `all`, from value `from` on, which it moves past them and up to
    // a multiple of four.
    Out(const at::Tensor &all, int64_t n, int64_t &from) {
        at::Tensor t = all.as_strided({n}, {1}, from);
        ptr = t.data_ptr();
        from += (n + 3) / 4 * 4;
        object = THPVariable_Wrap(std::move(t));
        if (!object) throw Raised{};
    }
    Out(const Out &) = delete;
    ~Out() { Py_XDECREF(object); }
    PyObject *give() {
        PyObject *o = object;
        object = nullptr;
        return o;
    }
};

int whole(PyObject *o, const char *name) {
    PyObject *n = PyNumber_Index(o);
    if (!n) throw Raised{};
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(n, &over);
    Py_DECREF(n);
    if (over || v > INT_MAX || v < INT_MIN) throw Refusal{GDN_ERR_OVERFLOW, std::string(name) + " is out of the int32 range"};
    return (int)v;
}

// A tensor size as the int that the C calls take.
int extent(int64_t n, const char *name) {
    if (n > INT_MAX) throw Refusal{GDN_ERR_OVERFLOW, std::string(name) + " exceeds int32"};
    return (int)n;
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

int activation(at::ScalarType t) {
    if (t == at::kBFloat16) return GDN_BF16;
    if (t == at::kFloat) return GDN_F32;
    throw Refusal{GDN_ERR_UNSUPPORTED, std::string("activation dtype ") + type_name(t) + " not supported (bf16 or fp32)"};
}

void *stream(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// The call, whose refusal becomes an exception.
template <typename F>
void launch(F call) {
    int status;
    {
        const Unlocked others;
        status = call();
    }
    if (status != GDN_OK) throw Refusal{status, gdn_last_error()};
}

// Runs a call and turns what it throws into a Python exception.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t expected, F f) {
    if (n != expected) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised &) {
    } catch (const Refusal &r) {
        PyObject *e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, g_error ? "is" : "i", r.status, r.message.c_str());
        if (e) {
            PyErr_SetObject((PyObject *)Py_TYPE(e), e);
            Py_DECREF(e);
        }
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject *tuple(std::initializer_list<Out *> outs) {
    PyObject *t = PyTuple_New((Py_ssize_t)outs.size());
    if (!t) throw Raised{};
    Py_ssize_t i = 0;
    for (Out *o : outs) {
        PyObject *x = o ? o->give() : nullptr;
        if (!x) {
            Py_INCREF(Py_None);
            x = Py_None;
        }
        PyTuple_SET_ITEM(t, i++, x);
    }
    return t;
}

// (new_lens, cached_lens, block_table, free_pages, page_size, N, cursor, offsets, kv_lens, positions, slots,
//  cursor_out, status)
PyObject *page_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const at::Tensor &table = tensor_of(a[2], "block_table", 2), &free = tensor(a[3], "free_pages");
        const c10::Device dev = cuda_device(table, "block_table");
        const int B = extent(table.size(0), "B"), M = extent(table.size(1), "max_pages"), F = extent(free.numel(), "n_free");
        const int ps = whole(a[4], "page_size"), N = whole(a[5], "N");
        if (N < 0) throw Refusal{GDN_ERR_SHAPE, "N must not be negative"};
        const c10::cuda::CUDAGuard guard(dev);
        const auto i32 = at::kInt;
        const int32_t *nl = (int32_t *)at(a[0], "new_lens", i32, {B}, dev), *cl = (int32_t *)at(a[1], "cached_lens", i32, {B}, dev);
        int32_t *bt = (int32_t *)at(a[2], "block_table", i32, {B, M}, dev);
        const int32_t *fp = (int32_t *)at(a[3], "free_pages", i32, {F}, dev), *cu = (int32_t *)at(a[6], "cursor", i32, {1}, dev);
        auto call = [&](Out &offsets, Out &kv, Out &pos, Out &slots, Out &cout, Out &status) {
            launch([&] {
                return gdn_page_plan(nl, cl, bt, fp, cu, (int32_t *)offsets.ptr, (int32_t *)kv.ptr, (int32_t *)pos.ptr,
                                     (int32_t *)slots.ptr, (int32_t *)cout.ptr, (int32_t *)status.ptr, B, N, ps, M, F, stream(dev));
            });
            return tuple({&offsets, &kv, &pos, &slots, &cout, &status});
        };
        bool fresh = N <= kSharedN;
        for (int i = 7; i < 13; ++i) fresh = fresh && a[i] == Py_None;
        if (fresh) {
            const at::AutoDispatchBelowADInplaceOrView plain;  // (nothing here is differentiated)
            const at::Tensor all = allocate({2 * ((int64_t)N + 3) + 2 * ((int64_t)B + 4) + 8}, i32, dev);
            int64_t from = 0;
            Out offsets(all, B + 1, from), kv(all, B, from), pos(all, N, from), slots(all, N, from), cout(all, 1, from),
                status(all, 1, from);
            return call(offsets, kv, pos, slots, cout, status);
        }
        Out offsets(a[7], "offsets", i32, {B + 1}, dev), kv(a[8], "kv_lens", i32, {B}, dev), pos(a[9], "positions", i32, {N}, dev),
            slots(a[10], "slots", i32, {N}, dev), cout(a[11], "cursor_out", i32, {1}, dev), status(a[12], "status", i32, {1}, dev);
        return call(offsets, kv, pos, slots, cout, status);
    });
}

// (qkv, cos_sin, positions, H, HKV, D, q_weight, k_weight, eps, style, q, k, slots, k_cache, v_cache)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const at::Tensor &qkv = tensor_of(a[0], "qkv", 2);
        const c10::Device dev = cuda_device(qkv, "qkv");
        const at::ScalarType T = qkv.scalar_type();
        const int N = extent(qkv.size(0), "N"), H = whole(a[3], "H"), HKV = whole(a[4], "HKV"), D = whole(a[5], "D");
        const int dtype = activation(T), style = whole(a[9], "style");
        const float eps = real(a[8]);
        if (H < 1 || HKV < 1 || D < 1) throw Refusal{GDN_ERR_SHAPE, "head geometry must be positive"};
        int64_t stride;
        const void *base = rows(qkv, "qkv", T, {N, ((int64_t)H + 2 * (int64_t)HKV) * D}, dev, stride);
        const c10::cuda::CUDAGuard guard(dev);
        const bool cached = a[12] != Py_None;
        int max_pos = 0, R = 0, num_slots = 0;
        const void *table = nullptr;
        if (a[1] != Py_None) {
            const at::Tensor &t = tensor_of(a[1], "cos_sin", 2);
            max_pos = extent(t.size(0), "max_pos"), R = extent(t.size(1), "R");
            if (R > 0) table = at(a[1], "cos_sin", at::kFloat, {max_pos, R}, dev);
        }
        const void *pos = at(a[2], "positions", at::kInt, {N}, dev, true), *slots = at(a[12], "slots", at::kInt, {N}, dev, true);
        void *kc = nullptr, *vc = nullptr;
        if (cached) {
            if (a[13] == Py_None || a[14] == Py_None) throw Refusal{GDN_ERR_NULL, "slots need k_cache and v_cache"};
            const at::Tensor &c = tensor_of(a[13], "k_cache", 4);
            const int64_t pages = c.size(0), ps = c.size(1);
            num_slots = extent(pages * ps, "cache slots");
            kc = at(a[13], "k_cache", T, {pages, ps, HKV, D}, dev), vc = at(a[14], "v_cache", T, {pages, ps, HKV, D}, dev);
        }
        const void *qw = at(a[6], "q_weight", at::kFloat, {D}, dev, true), *kw = at(a[7], "k_weight", at::kFloat, {D}, dev, true);
        Out q(a[10], "q", T, {N, H, D}, dev);
        // with slots a packed k is only written when the caller gives one
        const bool packed = a[11] != Py_None || !cached;
        std::optional<Out> k;
        if (packed) k.emplace(a[11], "k", T, at::IntArrayRef({N, HKV, D}), dev);
        launch([&] {
            return gdn_qk_norm_rope(base, stride, (const float *)qw, (const float *)kw, eps, (const float *)table,
                                    (const int32_t *)pos, max_pos, (const int32_t *)slots, q.ptr, k ? k->ptr : nullptr, kc, vc,
                                    num_slots, N, H, HKV, D, R, style, dtype, stream(dev));
        });
        return tuple({&q, k ? &*k : nullptr});
    });
}

// (q, k, v, offsets, scale, out)
PyObject *attention_varlen(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor &q = tensor_of(a[0], "q", 3), &k = tensor_of(a[1], "k", 3), &v = tensor_of(a[2], "v", 3),
                         &o = tensor(a[3], "offsets");
        const c10::Device dev = cuda_device(q, "q");
        const at::ScalarType T = q.scalar_type();
        const int N = extent(q.size(0), "N"), H = extent(q.size(1), "H"), D = extent(q.size(2), "D"), HKV = extent(k.size(1), "HKV");
        const int B = extent(o.numel(), "B + 1") - 1;
        int64_t qs, ks, vs;
        const void *qp = rows(q, "q", T, {N, H, D}, dev, qs), *kp = rows(k, "k", T, {N, HKV, D}, dev, ks),
                   *vp = rows(v, "v", T, {N, HKV, D}, dev, vs);
        const int dtype = activation(T);
        const void *offsets = at(a[3], "offsets", at::kInt, {B + 1}, dev);
        const float scale = real(a[4]);
        const c10::cuda::CUDAGuard guard(dev);
        Out out(a[5], "out", T, {N, H, D}, dev);
        launch([&] {
            return gdn_attention_varlen(qp, kp, vp, (const int32_t *)offsets, out.ptr, B, N, H, HKV, D, qs, ks, vs, scale, dtype,
                                        stream(dev));
        });
        return out.give();
    });
}

// (q, k_cache, v_cache, block_table, kv_lens, offsets, max_q, scale, out, workspace)
PyObject *attention_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &q = tensor_of(a[0], "q", 3), &c = tensor_of(a[1], "k_cache", 4), &table = tensor_of(a[3], "block_table", 2);
        const c10::Device dev = cuda_device(q, "q");
        const at::ScalarType T = q.scalar_type();
        const int N = extent(q.size(0), "N"), H = extent(q.size(1), "H"), D = extent(q.size(2), "D");
        const int pages = extent(c.size(0), "num_pages"), ps = extent(c.size(1), "page_size"), HKV = extent(c.size(2), "HKV");
        const int B = extent(table.size(0), "B"), M = extent(table.size(1), "max_pages"), max_q = whole(a[6], "max_q");
        int64_t qs;
        const void *qp = rows(q, "q", T, {N, H, D}, dev, qs);
        const int dtype = activation(T);
        const float scale = real(a[7]);
        const void *kc = at(a[1], "k_cache", T, {pages, ps, HKV, D}, dev), *vc = at(a[2], "v_cache", T, {pages, ps, HKV, D}, dev);
        const int32_t *bt = (int32_t *)at(a[3], "block_table", at::kInt, {B, M}, dev), *kv = (int32_t *)at(a[4], "kv_lens", at::kInt, {B}, dev),
                      *of = (int32_t *)at(a[5], "offsets", at::kInt, {B + 1}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Out out(a[8], "out", T, {N, H, D}, dev);
        at::Tensor ws;
        if (a[9] == Py_None) {
            const size_t need = gdn_attention_paged_workspace_bytes(B, N, H, HKV, D, max_q);
            ws = allocate({(int64_t)(need > 256 ? need : 256)}, at::kByte, dev);
        } else {
            ws = tensor(a[9], "workspace");
            check(ws, "workspace", at::kByte, ws.sizes(), dev);
            if (!ws.is_contiguous()) throw Refusal{GDN_ERR_SHAPE, "workspace must be contiguous"};
        }
        launch([&] {
            return gdn_attention_paged(qp, kc, vc, bt, kv, of, out.ptr, B, N, H, HKV, D, ps, M, pages, max_q, qs, scale, dtype,
                                       ws.data_ptr(), (size_t)ws.numel(), stream(dev));
        });
        return out.give();
    });
}

// The heads, pages and tokens to a page of a 4-bit cache [num_pages, HKV, page_size * D * 9/16] bytes.
struct Kv4Cache {
    int pages, HKV, page_size;
    void *k, *v;
    const float *k_scale, *v_scale;
    Kv4Cache(PyObject *kc, PyObject *vc, PyObject *ks, PyObject *vs, int D, c10::Device dev) {
        const at::Tensor &c = tensor_of(kc, "k_cache", 3);
        pages = extent(c.size(0), "num_pages"), HKV = extent(c.size(1), "HKV");
        if (D < 16 || D % 16 != 0 || D > 256)
            throw Refusal{GDN_ERR_UNSUPPORTED, "head width D=" + std::to_string(D) + " is not a multiple of 16 up to 256"};
        const int64_t token = D / 16 * 9, bytes = c.size(2);
        if (bytes < 1 || bytes % token != 0)
            throw Refusal{GDN_ERR_SHAPE, "k_cache has " + std::to_string(bytes) + " bytes a page and head, not a multiple of " +
                                             std::to_string(token) + " (D * 9/16)"};
        page_size = extent(bytes / token, "page_size");
        k = at(kc, "k_cache", at::kByte, {pages, HKV, bytes}, dev), v = at(vc, "v_cache", at::kByte, {pages, HKV, bytes}, dev);
        k_scale = (const float *)at(ks, "k_scale", at::kFloat, {HKV}, dev, true);
        v_scale = (const float *)at(vs, "v_scale", at::kFloat, {HKV}, dev, true);
    }
};

// A workspace that was given, or a new one of `need` bytes.
at::Tensor workspace(PyObject *o, size_t need, c10::Device dev) {
    if (o == Py_None) return allocate({(int64_t)(need > 256 ? need : 256)}, at::kByte, dev);
    const at::Tensor &ws = tensor(o, "workspace");
    check(ws, "workspace", at::kByte, ws.sizes(), dev);
    if (!ws.is_contiguous()) throw Refusal{GDN_ERR_SHAPE, "workspace must be contiguous"};
    return ws;
}

// Bytes or truth values: pointer of a contiguous tensor of either type.
void *flags_at(PyObject *o, const char *name, at::IntArrayRef shape, c10::Device dev) {
    const bool truth = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kBool;
    return at(o, name, truth ? at::kBool : at::kByte, shape, dev);
}

// Device pointers of a sequence of contiguous CUDA tensors on one device, whose first dimension is `rows` (-1: that of the
// first tensor), and the bytes of a row of each.
struct Tensors {
    std::vector<void *> ptr;
    std::vector<int64_t> row_bytes;
    std::optional<c10::Device> dev;
    int64_t rows = -1;
    Tensors(PyObject *o, const char *name) {
        PyObject *seq = PySequence_Fast(o, "a sequence of tensors is expected");
        if (!seq) throw Raised{};
        try {
            for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i) {
                const std::string at = std::string(name) + "[" + std::to_string(i) + "]";
                const at::Tensor &t = tensor(PySequence_Fast_GET_ITEM(seq, i), at.c_str());
                if (!dev) dev = cuda_device(t, at.c_str());
                if (t.device() != *dev) throw Refusal{GDN_ERR_CUDA, at + " is on " + t.device().str() + ", expected " + dev->str()};
                if (t.dim() < 1) throw Refusal{GDN_ERR_SHAPE, at + " has no dimensions"};
                if (rows < 0) rows = t.size(0);
                if (t.size(0) != rows)
                    throw Refusal{GDN_ERR_SHAPE, at + " has " + std::to_string(t.size(0)) + " rows, expected " + std::to_string(rows)};
                if (!t.is_contiguous()) throw Refusal{GDN_ERR_SHAPE, at + " must be contiguous"};
                ptr.push_back(t.data_ptr());
                row_bytes.push_back(rows > 0 ? (int64_t)t.nbytes() / rows : 0);
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
        Py_DECREF(seq);
    }
};

// (k, v, slots, k_cache, v_cache, k_scale, v_scale, values, k_out, v_out)
PyObject *kv4_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &k = tensor_of(a[0], "k", 3), &v = tensor_of(a[1], "v", 3);
        const c10::Device dev = cuda_device(k, "k");
        const at::ScalarType T = k.scalar_type();
        const int N = extent(k.size(0), "N"), HKV = extent(k.size(1), "HKV"), D = extent(k.size(2), "D");
        int64_t ks, vs;
        const void *kp = rows(k, "k", T, {N, HKV, D}, dev, ks), *vp = rows(v, "v", T, {N, HKV, D}, dev, vs);
        const int dtype = activation(T);
        const Kv4Cache c(a[3], a[4], a[5], a[6], D, dev);
        if (c.HKV != HKV)
            throw Refusal{GDN_ERR_SHAPE, "k_cache has " + std::to_string(c.HKV) + " heads, expected " + std::to_string(HKV)};
        const int32_t *slots = (int32_t *)at(a[2], "slots", at::kInt, {N}, dev);
        const int wanted = PyObject_IsTrue(a[7]);
        if (wanted < 0) throw Raised{};
        const c10::cuda::CUDAGuard guard(dev);
        std::optional<Out> ko, vo;
        if (wanted || a[8] != Py_None || a[9] != Py_None)
            ko.emplace(a[8], "k_out", T, at::IntArrayRef({N, HKV, D}), dev), vo.emplace(a[9], "v_out", T, at::IntArrayRef({N, HKV, D}), dev);
        launch([&] {
            return gdn_kv4_write(kp, vp, ks, vs, slots, c.k_scale, c.v_scale, c.k, c.v, ko ? ko->ptr : nullptr, vo ? vo->ptr : nullptr, N,
                                 HKV, D, c.page_size, c.pages, dtype, stream(dev));
        });
        return tuple({ko ? &*ko : nullptr, vo ? &*vo : nullptr});
    });
}

// (q, k_cache, v_cache, block_table, kv_lens, offsets, max_q, k_scale, v_scale, scale, out, workspace)
PyObject *attention_paged_kv4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const at::Tensor &q = tensor_of(a[0], "q", 3), &table = tensor_of(a[3], "block_table", 2);
        const c10::Device dev = cuda_device(q, "q");
        const at::ScalarType T = q.scalar_type();
        const int N = extent(q.size(0), "N"), H = extent(q.size(1), "H"), D = extent(q.size(2), "D");
        const int B = extent(table.size(0), "B"), M = extent(table.size(1), "max_pages"), max_q = whole(a[6], "max_q");
        int64_t qs;
        const void *qp = rows(q, "q", T, {N, H, D}, dev, qs);
        const int dtype = activation(T);
        const Kv4Cache c(a[1], a[2], a[7], a[8], D, dev);
        const float scale = real(a[9]);
        const int32_t *bt = (int32_t *)at(a[3], "block_table", at::kInt, {B, M}, dev), *kv = (int32_t *)at(a[4], "kv_lens", at::kInt, {B}, dev),
                      *of = (int32_t *)at(a[5], "offsets", at::kInt, {B + 1}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Out out(a[10], "out", T, {N, H, D}, dev);
        const at::Tensor ws = workspace(a[11], gdn_attention_paged_kv4_workspace_bytes(B, N, H, c.HKV, D, max_q), dev);
        launch([&] {
            return gdn_attention_paged_kv4(qp, c.k, c.v, c.k_scale, c.v_scale, bt, kv, of, out.ptr, B, N, H, c.HKV, D, c.page_size, M,
                                           c.pages, max_q, qs, scale, dtype, ws.data_ptr(), (size_t)ws.numel(), stream(dev));
        });
        return out.give();
    });
}

// (logits, scores, n, finished, end_token, keep_rows, tokens, parents, scores_out, finished_out, workspace)
PyObject *beam_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Tensor &x = tensor_of(a[0], "logits", 2), &scores = tensor_of(a[1], "scores", 2);
        const c10::Device dev = cuda_device(x, "logits");
        const at::ScalarType T = x.scalar_type();
        const int G = extent(scores.size(0), "G"), K = extent(scores.size(1), "K"), V = extent(x.size(1), "V");
        const int many = a[2] == Py_None ? K : whole(a[2], "n"), end = whole(a[4], "end_token"), keep = PyObject_IsTrue(a[5]);
        if (keep < 0) throw Raised{};
        if (G < 1 || K < 1 || V < 1 || many < 1) throw Refusal{GDN_ERR_SHAPE, "groups, beams, vocabulary and n must be positive"};
        int64_t stride;
        const void *xp = rows(x, "logits", T, {(int64_t)G * K, V}, dev, stride);
        const int dtype = activation(T);
        const float *sp = (const float *)at(a[1], "scores", at::kFloat, {G, K}, dev);
        const uint8_t *done = a[3] == Py_None ? nullptr : (const uint8_t *)flags_at(a[3], "finished", {G, K}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Out tokens(a[6], "tokens", at::kInt, {G, many}, dev), parents(a[7], "parents", at::kInt, {G, many}, dev),
            so(a[8], "scores_out", at::kFloat, {G, many}, dev);
        std::optional<Out> fo;
        if (a[9] != Py_None) {
            const bool truth = THPVariable_Check(a[9]) && THPVariable_Unpack(a[9]).scalar_type() == at::kBool;
            fo.emplace(a[9], "finished_out", truth ? at::kBool : at::kByte, at::IntArrayRef({G, many}), dev);
        } else if (done) {
            fo.emplace(a[9], "finished_out", THPVariable_Unpack(a[3]).scalar_type(), at::IntArrayRef({G, many}), dev);
        }
        const at::Tensor ws = workspace(a[10], gdn_beam_select_workspace_bytes(G, K, V, many), dev);
        launch([&] {
            return gdn_beam_select(xp, stride, sp, done, end, keep, (int32_t *)tokens.ptr, (int32_t *)parents.ptr, (float *)so.ptr,
                                   fo ? (uint8_t *)fo->ptr : nullptr, G, K, V, many, dtype, ws.data_ptr(), (size_t)ws.numel(), stream(dev));
        });
        return tuple({&tokens, &parents, &so, fo ? &*fo : nullptr});
    });
}

PyObject *none() {
    Py_INCREF(Py_None);
    return Py_None;
}

// (states, parents)
PyObject *state_reorder(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 2, [&] {
        const Tensors t(a[0], "states");
        if (t.ptr.empty()) return none();
        const int B = extent(t.rows, "B"), count = extent((int64_t)t.ptr.size(), "states");
        const int32_t *parents = (int32_t *)at(a[1], "parents", at::kInt, {B}, *t.dev);
        const c10::cuda::CUDAGuard guard(*t.dev);
        launch([&] { return gdn_state_reorder(t.ptr.data(), t.row_bytes.data(), count, parents, B, stream(*t.dev)); });
        return none();
    });
}

// (parents, kv_lens, block_table, free_pages, page_size, num_pages, cursor, table_out, kv_lens_out, copies, cursor_out, status,
//  workspace)
PyObject *page_fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const at::Tensor &parents = tensor_of(a[0], "parents", 1), &table = tensor_of(a[2], "block_table", 2), &free = tensor(a[3], "free_pages");
        const c10::Device dev = cuda_device(table, "block_table");
        const int B = extent(table.size(0), "B"), M = extent(table.size(1), "max_pages"), R = extent(parents.size(0), "B_out"),
                  F = extent(free.numel(), "n_free"), ps = whole(a[4], "page_size"), pages = whole(a[5], "num_pages");
        const auto i32 = at::kInt;
        const int32_t *pp = (int32_t *)at(a[0], "parents", i32, {R}, dev), *kv = (int32_t *)at(a[1], "kv_lens", i32, {B}, dev),
                      *bt = (int32_t *)at(a[2], "block_table", i32, {B, M}, dev), *cu = (int32_t *)at(a[6], "cursor", i32, {1}, dev);
        int32_t *fp = (int32_t *)at(a[3], "free_pages", i32, {F}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Out to(a[7], "table_out", i32, {R, M}, dev), ko(a[8], "kv_lens_out", i32, {R}, dev), copies(a[9], "copies", i32, {R, 2}, dev),
            co(a[10], "cursor_out", i32, {1}, dev), status(a[11], "status", i32, {1}, dev);
        const at::Tensor ws = workspace(a[12], gdn_page_fork_workspace_bytes(B, M, pages), dev);
        launch([&] {
            return gdn_page_fork(pp, kv, bt, fp, cu, (int32_t *)to.ptr, (int32_t *)ko.ptr, (int32_t *)copies.ptr, (int32_t *)co.ptr,
                                 (int32_t *)status.ptr, B, R, ps, M, pages, F, ws.data_ptr(), (size_t)ws.numel(), stream(dev));
        });
        return tuple({&to, &ko, &copies, &co, &status});
    });
}

// (kv_lens, block_table, page_size, num_pages, table_out, copies, free_pages, cursor_out, status, workspace)
PyObject *page_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &table = tensor_of(a[1], "block_table", 2);
        const c10::Device dev = cuda_device(table, "block_table");
        const int B = extent(table.size(0), "B"), M = extent(table.size(1), "max_pages"), ps = whole(a[2], "page_size"),
                  pages = whole(a[3], "num_pages");
        if (pages < 1) throw Refusal{GDN_ERR_SHAPE, "num_pages must be positive"};
        const auto i32 = at::kInt;
        const int32_t *kv = (int32_t *)at(a[0], "kv_lens", i32, {B}, dev), *bt = (int32_t *)at(a[1], "block_table", i32, {B, M}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Out to(a[4], "table_out", i32, {B, M}, dev), copies(a[5], "copies", i32, {pages / 2, 2}, dev), free(a[6], "free_pages", i32, {pages}, dev),
            co(a[7], "cursor_out", i32, {1}, dev), status(a[8], "status", i32, {1}, dev);
        const at::Tensor ws = workspace(a[9], gdn_page_compact_workspace_bytes(pages), dev);
        launch([&] {
            return gdn_page_compact(kv, bt, (int32_t *)to.ptr, (int32_t *)copies.ptr, (int32_t *)free.ptr, (int32_t *)co.ptr,
                                    (int32_t *)status.ptr, B, ps, M, pages, ws.data_ptr(), (size_t)ws.numel(), stream(dev));
        });
        return tuple({&to, &copies, &free, &co, &status});
    });
}

// (caches, copies)
PyObject *page_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 2, [&] {
        const Tensors t(a[0], "caches");
        if (t.ptr.empty()) return none();
        const at::Tensor &copies = tensor_of(a[1], "copies", 2);
        const int pairs = extent(copies.size(0), "copies"), pages = extent(t.rows, "num_pages"), count = extent((int64_t)t.ptr.size(), "caches");
        const int32_t *cp = (int32_t *)at(a[1], "copies", at::kInt, {pairs, 2}, *t.dev);
        const c10::cuda::CUDAGuard guard(*t.dev);
        launch([&] { return gdn_page_copy(t.ptr.data(), t.row_bytes.data(), count, cp, pairs, pages, stream(*t.dev)); });
        return none();
    });
}

// (GdnError)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 1, [&] {
        Py_INCREF(a[0]);
        Py_XDECREF(g_error);
        g_error = a[0];
        Py_INCREF(Py_None);
        return Py_None;
    });
}

#define CALL(f) (PyCFunction)(void *)f, METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"init", CALL(init)},
                           {"page_plan", CALL(page_plan)},
                           {"qk_norm_rope", CALL(qk_norm_rope)},
                           {"attention_varlen", CALL(attention_varlen)},
                           {"attention_paged", CALL(attention_paged)},
                           {"kv4_write", CALL(kv4_write)},
                           {"attention_paged_kv4", CALL(attention_paged_kv4)},
                           {"beam_select", CALL(beam_select)},
                           {"state_reorder", CALL(state_reorder)},
                           {"page_fork", CALL(page_fork)},
                           {"page_compact", CALL(page_compact)},
                           {"page_copy", CALL(page_copy)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
