// Python half of the serving operators: checks of tensors and the call of the
// C ABI (include/fa.h), as a CPython module.
//
// These calls are made once per layer and step on small tensors and take a few
// microseconds on the GPU; checked and marshalled in Python they took 7 to
// 14 us on the host of a GB300, here 2 to 4.  binding.py has their signatures
// and documentation; every function here takes its arguments by position
// (None where an optional one is absent), raises ValueError or TypeError for
// tensors that do not fit, and returns the outputs, or the status of the C
// call as an int where it is not FA_OK.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/fa.h"

namespace {

using at::Tensor;

struct BadValue : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct BadType : std::runtime_error {
    using std::runtime_error::runtime_error;
};

const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) throw BadType(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// Index of the CUDA device that holds t, which has to be the current one.
int device_of(const char* name, const Tensor& t) {
    if (!t.is_cuda()) throw BadValue(std::string(name) + " must be a CUDA tensor");
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device())
        throw BadValue(std::string(name) + " is on cuda:" + std::to_string(dev) +
                       ", which is not the current device");
    return dev;
}

bool on(const Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

bool has_shape(const Tensor& t, std::initializer_list<int64_t> shape) {
    return t.sizes() == at::IntArrayRef(shape);
}

std::string text(at::IntArrayRef shape) {
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

// A contiguous tensor of the given type and shape that a kernel reads, or
// reads and writes in place.
void* dense(const char* name, const Tensor& t, at::ScalarType type,
            std::initializer_list<int64_t> shape, int dev) {
    if (t.scalar_type() != type || !has_shape(t, shape) || !on(t, dev) || !t.is_contiguous())
        throw BadValue(std::string(name) + " must be a contiguous " + c10::toString(type) +
                       " tensor " + text(at::IntArrayRef(shape)) + " on cuda:" +
                       std::to_string(dev) + ", not " + c10::toString(t.scalar_type()) + " " +
                       text(t.sizes()) + " on " + t.device().str());
    return t.data_ptr();
}
int* ints(const char* name, const Tensor& t, std::initializer_list<int64_t> shape, int dev) {
    return static_cast<int*>(dense(name, t, at::kInt, shape, dev));
}
int* ints_or_null(const char* name, PyObject* o, std::initializer_list<int64_t> shape, int dev) {
    return o == Py_None ? nullptr : ints(name, tensor(name, o), shape, dev);
}

// The stream of a call, and whether it is another than the current one.
struct Stream {
    fa_stream_t handle;
    bool other;
    operator fa_stream_t() const { return handle; }
};
Stream stream_of(PyObject* handle, int dev) {
    const cudaStream_t current =
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    if (handle == Py_None) return {reinterpret_cast<fa_stream_t>(current), false};
    void* p = PyLong_AsVoidPtr(handle);
    if (p == nullptr && PyErr_Occurred()) {
        PyErr_Clear();
        throw BadType("stream must be a CUDA stream");
    }
    return {static_cast<fa_stream_t>(p), p != reinterpret_cast<void*>(current)};
}

c10::cuda::CUDAStream torch_stream(const Stream& s, int dev) {
    const auto d = static_cast<c10::DeviceIndex>(dev);
    return s.other ? c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(s.handle), d)
                   : c10::cuda::getCurrentCUDAStream(d);
}

// A new contiguous tensor for a call on `stream` (without the dispatcher: 0.5 us
// where at::empty takes 1.5).  Its memory comes from that stream's pool, so that
// nothing still at work on the current stream uses it; and where that is another
// stream the allocator is told of the current one, which is to read it: the
// caller may drop it at any time.
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev, const Stream& stream) {
    const c10::Device device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev));
    if (!stream.other) return at::detail::empty_cuda(shape, type, device, std::nullopt);
    Tensor t;
    {
        const c10::cuda::CUDAStreamGuard guard(torch_stream(stream, dev));
        t = at::detail::empty_cuda(shape, type, device, std::nullopt);
    }
    if (t.numel() > 0)
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(),
                                                      c10::cuda::getCurrentCUDAStream(device.index()));
    return t;
}

// An input as a kernel on `stream` reads it: copied there where it is on the
// device and not contiguous (the copy's memory is of that stream's pool, so that
// it may go as soon as the call is enqueued).
Tensor laid_out(const Tensor& t, int dev, const Stream& stream) {
    if (!on(t, dev) || t.is_contiguous()) return t;
    const c10::cuda::CUDAStreamGuard guard(torch_stream(stream, dev));
    return t.clone(at::MemoryFormat::Contiguous);
}

// Sizes beyond int are refused here rather than cut.
int small(int64_t n) {
    if (n > INT32_MAX) throw BadValue("a dimension exceeds 2^31 - 1");
    return static_cast<int>(n);
}
int whole(const char* name, PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw BadType(std::string(name) + " must be a whole number");
    }
    if (x > INT32_MAX || x < INT32_MIN) throw BadValue(std::string(name) + " is out of range");
    return static_cast<int>(x);
}
float scale_of(PyObject* o, int64_t d) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw BadType("scale must be a number");
    }
    return static_cast<float>(x);
}

int truth(const char* name, PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
        PyErr_Clear();
        throw BadType(std::string(name) + " must be true or false");
    }
    return x;
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) throw BadType("wrong number of arguments");
}

PyObject* status_or(fa_status st, PyObject* value) {
    if (st == FA_OK) return value;
    Py_DECREF(value);
    return PyLong_FromLong(st);
}
PyObject* pair(const Tensor& a, const Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = THPVariable_Wrap(b);
    PyObject* t = PyTuple_Pack(2, x, y);
    Py_DECREF(x);
    Py_DECREF(y);
    return t;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(a, n);
    } catch (const BadValue& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const BadType& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (...) {   // torch's own (out of memory, ...) as what torch raises for them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// ---------------------------------------------------------- attention ----

// q [B, Hq, n, d], keys and values of one shape [*, Hkv, m, d], sinks, out and
// lse of an attention call.  Lengths, tables and sinks come in any layout.
struct Attention {
    Tensor q, k, v, out, lse;
    const float* sinks = nullptr;
    int dev;
    int B, Hq, n, d;

    Stream stream;
    Tensor held[4];   // copies of small inputs
    int n_held = 0;

    const Tensor& hold(const Tensor& t) {
        if (t.is_contiguous()) return t;
        held[n_held] = laid_out(t, dev, stream);
        return held[n_held++];
    }
    int* lengths(const char* name, PyObject* o) {   // int32 [B], or nullptr for None
        return o == Py_None ? nullptr : ints(name, hold(tensor(name, o)), {B}, dev);
    }

    // as_paged: with the contract of the paged decode call of the plain kind, which
    // takes q and the caches in any layout too and raises ValueError for their type
    Attention(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* sinks_, PyObject* out_,
              PyObject* lse_, PyObject* stream_, bool as_paged = false)
        : q(tensor("q", q_)), k(tensor("k", k_)), v(tensor("v", v_)), dev(device_of("q", q)),
          stream(stream_of(stream_, dev)) {
        if (as_paged)
            for (Tensor* t : {&q, &k, &v}) *t = laid_out(*t, dev, stream);
        const char* names[3] = {"q", "k", "v"};
        const Tensor* all[3] = {&q, &k, &v};
        for (int i = 0; i < 3; ++i) {
            if (all[i]->scalar_type() != at::kBFloat16) {
                if (as_paged) throw BadValue("q and the caches must be bf16");
                throw BadType(std::string(names[i]) + " must be bfloat16");
            }
            if (!on(*all[i], dev) || all[i]->dim() != 4 || !all[i]->is_contiguous())
                throw BadValue(std::string(names[i]) +
                               " must be a contiguous 4-D tensor on cuda:" + std::to_string(dev));
        }
        if (v.sizes() != k.sizes() || k.size(3) != q.size(3))
            throw BadValue("shape mismatch q" + text(q.sizes()) + " k" + text(k.sizes()) + " v" +
                           text(v.sizes()));
        B = small(q.size(0)), Hq = small(q.size(1)), n = small(q.size(2)), d = small(q.size(3));
        if (sinks_ != Py_None)
            sinks = static_cast<const float*>(
                dense("sinks", hold(tensor("sinks", sinks_)), at::kFloat, {Hq}, dev));
        if (out_ == Py_None) {
            out = fresh(q.sizes(), at::kBFloat16, dev, stream);
        } else {
            out = tensor("out", out_);
            dense("out", out, at::kBFloat16, {B, Hq, n, d}, dev);
        }
        if (lse_ == Py_None) {
            lse = fresh({B, Hq, n}, at::kFloat, dev, stream);
        } else {
            lse = tensor("lse", lse_);
            dense("lse", lse, at::kFloat, {B, Hq, n}, dev);
        }
    }
    float* lse_ptr() const { return static_cast<float*>(lse.data_ptr()); }
    PyObject* result(fa_status st) const { return status_or(st, pair(out, lse)); }
};

struct Pages {
    const int* table;
    int max_pages, page_size, num_pages, hkv;

    Pages(Attention& c, PyObject* table_) {
        const Tensor& t = c.hold(tensor("block_table", table_));
        if (t.dim() != 2) throw BadValue("block_table must be [B, max_pages]");
        max_pages = small(t.size(1));
        table = ints("block_table", t, {c.B, t.size(1)}, c.dev);
        num_pages = small(c.k.size(0));
        hkv = small(c.k.size(1));
        page_size = small(c.k.size(2));
    }
};

struct TreeMask {
    const unsigned int* words;
    int shared;
    const int* lens;

    TreeMask(Attention& c, PyObject* mask_, PyObject* lens_) {
        const Tensor& m = tensor("tree_mask", mask_);
        const int64_t w = (c.n + 31) / 32;
        shared = m.dim() == 2;
        words = reinterpret_cast<const unsigned int*>(
            shared ? ints("tree_mask", m, {c.n, w}, c.dev)
                   : ints("tree_mask", m, {c.B, c.n, w}, c.dev));
        lens = c.lengths("tree_lens", lens_);
    }
};

void same_batch(const Attention& c) {
    if (c.k.size(0) != c.B) throw BadValue("k and v must have q's batch");
}

// q, k, v, tree_mask, scale, seqlens_k, tree_lens, sinks, out, lse, stream
PyObject* decode_tree(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 11);
    Attention c(a[0], a[1], a[2], a[7], a[8], a[9], a[10]);
    same_batch(c);
    const TreeMask m(c, a[3], a[6]);
    return c.result(fa_fwd_decode_tree(
        c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.out.data_ptr(), c.lse_ptr(), c.B, c.Hq,
        small(c.k.size(1)), c.n, small(c.k.size(2)), c.lengths("seqlens_k", a[5]),
        m.words, m.shared, m.lens, c.d, scale_of(a[4], c.d), c.sinks, c.stream));
}

// q, k_cache, v_cache, block_table, seqlens_k, tree_mask, scale, tree_lens,
// sinks, out, lse, stream
PyObject* decode_tree_paged(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 12);
    Attention c(a[0], a[1], a[2], a[8], a[9], a[10], a[11]);
    const Pages p(c, a[3]);
    const TreeMask m(c, a[5], a[7]);
    return c.result(fa_fwd_decode_tree_paged(
        c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.out.data_ptr(), c.lse_ptr(), c.B, c.Hq,
        p.hkv, c.n, ints("seqlens_k", c.hold(tensor("seqlens_k", a[4])), {c.B}, c.dev), p.table,
        p.max_pages, p.page_size, p.num_pages, m.words, m.shared, m.lens, c.d,
        scale_of(a[6], c.d), c.sinks, c.stream));
}

// q, k, v, scale, causal, seqlens_k, out, lse, stream, window, sinks, first
PyObject* decode_first(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 12);
    Attention c(a[0], a[1], a[2], a[10], a[6], a[7], a[8]);
    same_batch(c);
    return c.result(fa_fwd_decode_first(
        c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.out.data_ptr(), c.lse_ptr(), c.B, c.Hq,
        small(c.k.size(1)), c.n, small(c.k.size(2)), c.lengths("seqlens_k", a[5]),
        c.d, scale_of(a[3], c.d), truth("causal", a[4]), whole("window", a[9]),
        whole("first", a[11]), c.sinks, c.stream));
}

// q, k_cache, v_cache, block_table, seqlens_k, scale, causal, out, lse, stream,
// window, sinks, first
PyObject* decode_paged_first(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 13);
    Attention c(a[0], a[1], a[2], a[11], a[7], a[8], a[9], true);
    const Pages p(c, a[3]);
    return c.result(fa_fwd_decode_paged_first(
        c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.out.data_ptr(), c.lse_ptr(), c.B, c.Hq,
        p.hkv, c.n, ints("seqlens_k", c.hold(tensor("seqlens_k", a[4])), {c.B}, c.dev), p.table,
        p.max_pages, p.page_size, p.num_pages, c.d, scale_of(a[5], c.d),
        truth("causal", a[6]), whole("window", a[10]), whole("first", a[12]), c.sinks, c.stream));
}

// parents, out, stream
PyObject* tree_mask(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 3);
    const Tensor& parents = tensor("parents", a[0]);
    const int dev = device_of("parents", parents);
    if (parents.dim() != 2) throw BadValue("parents must be [B, T]");
    const int64_t B = parents.size(0), T = parents.size(1), W = (T + 31) / 32;
    const Stream stream = stream_of(a[2], dev);
    Tensor out = a[1] == Py_None ? fresh({B, T, W}, at::kInt, dev, stream)
                                 : tensor("out", a[1]);
    const fa_status st = fa_tree_mask(
        ints("parents", parents, {B, T}, dev),
        reinterpret_cast<unsigned int*>(ints("out", out, {B, T, W}, dev)), small(B), small(T), stream);
    return status_or(st, THPVariable_Wrap(out));
}

// --------------------------------------------------------- page tables ----

struct Table {
    int dev, num_pages, max_pages, batch;
    int *refs, *table, *lens;

    Table(PyObject* refs_, PyObject* table_, PyObject* lens_) {
        const Tensor& t = tensor("block_table", table_);
        const Tensor& r = tensor("refs", refs_);
        dev = device_of("block_table", t);
        if (t.dim() != 2) throw BadValue("block_table must be [B, max_pages]");
        batch = small(t.size(0));
        max_pages = small(t.size(1));
        num_pages = small(r.numel());
        refs = ints("refs", r, {num_pages}, dev);
        table = ints("block_table", t, {batch, max_pages}, dev);
        lens = ints("seqlens", tensor("seqlens", lens_), {batch}, dev);
    }
    Tensor status(PyObject* o, const Stream& stream) const {
        Tensor t = o == Py_None ? fresh({1}, at::kInt, dev, stream) : tensor("status", o);
        ints("status", t, {1}, dev);
        return t;
    }
};

// refs, block_table, seqlens, src, dst, status, stream
PyObject* cache_fork(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 7);
    const Table t(a[0], a[1], a[2]);
    const Tensor& src = tensor("src", a[3]);
    const Stream stream = stream_of(a[6], t.dev);
    const Tensor status = t.status(a[5], stream);
    const int64_t m = src.numel();
    const fa_status st = fa_cache_fork(
        t.refs, t.num_pages, t.table, t.max_pages, t.lens, t.batch, ints("src", src, {m}, t.dev),
        ints("dst", tensor("dst", a[4]), {m}, t.dev), small(m),
        static_cast<int*>(status.data_ptr()), stream);
    return status_or(st, THPVariable_Wrap(status));
}

// refs, block_table, seqlens, extra, page_size, copies, status, stream
PyObject* cache_reserve(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 8);
    const Table t(a[0], a[1], a[2]);
    const Stream stream = stream_of(a[7], t.dev);
    const Tensor status = t.status(a[6], stream);
    const Tensor copies =
        a[5] == Py_None ? fresh({t.batch, 3}, at::kInt, t.dev, stream) : tensor("copies", a[5]);
    const fa_status st = fa_cache_reserve(
        t.refs, t.num_pages, t.table, t.max_pages, t.lens, t.batch,
        ints("extra", tensor("extra", a[3]), {t.batch}, t.dev), whole("page_size", a[4]),
        ints("copies", copies, {t.batch, 3}, t.dev), static_cast<int*>(status.data_ptr()),
        stream);
    return status_or(st, pair(copies, status));
}

// refs, block_table, seqlens, rows, stream
PyObject* cache_free(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 5);
    const Table t(a[0], a[1], a[2]);
    const Tensor& rows = tensor("rows", a[3]);
    const int64_t m = rows.numel();
    return PyLong_FromLong(fa_cache_free(t.refs, t.num_pages, t.table, t.max_pages, t.lens, t.batch,
                                         ints("rows", rows, {m}, t.dev), small(m),
                                         stream_of(a[4], t.dev)));
}

// --------------------------------------------------------- page contents ----

struct Caches {
    int dev, num_pages, hkv, page_size, d;
    void *k, *v;

    Caches(PyObject* k_, PyObject* v_) {
        const Tensor& kc = tensor("k_cache", k_);
        const Tensor& vc = tensor("v_cache", v_);
        dev = device_of("k_cache", kc);
        if (kc.scalar_type() != at::kBFloat16 || vc.scalar_type() != at::kBFloat16 ||
            kc.dim() != 4 || vc.sizes() != kc.sizes() || !on(vc, dev) || !kc.is_contiguous() ||
            !vc.is_contiguous())
            throw BadValue("the caches must be contiguous bf16 tensors of one shape "
                           "[num_pages, Hkv, page_size, d] on cuda:" +
                           std::to_string(dev));
        num_pages = small(kc.size(0)), hkv = small(kc.size(1));
        page_size = small(kc.size(2)), d = small(kc.size(3));
        k = kc.data_ptr();
        v = vc.data_ptr();
    }
};

// New rows [B, Hkv, n, d] of any strides that are multiples of 8 elements over
// a contiguous last dimension; others are copied first, on the call's stream
// (whose pool the copy then belongs to: it may go as soon as the call is
// enqueued).
struct Rows {
    Tensor t;
    long long strides[3];

    Rows(const char* name, PyObject* o, const Caches& c, int64_t B, int64_t n, const Stream& stream)
        : t(tensor(name, o)) {
        if (t.scalar_type() != at::kBFloat16 || !has_shape(t, {B, c.hkv, n, c.d}) || !on(t, c.dev))
            throw BadValue(std::string(name) + " must be a bf16 tensor " +
                           text({B, c.hkv, n, c.d}) + " on cuda:" + std::to_string(c.dev));
        const bool fits = t.stride(3) == 1 &&
                          ((t.stride(0) | t.stride(1) | t.stride(2)) & 7) == 0 &&
                          (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15) == 0;
        if (!fits) {
            const c10::cuda::CUDAStreamGuard guard(torch_stream(stream, c.dev));
            t = t.clone(at::MemoryFormat::Contiguous);
        }
        for (int i = 0; i < 3; ++i) strides[i] = t.stride(i);
    }
};

// k_cache, v_cache, block_table, seqlens, k_new, v_new, n_new, copies, stream
PyObject* cache_append(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 9);
    const Caches c(a[0], a[1]);
    const Tensor& table = tensor("block_table", a[2]);
    const Tensor& kn = tensor("k_new", a[4]);
    if (table.dim() != 2 || kn.dim() != 4)
        throw BadValue("block_table must be [B, max_pages], k_new and v_new [B, Hkv, n, d]");
    const int64_t B = table.size(0), m = kn.size(2);
    const Stream stream = stream_of(a[8], c.dev);
    const Rows k("k_new", a[4], c, B, m, stream), v("v_new", a[5], c, B, m, stream);
    return PyLong_FromLong(fa_cache_append(
        c.k, c.v, c.num_pages, c.hkv, c.page_size, c.d,
        ints("block_table", table, {B, table.size(1)}, c.dev), small(table.size(1)),
        ints("seqlens", tensor("seqlens", a[3]), {B}, c.dev), small(B), k.t.data_ptr(), k.strides,
        v.t.data_ptr(), v.strides, small(m), ints_or_null("n_new", a[6], {B}, c.dev),
        ints_or_null("copies", a[7], {B, 3}, c.dev), stream));
}

// k_cache, v_cache, copies, stream
PyObject* cache_copy(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 4);
    const Caches c(a[0], a[1]);
    const Tensor& copies = tensor("copies", a[2]);
    if (copies.dim() != 2) throw BadValue("copies must be [n, 3]");
    const int64_t m = copies.size(0);
    return PyLong_FromLong(fa_cache_copy(c.k, c.v, c.num_pages, c.hkv, c.page_size, c.d,
                                         ints("copies", copies, {m, 3}, c.dev), small(m),
                                         stream_of(a[3], c.dev)));
}

// k_cache, v_cache, block_table, start, keep, n_keep, stream
PyObject* cache_compact(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 7);
    const Caches c(a[0], a[1]);
    const Tensor& table = tensor("block_table", a[2]);
    const Tensor& keep = tensor("keep", a[4]);
    if (table.dim() != 2 || keep.dim() != 2)
        throw BadValue("block_table must be [B, max_pages], keep [B, n]");
    const int64_t B = table.size(0), m = keep.size(1);
    return PyLong_FromLong(fa_cache_compact(
        c.k, c.v, c.num_pages, c.hkv, c.page_size, c.d,
        ints("block_table", table, {B, table.size(1)}, c.dev), small(table.size(1)),
        ints("start", tensor("start", a[3]), {B}, c.dev), small(B),
        ints("keep", keep, {B, m}, c.dev), small(m),
        ints("n_keep", tensor("n_keep", a[5]), {B}, c.dev), stream_of(a[6], c.dev)));
}

#define ENTRY(f) \
    {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    ENTRY(decode_tree), ENTRY(decode_tree_paged), ENTRY(decode_first), ENTRY(decode_paged_first),
    ENTRY(tree_mask),   ENTRY(cache_fork),        ENTRY(cache_reserve), ENTRY(cache_free),
    ENTRY(cache_append), ENTRY(cache_copy),       ENTRY(cache_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, kMethods,
                       nullptr,               nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&kModule); }
