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
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>

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
    // kv: type of the keys and values
    Attention(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* sinks_, PyObject* out_,
              PyObject* lse_, PyObject* stream_, bool as_paged = false,
              at::ScalarType kv = at::kBFloat16)
        : q(tensor("q", q_)), k(tensor("k", k_)), v(tensor("v", v_)), dev(device_of("q", q)),
          stream(stream_of(stream_, dev)) {
        if (as_paged)
            for (Tensor* t : {&q, &k, &v}) *t = laid_out(*t, dev, stream);
        const char* names[3] = {"q", "k", "v"};
        const Tensor* all[3] = {&q, &k, &v};
        for (int i = 0; i < 3; ++i) {
            if (all[i]->scalar_type() != (i == 0 ? at::kBFloat16 : kv)) {
                if (kv != at::kBFloat16)
                    throw BadValue("q must be bf16 and the caches " + std::string(c10::toString(kv)));
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

    Caches(PyObject* k_, PyObject* v_, at::ScalarType type = at::kBFloat16) {
        const Tensor& kc = tensor("k_cache", k_);
        const Tensor& vc = tensor("v_cache", v_);
        dev = device_of("k_cache", kc);
        if (kc.scalar_type() != type || vc.scalar_type() != type ||
            kc.dim() != 4 || vc.sizes() != kc.sizes() || !on(vc, dev) || !kc.is_contiguous() ||
            !vc.is_contiguous())
            throw BadValue(std::string("the caches must be contiguous ") +
                           (type == at::kBFloat16 ? "bf16" : c10::toString(type)) +
                           " tensors of one shape [num_pages, Hkv, page_size, d] on cuda:" +
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
bool rows_fit(const Tensor& t) {
    const int64_t last = t.dim() - 1;
    int64_t all = 0;
    for (int64_t i = 0; i < last; ++i) all |= t.stride(i);
    return t.stride(last) == 1 && (all & 7) == 0 && (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15) == 0;
}
struct Rows {
    Tensor t;
    long long strides[3];

    Rows(const char* name, PyObject* o, const Caches& c, int64_t heads, int64_t B, int64_t n,
         const Stream& stream)
        : t(tensor(name, o)) {
        if (t.scalar_type() != at::kBFloat16 || !has_shape(t, {B, heads, n, c.d}) || !on(t, c.dev))
            throw BadValue(std::string(name) + " must be a bf16 tensor " +
                           text({B, heads, n, c.d}) + " on cuda:" + std::to_string(c.dev));
        if (!rows_fit(t)) {
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
    const Rows k("k_new", a[4], c, c.hkv, B, m, stream), v("v_new", a[5], c, c.hkv, B, m, stream);
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

// ---------------------------------------------------- rotated positions ----

float factor_of(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw BadType("factor must be a number");
    }
    return static_cast<float>(x);
}

// Frequencies int64 [rot / 2], or none.
struct Freqs {
    Tensor t;
    const long long* p = nullptr;
    int rot = 0;

    Freqs(PyObject* o, int dev, const Stream& stream, bool optional) {
        if (o == Py_None && optional) return;
        t = laid_out(tensor("freqs", o), dev, stream);
        if (t.dim() != 1) throw BadValue("freqs must be [rot / 2]");
        p = static_cast<const long long*>(dense("freqs", t, at::kLong, {t.size(0)}, dev));
        rot = small(2 * t.size(0));
    }
};

// Positions int32 [B, n], or [n] for every batch entry.
struct Positions {
    Tensor t;
    const int* p = nullptr;
    long long stride = 0;

    Positions(PyObject* o, int64_t B, int64_t n, int dev, const Stream& stream) {
        t = laid_out(tensor("positions", o), dev, stream);
        if (t.dim() == 2) {
            p = ints("positions", t, {B, n}, dev);
            stride = n;
        } else {
            p = ints("positions", t, {n}, dev);
        }
    }
    Positions() = default;
};

bool same_memory(const Tensor& a, const Tensor& b) {
    return a.data_ptr() == b.data_ptr() && a.sizes() == b.sizes() && a.strides() == b.strides();
}
// Whether the strides show that no two elements of t are the same: each one reaches past
// all that the smaller ones do.
bool no_element_twice(const Tensor& t) {
    int64_t size[4], stride[4];
    int n = 0;
    for (int64_t i = 0; i < t.dim(); ++i) {
        if (t.size(i) < 2) continue;
        int at = n++;
        for (; at > 0 && stride[at - 1] > t.stride(i); --at) size[at] = size[at - 1], stride[at] = stride[at - 1];
        size[at] = t.size(i), stride[at] = t.stride(i);
    }
    int64_t past = 1;
    for (int i = 0; i < n; ++i) {
        if (stride[i] < past) return false;
        past += (size[i] - 1) * stride[i];
    }
    return true;
}
// Refuses an output `a` that shares memory with another tensor `b` of rows -- or may: their
// ranges of addresses are apart, or else some stride is a period in which they are.  The
// dimensions whose strides are multiples of the period leave the place in it as it is, the
// others reach from a tensor's first element over its extent: so lie the parts of one
// projection, whatever the order of its dimensions.
void apart_from(const char* a_name, const Tensor& a, const char* b_name, const Tensor& b) {
    if (a.numel() == 0 || b.numel() == 0) return;
    // elements from the first to past the last, in a period (0: none)
    auto extent = [](const Tensor& t, int64_t period) {
        int64_t n = 1;
        for (int64_t i = 0; i < t.dim(); ++i)
            if (t.size(i) > 1 && (period == 0 || t.stride(i) % period != 0)) n += (t.size(i) - 1) * t.stride(i);
        return n;
    };
    const auto pa = reinterpret_cast<intptr_t>(a.data_ptr()), pb = reinterpret_cast<intptr_t>(b.data_ptr());
    if (pa + 2 * extent(a, 0) <= pb || pb + 2 * extent(b, 0) <= pa) return;
    if ((pb - pa) % 2 == 0)
        for (const Tensor* t : {&a, &b})
            for (int64_t i = 0; i + 1 < t->dim(); ++i) {
                const int64_t period = t->stride(i);
                if (t->size(i) < 2 || period <= 0) continue;
                const int64_t of_a = extent(a, period), of_b = extent(b, period);
                const int64_t off = ((pb - pa) / 2 % period + period) % period;
                if (of_a <= period && off >= of_a && off + of_b <= period) return;
            }
    throw BadValue(std::string(a_name) + " may share memory with " + b_name);
}

// Rows to turn: [T, heads, d] or [B, heads, n, d] with the strides of batch, head
// and token; and where they go.
struct Turned {
    Tensor in, out;
    long long is[3], os[3];
    int heads = 0;

    static void strides_of(const Tensor& t, long long (&s)[3]) {
        const bool packed = t.dim() == 3;
        s[0] = packed ? 0 : t.stride(0);
        s[1] = t.stride(1);
        s[2] = packed ? t.stride(0) : t.stride(2);
    }
    Turned(const char* name, PyObject* in_, const char* out_name, PyObject* out_, int dev,
           const Stream& stream)
        : in(tensor(name, in_)) {
        if (in.scalar_type() != at::kBFloat16) throw BadType(std::string(name) + " must be bfloat16");
        if (!on(in, dev) || (in.dim() != 3 && in.dim() != 4))
            throw BadValue(std::string(name) + " must be [T, heads, d] or [B, heads, n, d] on cuda:" +
                           std::to_string(dev));
        heads = small(in.size(1));
        if (out_ == Py_None) {
            out = fresh(in.sizes(), at::kBFloat16, dev, stream);
        } else {
            out = tensor(out_name, out_);
            if (out.scalar_type() != at::kBFloat16 || out.sizes() != in.sizes() || !on(out, dev))
                throw BadValue(std::string(out_name) + " must be a bf16 tensor " + text(in.sizes()) +
                               " on cuda:" + std::to_string(dev));
            if (!rows_fit(out))
                throw BadValue(std::string(out_name) + " must have contiguous, 16-byte aligned rows");
            if (out.numel() > 0 && !no_element_twice(out))
                throw BadValue(std::string(out_name) + " may have rows that overlap");
            if (!same_memory(in, out)) apart_from(out_name, out, name, in);
        }
        if (!rows_fit(in)) {
            const c10::cuda::CUDAStreamGuard guard(torch_stream(stream, dev));
            in = in.clone(at::MemoryFormat::Contiguous);
        }
        strides_of(in, is);
        strides_of(out, os);
    }
};

// q, k, positions, freqs, interleaved, inverse, factor, q_out, k_out, stream
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 10);
    const int dev = device_of("q", tensor("q", a[0]));
    const Stream stream = stream_of(a[9], dev);
    const Turned q("q", a[0], "q_out", a[7], dev, stream);
    std::optional<Turned> k;
    if (a[1] != Py_None) k.emplace("k", a[1], "k_out", a[8], dev, stream);
    else if (a[8] != Py_None) throw BadValue("k_out without k");
    const Tensor& x = q.in;
    const bool packed = x.dim() == 3;
    if (k) {   // (rows of one are read while the other's are written)
        const Tensor &q_in = tensor("q", a[0]), &k_in = tensor("k", a[1]);
        apart_from("q_out", q.out, "k", k_in);
        apart_from("k_out", k->out, "q", q_in);
        apart_from("q_out", q.out, "k_out", k->out);
    }
    if (k && (k->in.dim() != x.dim() || k->in.size(0) != x.size(0) ||
              k->in.size(x.dim() - 1) != x.size(x.dim() - 1) || (!packed && k->in.size(2) != x.size(2))))
        throw BadValue("k " + text(k->in.sizes()) + " does not go with q " + text(x.sizes()));
    const int64_t B = packed ? 1 : x.size(0), rows = packed ? x.size(0) : x.size(2);
    const Positions at(a[2], B, rows, dev, stream);
    const Freqs f(a[3], dev, stream, false);
    const fa_status st = fa_rope(
        x.data_ptr(), q.is, q.out.data_ptr(), q.os, q.heads, k ? k->in.data_ptr() : nullptr,
        k ? k->is : nullptr, k ? k->out.data_ptr() : nullptr, k ? k->os : nullptr, k ? k->heads : 0,
        small(B), small(rows), small(x.size(x.dim() - 1)), at.p, at.stride, f.p, f.rot,
        truth("interleaved", a[4]), truth("inverse", a[5]), factor_of(a[6]), stream);
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject* qo = THPVariable_Wrap(q.out);
    PyObject* ko = k ? THPVariable_Wrap(k->out) : Py_NewRef(Py_None);
    PyObject* both = PyTuple_Pack(2, qo, ko);
    Py_DECREF(qo);
    Py_DECREF(ko);
    return both;
}

// What the appends of turned rows share: block_table, seqlens, k_new, v_new,
// freqs, n_new, copies, positions, q, q_out, interleaved, factor from a[0] on.
struct Append {
    int64_t B, n;
    int max_pages;
    const int *table, *lens, *n_new, *copies;
    std::optional<Rows> k, v, q;
    std::optional<Freqs> freqs;
    Positions at;
    Tensor q_out;
    fa_turn turn{};

    Append(PyObject* const* a, const Caches& c, const Stream& stream, bool freqs_optional) {
        const Tensor& t = tensor("block_table", a[0]);
        const Tensor& kn = tensor("k_new", a[2]);
        if (t.dim() != 2 || kn.dim() != 4)
            throw BadValue("block_table must be [B, max_pages], k_new and v_new [B, Hkv, n, d]");
        B = t.size(0), n = kn.size(2);
        max_pages = small(t.size(1));
        table = ints("block_table", t, {B, t.size(1)}, c.dev);
        lens = ints("seqlens", tensor("seqlens", a[1]), {B}, c.dev);
        k.emplace("k_new", a[2], c, c.hkv, B, n, stream);
        v.emplace("v_new", a[3], c, c.hkv, B, n, stream);
        freqs.emplace(a[4], c.dev, stream, freqs_optional);
        n_new = ints_or_null("n_new", a[5], {B}, c.dev);
        copies = ints_or_null("copies", a[6], {B, 3}, c.dev);
        if (a[7] != Py_None) at = Positions(a[7], B, n, c.dev, stream);
        if (a[8] != Py_None) {
            const Tensor& qn = tensor("q", a[8]);
            if (qn.dim() != 4) throw BadValue("q must be [B, Hq, n, d]");
            q.emplace("q", a[8], c, qn.size(1), B, n, stream);
            turn.hq = small(qn.size(1));
            if (a[9] == Py_None) {
                q_out = fresh({B, qn.size(1), n, c.d}, at::kBFloat16, c.dev, stream);
            } else {
                q_out = tensor("q_out", a[9]);
                dense("q_out", q_out, at::kBFloat16, {B, qn.size(1), n, c.d}, c.dev);
                if (!same_memory(qn, q_out)) apart_from("q_out", q_out, "q", qn);
                apart_from("q_out", q_out, "k_new", kn);
                apart_from("q_out", q_out, "v_new", tensor("v_new", a[3]));
            }
            turn.q = q->t.data_ptr();
            turn.q_strides = q->strides;
            turn.q_out = q_out.data_ptr();
        } else if (a[9] != Py_None) {
            throw BadValue("q_out without q");
        }
        turn.freqs = freqs->p;
        turn.rot = freqs->rot;
        turn.interleaved = truth("interleaved", a[10]);
        turn.factor = factor_of(a[11]);
        turn.positions = at.p;
        turn.position_stride = at.stride;
    }
    PyObject* result(fa_status st) const {
        if (st != FA_OK) return PyLong_FromLong(st);
        return q ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None);
    }
};

// k_cache, v_cache, then Append's twelve, stream
PyObject* cache_append_rope(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 15);
    const Caches c(a[0], a[1]);
    const Stream stream = stream_of(a[14], c.dev);
    const Append x(a + 2, c, stream, false);
    return x.result(fa_cache_append_rope(
        c.k, c.v, c.num_pages, c.hkv, c.page_size, c.d, x.table, x.max_pages, x.lens, small(x.B),
        x.k->t.data_ptr(), x.k->strides, x.v->t.data_ptr(), x.v->strides, small(x.n), x.n_new,
        x.copies, &x.turn, stream));
}

// -------------------------------------------------------- 8-bit caches ----

// Scales fp32 [num_pages, Hkv, page_size / block] of both caches.
struct Scales {
    float *k, *v;
    int block;

    Scales(PyObject* k_, PyObject* v_, const Tensor& cache, int dev) {
        const Tensor& ks = tensor("k_scale", k_);
        const Tensor& vs = tensor("v_scale", v_);
        const int64_t blocks = ks.dim() == 3 ? ks.size(2) : 0, page = cache.size(2);
        if (blocks < 1 || page % blocks != 0)
            throw BadValue("k_scale must be [num_pages, Hkv, page_size / block]");
        k = static_cast<float*>(dense("k_scale", ks, at::kFloat, {cache.size(0), cache.size(1), blocks}, dev));
        v = static_cast<float*>(dense("v_scale", vs, at::kFloat, {cache.size(0), cache.size(1), blocks}, dev));
        block = small(page / blocks);
    }
};

// k_cache, v_cache, k_scale, v_scale, then Append's twelve, stream
PyObject* cache_append_q8(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 17);
    const Caches c(a[0], a[1], at::kFloat8_e4m3fn);
    const Scales s(a[2], a[3], tensor("k_cache", a[0]), c.dev);
    const Stream stream = stream_of(a[16], c.dev);
    const Append x(a + 4, c, stream, true);
    return x.result(fa_cache_append_q8(
        c.k, c.v, s.k, s.v, c.num_pages, c.hkv, c.page_size, s.block, c.d, x.table, x.max_pages, x.lens,
        small(x.B), x.k->t.data_ptr(), x.k->strides, x.v->t.data_ptr(), x.v->strides, small(x.n), x.n_new,
        x.copies, &x.turn, stream));
}

// k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, total, max_seqlen,
// k_out, v_out, stream
PyObject* cache_read_q8(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 11);
    const Caches c(a[0], a[1], at::kFloat8_e4m3fn);
    const Scales s(a[2], a[3], tensor("k_cache", a[0]), c.dev);
    const Stream stream = stream_of(a[10], c.dev);
    const Tensor table = laid_out(tensor("block_table", a[4]), c.dev, stream);
    const Tensor cu = laid_out(tensor("cu_seqlens", a[5]), c.dev, stream);
    if (table.dim() != 2) throw BadValue("block_table must be [B, max_pages]");
    const int64_t B = table.size(0);
    const int total = whole("total", a[6]), longest = whole("max_seqlen", a[7]);
    if (total < 0) throw BadValue("total must not be negative");
    Tensor out[2];
    const char* names[2] = {"k_out", "v_out"};
    for (int i = 0; i < 2; ++i) {
        out[i] = a[8 + i] == Py_None ? fresh({total, c.hkv, c.d}, at::kBFloat16, c.dev, stream)
                                     : tensor(names[i], a[8 + i]);
        dense(names[i], out[i], at::kBFloat16, {total, c.hkv, c.d}, c.dev);
    }
    apart_from("k_out", out[0], "v_out", out[1]);
    return status_or(fa_cache_read_q8(c.k, c.v, s.k, s.v, c.num_pages, c.hkv, c.page_size, s.block, c.d,
                                      ints("block_table", table, {B, table.size(1)}, c.dev),
                                      small(table.size(1)), ints("cu_seqlens", cu, {B + 1}, c.dev),
                                      small(B), longest, total, out[0].data_ptr(), out[1].data_ptr(),
                                      stream),
                     pair(out[0], out[1]));
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, scale, causal,
// out, lse, stream, window, sinks, first
PyObject* decode_paged_q8(PyObject* const* a, Py_ssize_t n) {
    need_args(n, 15);
    Attention c(a[0], a[1], a[2], a[13], a[9], a[10], a[11], true, at::kFloat8_e4m3fn);
    const Scales s(a[3], a[4], c.k, c.dev);
    const Pages p(c, a[5]);
    return c.result(fa_fwd_decode_paged_q8(
        c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), s.k, s.v, c.out.data_ptr(), c.lse_ptr(), c.B,
        c.Hq, p.hkv, c.n, ints("seqlens_k", c.hold(tensor("seqlens_k", a[6])), {c.B}, c.dev), p.table,
        p.max_pages, p.page_size, p.num_pages, s.block, c.d, scale_of(a[7], c.d),
        truth("causal", a[8]), whole("window", a[12]), whole("first", a[14]), c.sinks, c.stream));
}

#define ENTRY(f) \
    {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    ENTRY(decode_tree), ENTRY(decode_tree_paged), ENTRY(decode_first), ENTRY(decode_paged_first),
    ENTRY(tree_mask),   ENTRY(cache_fork),        ENTRY(cache_reserve), ENTRY(cache_free),
    ENTRY(cache_append), ENTRY(cache_copy),       ENTRY(cache_compact), ENTRY(rope),
    ENTRY(cache_append_rope), ENTRY(cache_append_q8), ENTRY(cache_read_q8), ENTRY(decode_paged_q8),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, kMethods,
                       nullptr,               nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&kModule); }
