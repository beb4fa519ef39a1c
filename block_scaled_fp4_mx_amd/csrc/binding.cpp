// Host side of the attention path's Python entry points: the checks of a call's
// tensors, and the call of the C ABI with their pointers and sizes.
//
// A serving step makes several of these calls, each with a kernel of a few
// microseconds, so its time is the host's.  With the checks in Python and the call
// through ctypes a call cost 8 to 10 us on the host; here 3 to 4, most of it the
// launch itself.  What is checked, in which order, and what an error says is as in
// the package's other functions: type, dtype and layout of every tensor, then the
// shapes, then the device.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <exception>
#include <string>

#include "fp4.h"

namespace {

using at::Tensor;

struct PythonError {};                     // thrown where the Python error is set

template <class... A>
[[noreturn]] void fail(PyObject* type, const char* format, A... args) {
    PyErr_Format(type, format, args...);
    throw PythonError();
}

std::string text(at::IntArrayRef sizes) {
    std::string s = "(";
    for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
    return s + (sizes.size() == 1 ? ",)" : ")");
}

// Dtypes of an argument.
struct Dtypes {
    at::ScalarType a, b;
    const char* names;
};
constexpr Dtypes kU8{at::kByte, at::kByte, "torch.uint8"}, kI32{at::kInt, at::kInt, "torch.int32"},
    kI64{at::kLong, at::kLong, "torch.int64"}, kF32{at::kFloat, at::kFloat, "torch.float32"},
    kBF16{at::kBFloat16, at::kBFloat16, "torch.bfloat16"},
    kWeight{at::kBFloat16, at::kFloat, "torch.bfloat16 or torch.float32"};

// Without the interpreter's lock, as a ctypes call is.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
struct OnDevice {
    int before = -1;
    explicit OnDevice(int dev) {
        if (hipGetDevice(&before) != hipSuccess || before != dev)
            (void)hipSetDevice(dev);
        else
            before = -1;
    }
    ~OnDevice() {
        if (before >= 0) (void)hipSetDevice(before);
    }
};

// One call: its tensors, the GPU that all of them are on, its stream.
class Call {
public:
    explicit Call(const char* fn) : fn_(fn) {}

    const Tensor& operator()(const char* name, PyObject* o, const Dtypes& types, bool dense = true) {
        if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s: %s must be a torch tensor, got %s", fn_, name, Py_TYPE(o)->tp_name);
        const Tensor& t = THPVariable_Unpack(o);
        const at::ScalarType type = t.scalar_type();
        if (type != types.a && type != types.b) {
            PyObject* got = PyObject_GetAttrString(o, "dtype");
            if (got == nullptr) throw PythonError();
            PyErr_Format(PyExc_TypeError, "%s: %s must be %s, got %S", fn_, name, types.names, got);
            Py_DECREF(got);
            throw PythonError();
        }
        if (!t.is_contiguous() && t.numel()) {
            if (t.dim() && t.size(-1) > 1 && t.stride(-1) != 1)
                fail(PyExc_ValueError, "%s: %s must be contiguous along its last axis", fn_, name);
            if (dense) fail(PyExc_ValueError, "%s: %s must be contiguous", fn_, name);
        }
        if (count_ == kMost) fail(PyExc_RuntimeError, "%s: too many tensors", fn_);
        names_[count_] = name;
        tensors_[count_++] = &t;
        return t;
    }
    const Tensor* optional(const char* name, PyObject* o, const Dtypes& types) {
        return o == Py_None ? nullptr : &(*this)(name, o, types);
    }
    // Calls f(args..., stream) with the tensors' GPU as the current device.
    template <class F>
    PyObject* go(PyObject* stream, F&& f) {
        int dev = -1;
        for (int i = 0; i < count_; ++i) {
            if (!tensors_[i]->is_cuda())
                fail(PyExc_ValueError, "%s: %s must be on the GPU, got a %s tensor", fn_, names_[i],
                     c10::DeviceTypeName(tensors_[i]->device().type(), true).c_str());
            if (i && tensors_[i]->get_device() != dev) {
                std::string all;
                for (int j = 0; j < count_; ++j)
                    all += (j ? ", " : "") + std::string(names_[j]) + " on " + tensors_[j]->device().str();
                fail(PyExc_ValueError, "%s: the tensors are on several GPUs: %s", fn_, all.c_str());
            }
            dev = tensors_[i]->get_device();
        }
        void* handle = stream_of(stream, dev);
        int status;
        {
            const Unlocked unlocked;
            const OnDevice on(dev);
            status = f(handle);
        }
        return PyLong_FromLong(status);
    }
    const char* name() const { return fn_; }

private:
    static void* stream_of(PyObject* stream, int dev) {
        if (stream == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
        PyObject* number = PyObject_HasAttrString(stream, "cuda_stream") ? PyObject_GetAttrString(stream, "cuda_stream")
                                                                         : (Py_INCREF(stream), stream);
        void* handle = number ? PyLong_AsVoidPtr(number) : nullptr;
        Py_XDECREF(number);
        if (PyErr_Occurred()) throw PythonError();
        return handle;
    }

    static constexpr int kMost = 16;
    const char* fn_;
    const Tensor* tensors_[kMost];
    const char* names_[kMost];
    int count_ = 0;
};

template <class T = void>
T* pointer(const Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <class T = void>
T* pointer(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}

// An attention's scale; None: head_dim ** -0.5.
float scale_of(PyObject* o, int64_t head_dim) {
    return (float)(o == Py_None ? 1.0 / std::sqrt((double)head_dim) : number(o));
}

// The members of a KvCache or KvPages.
void members(const char* fn, const char* what, PyObject* o, Py_ssize_t n, PyObject** out) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != n) fail(PyExc_TypeError, "%s: expected a %s, got %s", fn, what, Py_TYPE(o)->tp_name);
    for (Py_ssize_t i = 0; i < n; ++i) out[i] = PyTuple_GET_ITEM(o, i);
}

struct Cache {
    const Tensor *kc, *ks, *vc, *vs;
    int64_t page_size;
    fp4_kv_cache c;
};
// names: of k_codes, k_scales, v_codes, v_scales.
Cache cache_of(Call& call, PyObject* o, const char* const* names) {
    PyObject* m[5];
    members(call.name(), "KvCache", o, 5, m);
    Cache x;
    x.kc = &call(names[0], m[0], kU8), x.ks = &call(names[1], m[1], kU8);
    x.vc = call.optional(names[2], m[2], kU8), x.vs = call.optional(names[3], m[3], kU8);
    x.page_size = integer(m[4]);
    return x;
}
constexpr const char* kCacheNames[] = {"k_codes", "k_scales", "v_codes", "v_scales"};
constexpr const char* kSrcNames[] = {"src.k_codes", "src.k_scales", "src.v_codes", "src.v_scales"};
constexpr const char* kDstNames[] = {"dst.k_codes", "dst.k_scales", "dst.v_codes", "dst.v_scales"};

// Checks the shapes of a cache's (checked) tensors and fills in its C struct.
void check_shapes(const Call& call, Cache& x) {
    const char* fn = call.name();
    if ((x.vc == nullptr) != (x.vs == nullptr))
        fail(PyExc_ValueError, "%s: v_codes and v_scales must both be given or both be None", fn);
    if (x.kc->dim() != 2 || x.page_size <= 0 || x.kc->size(0) % x.page_size)
        fail(PyExc_ValueError, "%s: k_codes must be [num_pages * %lld, d/2], got %s", fn, (long long)x.page_size,
             text(x.kc->sizes()).c_str());
    const int64_t rows = x.kc->size(0), half = x.kc->size(1);
    if (x.ks->dim() != 2 || x.ks->size(0) != rows || x.ks->size(1) != half / 16)
        fail(PyExc_ValueError, "%s: k_scales has shape %s, expected %s", fn, text(x.ks->sizes()).c_str(),
             text({rows, half / 16}).c_str());
    if (x.vc && (!x.vc->sizes().equals(x.kc->sizes()) || !x.vs->sizes().equals(x.ks->sizes())))
        fail(PyExc_ValueError, "%s: the cache's values must have the shapes of its keys", fn);
    x.c = {pointer<uint8_t>(x.kc), pointer<uint8_t>(x.ks), pointer<uint8_t>(x.vc), pointer<uint8_t>(x.vs),
           rows / x.page_size, 2 * half, x.page_size};
}

struct Pages {
    const Tensor *table, *counts, *lens, *refs;
    fp4_kv_pages c;
};
Pages pages_of(Call& call, PyObject* o) {
    PyObject* m[4];
    members(call.name(), "KvPages", o, 4, m);
    Pages x;
    x.table = &call("page_table", m[0], kI32), x.counts = &call("page_counts", m[1], kI32);
    x.lens = &call("seq_lens", m[2], kI32), x.refs = &call("page_refs", m[3], kI32);
    return x;
}
void check_shapes(const Call& call, Pages& x) {
    if (x.table->dim() != 2 || x.counts->dim() != 1 || x.lens->dim() != 1 || x.refs->dim() != 1 ||
        x.counts->size(0) != x.table->size(0) || x.lens->size(0) != x.table->size(0))
        fail(PyExc_ValueError, "%s: page_table must be [batch, max_pages], page_counts and seq_lens [batch], page_refs [num_pages]",
             call.name());
    x.c = {pointer<int32_t>(x.table), pointer<int32_t>(x.counts), pointer<int32_t>(x.lens), pointer<int32_t>(x.refs),
           x.table->size(0), x.table->size(1), x.refs->size(0)};
}

void has_shape(const Call& call, const char* name, const Tensor* t, at::IntArrayRef shape) {
    if (t && !t->sizes().equals(shape))
        fail(PyExc_ValueError, "%s: %s has shape %s, expected %s", call.name(), name, text(t->sizes()).c_str(), text(shape).c_str());
}
// [n] or [n, 2]: a list of ids.
void is_list(const Call& call, const char* name, const Tensor& t, int64_t dim, const char* expected) {
    if (t.dim() != dim || (dim == 2 && t.size(1) != 2))
        fail(PyExc_ValueError, "%s: %s has shape %s, expected %s", call.name(), name, text(t.sizes()).c_str(), expected);
}

// The leading dimension of a [tokens, heads, head_dim] tensor, whose heads must lie
// one after another; tokens may be any number of elements apart.
int64_t heads_of(const Call& call, const char* name, const Tensor& t) {
    if (t.dim() != 3)
        fail(PyExc_ValueError, "%s: %s must be [tokens, heads, head_dim], got shape %s", call.name(), name, text(t.sizes()).c_str());
    if (t.stride(1) != t.size(2) && t.size(1) > 1 && t.numel())
        fail(PyExc_ValueError, "%s: the heads of %s must be contiguous", call.name(), name);
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}
// The pitch of the tokens of a [batch, drafts, q_heads, head_dim] tensor, which must be one.
int64_t drafted(const Call& call, const char* name, const Tensor& t) {
    if (t.dim() != 4)
        fail(PyExc_ValueError, "%s: %s must be [batch, drafts, q_heads, head_dim], got shape %s", call.name(), name,
             text(t.sizes()).c_str());
    const int64_t batch = t.size(0), drafts = t.size(1), heads = t.size(2), d = t.size(3);
    const bool empty = t.numel() == 0;
    if (heads > 1 && t.stride(2) != d && !empty) fail(PyExc_ValueError, "%s: the heads of %s must be contiguous", call.name(), name);
    const int64_t ld = drafts > 1 ? t.stride(1) : batch > 1 ? t.stride(0) : heads * d;
    if (batch > 1 && t.stride(0) != drafts * ld && !empty)
        fail(PyExc_ValueError, "%s: the tokens of %s must be one pitch apart", call.name(), name);
    return ld;
}

// ---- the entry points; each takes its arguments in the order of the package's function

PyObject* kv_append_mx(PyObject* const* v) {
    Call call("fp4_kv_append_mx");
    const Tensor& x = call("x", v[0], kBF16, false);
    const Tensor& slots = call("slots", v[1], kI32);
    const Tensor& codes = call("cache_codes", v[2], kU8);
    const Tensor& scales = call("cache_scales", v[3], kU8);
    const int64_t tokens = integer(v[4]), d = integer(v[5]), ld = integer(v[6]);
    return call.go(v[7], [&](void* s) {
        return fp4_kv_append_mx(pointer(x), tokens, d, ld, pointer<int32_t>(slots), pointer<uint8_t>(codes),
                                pointer<uint8_t>(scales), codes.size(0), s);
    });
}

PyObject* qk_norm_rope(PyObject* const* v) {
    Call call("fp4_qk_norm_rope");
    const char* fn = call.name();
    const Tensor& q = call("q", v[0], kBF16, false);
    const Tensor& k = call("k", v[1], kBF16, false);
    const Tensor& qo = call("q_out", v[2], kBF16, false);
    const Tensor& ko = call("k_out", v[3], kBF16, false);
    const Tensor* qw = call.optional("q_weight", v[6], kWeight);
    const Dtypes same = !qw ? kWeight : qw->scalar_type() == at::kFloat ? kF32 : kBF16;
    const Tensor* kw = call.optional("k_weight", v[7], same);
    const Tensor* table = call.optional("cos_sin", v[5], kF32);
    const Tensor* where = table ? &call("positions", v[4], kI32) : nullptr;
    const float eps = (float)number(v[8]);
    const int interleaved = PyObject_IsTrue(v[9]);
    if (interleaved < 0) throw PythonError();
    const int64_t ld_q = heads_of(call, "q", q), ld_k = heads_of(call, "k", k), ld_qo = heads_of(call, "q_out", qo),
                  ld_ko = heads_of(call, "k_out", ko);
    const int64_t tokens = q.size(0), d = q.size(2);
    if (k.size(0) != tokens || k.size(2) != d)
        fail(PyExc_ValueError, "%s: k has shape %s, q %s", fn, text(k.sizes()).c_str(), text(q.sizes()).c_str());
    if (!qo.sizes().equals(q.sizes()) || !ko.sizes().equals(k.sizes()))
        fail(PyExc_ValueError, "%s: q_out and k_out must have the shapes of q and k", fn);
    has_shape(call, "q_weight", qw, {d});
    has_shape(call, "k_weight", kw, {d});
    if (table && (table->dim() != 2 || where->dim() != 1 || where->size(0) != tokens))
        fail(PyExc_ValueError, "%s: cos_sin must be [max_positions, rot_dim] and positions [tokens]", fn);
    const bool f32 = (qw && qw->scalar_type() == at::kFloat) || (kw && kw->scalar_type() == at::kFloat);
    return call.go(v[10], [&](void* s) {
        return fp4_qk_norm_rope(pointer(q), pointer(k), tokens, (int)q.size(1), (int)k.size(1), (int)d, ld_q, ld_k, pointer(qw),
                                pointer(kw), f32 ? FP4_DT_F32 : FP4_DT_BF16, eps, pointer<float>(table),
                                table ? table->size(0) : 0, table ? (int)table->size(1) : 0, interleaved,
                                pointer<int32_t>(where), pointer(qo), ld_qo, pointer(ko), ld_ko, s);
    });
}

PyObject* kv_reserve(PyObject* const* v) {
    Call call("fp4_kv_reserve");
    Cache cache = cache_of(call, v[0], kCacheNames);
    Pages pages = pages_of(call, v[1]);
    const Tensor& add = call("new_tokens", v[2], kI32);
    const Tensor& n_short = call("n_short", v[4], kI32);
    const Tensor& ws = call("workspace", v[5], kU8);
    const Tensor* slots = call.optional("slots", v[3], kI32);
    check_shapes(call, cache);
    check_shapes(call, pages);
    has_shape(call, "new_tokens", &add, {pages.c.batch});
    has_shape(call, "n_short", &n_short, {1});
    if (slots && (slots->dim() != 2 || slots->size(0) != pages.c.batch))
        fail(PyExc_ValueError, "%s: slots has shape %s, expected [%lld, max_new]", call.name(), text(slots->sizes()).c_str(),
             (long long)pages.c.batch);
    return call.go(v[6], [&](void* s) {
        return fp4_kv_reserve(&cache.c, &pages.c, pointer<int32_t>(add), pointer<int32_t>(slots), slots ? slots->size(1) : 0,
                              pointer<int32_t>(n_short), pointer(ws), (size_t)ws.numel(), s);
    });
}

PyObject* kv_fork(PyObject* const* v) {
    Call call("fp4_kv_fork");
    Pages pages = pages_of(call, v[0]);
    const Tensor& pairs = call("pairs", v[1], kI32);
    const int64_t page_size = integer(v[2]);
    check_shapes(call, pages);
    is_list(call, "pairs", pairs, 2, "[n, 2]");
    return call.go(v[3], [&](void* s) { return fp4_kv_fork(&pages.c, pointer<int32_t>(pairs), pairs.size(0), page_size, s); });
}

PyObject* kv_free(PyObject* const* v) {
    Call call("fp4_kv_free");
    Pages pages = pages_of(call, v[0]);
    const Tensor& seqs = call("seqs", v[1], kI32);
    const int64_t page_size = integer(v[2]);
    const Tensor* keep = call.optional("keep_lens", v[3], kI32);
    check_shapes(call, pages);
    is_list(call, "seqs", seqs, 1, "[n]");
    has_shape(call, "keep_lens", keep, {seqs.size(0)});
    return call.go(v[4], [&](void* s) {
        return fp4_kv_free(&pages.c, pointer<int32_t>(seqs), seqs.size(0), pointer<int32_t>(keep), page_size, s);
    });
}

// kReserved: with the slots of a reservation.
template <bool kReserved>
PyObject* kv_compact(PyObject* const* v) {
    Call call(kReserved ? "fp4_kv_compact_reserved" : "fp4_kv_compact");
    Cache cache = cache_of(call, v[0], kCacheNames);
    Pages pages = pages_of(call, v[1]);
    const Tensor& lens = call("accepted_lens", v[3], kI32);
    const Tensor* accepted = call.optional("accepted", v[2], kI32);
    const Tensor* slots = kReserved ? &call("slots", v[4], kI32) : nullptr;
    check_shapes(call, cache);
    check_shapes(call, pages);
    has_shape(call, "accepted_lens", &lens, {pages.c.batch});
    if (accepted && (accepted->dim() != 2 || accepted->size(0) != pages.c.batch))
        fail(PyExc_ValueError, "%s: accepted has shape %s, expected [%lld, max_accepted]", call.name(),
             text(accepted->sizes()).c_str(), (long long)pages.c.batch);
    if (slots && (slots->dim() != 2 || slots->size(0) != pages.c.batch))
        fail(PyExc_ValueError, "%s: slots has shape %s, expected [%lld, max_new]", call.name(), text(slots->sizes()).c_str(),
             (long long)pages.c.batch);
    if ((accepted && accepted->size(1) == 0) || (slots && slots->size(1) == 0))
        return PyLong_FromLong(0);                        // nothing can be accepted, or was reserved
    return call.go(v[kReserved ? 5 : 4], [&](void* s) {
        const int32_t* which = pointer<int32_t>(accepted);
        const int64_t most = accepted ? accepted->size(1) : 0;
        return kReserved ? fp4_kv_compact_reserved(&cache.c, &pages.c, which, most, pointer<int32_t>(lens),
                                                   pointer<int32_t>(slots), slots->size(1), s)
                         : fp4_kv_compact(&cache.c, &pages.c, which, most, pointer<int32_t>(lens), s);
    });
}

PyObject* kv_copy_pages(PyObject* const* v) {
    Call call("fp4_kv_copy_pages");
    Cache src = cache_of(call, v[0], kSrcNames), dst = cache_of(call, v[1], kDstNames);
    const Tensor& from = call("src_pages", v[2], kI32);
    const Tensor& to = call("dst_pages", v[3], kI32);
    check_shapes(call, src);
    check_shapes(call, dst);
    is_list(call, "src_pages", from, 1, "[n]");
    has_shape(call, "dst_pages", &to, {from.size(0)});
    return call.go(v[4], [&](void* s) {
        return fp4_kv_copy_pages(&src.c, &dst.c, pointer<int32_t>(from), pointer<int32_t>(to), from.size(0), s);
    });
}

PyObject* attn_tree_mx(PyObject* const* v) {
    Call call("fp4_attn_tree_mx");
    const char* fn = call.name();
    const Tensor& q = call("q", v[0], kBF16, false);
    const Tensor& out = call("out", v[4], kBF16, false);
    Cache cache = cache_of(call, v[1], kCacheNames);
    const Tensor& table = call("page_table", v[2], kI32);
    const Tensor& lens = call("seq_lens", v[3], kI32);
    const Tensor& ws = call("workspace", v[5], kU8);
    const Tensor* draft_lens = call.optional("draft_lens", v[6], kI32);
    const Tensor* mask = call.optional("tree_mask", v[7], kI64);
    const int64_t ld_q = drafted(call, "q", q), ld_out = drafted(call, "out", out);
    const int64_t batch = q.size(0), drafts = q.size(1), heads = q.size(2), d = q.size(3);
    has_shape(call, "out", &out, q.sizes());
    check_shapes(call, cache);
    if (!cache.vc) fail(PyExc_ValueError, "%s: the cache has no values", fn);
    if (!d || !cache.c.d || cache.c.d % d)
        fail(PyExc_ValueError, "%s: the cache's rows hold %lld values, not a multiple of head_dim %lld", fn, (long long)cache.c.d,
             (long long)d);
    if (table.dim() != 2 || table.size(0) != batch)
        fail(PyExc_ValueError, "%s: page_table has shape %s, expected [%lld, max_pages]", fn, text(table.sizes()).c_str(),
             (long long)batch);
    has_shape(call, "seq_lens", &lens, {batch});
    has_shape(call, "draft_lens", draft_lens, {batch});
    has_shape(call, "tree_mask", mask, {batch, drafts});
    const float scale = scale_of(v[8], d);
    return call.go(v[9], [&](void* s) {
        return fp4_attn_tree_mx(pointer(q), ld_q, &cache.c, pointer<int32_t>(table), table.size(1), pointer<int32_t>(lens),
                                pointer<int32_t>(draft_lens), pointer<uint64_t>(mask), batch, (int)drafts, (int)heads,
                                (int)(cache.c.d / d), (int)d, scale, pointer(out), ld_out, pointer(ws), (size_t)ws.numel(), s);
    });
}

PyObject* attn_prompt(PyObject* const* v) {
    Call call("fp4_attn_prompt");
    const char* fn = call.name();
    const Tensor& q = call("q", v[0], kBF16, false);
    const Tensor& k = call("k", v[1], kBF16, false);
    const Tensor& val = call("v", v[2], kBF16, false);
    const Tensor& out = call("out", v[4], kBF16, false);
    const Tensor& cu = call("cu_seqlens", v[3], kI32);
    const int64_t ld_q = heads_of(call, "q", q), ld_k = heads_of(call, "k", k), ld_v = heads_of(call, "v", val),
                  ld_out = heads_of(call, "out", out);
    if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || !val.sizes().equals(k.sizes()))
        fail(PyExc_ValueError, "%s: k and v have shapes %s and %s, q %s", fn, text(k.sizes()).c_str(), text(val.sizes()).c_str(),
             text(q.sizes()).c_str());
    has_shape(call, "out", &out, q.sizes());
    if (cu.dim() != 1 || cu.size(0) < 1)
        fail(PyExc_ValueError, "%s: cu_seqlens has shape %s, expected [seqs + 1]", fn, text(cu.sizes()).c_str());
    const float scale = scale_of(v[5], q.size(2));
    return call.go(v[6], [&](void* s) {
        return fp4_attn_prompt(pointer(q), pointer(k), pointer(val), pointer<int32_t>(cu), cu.size(0) - 1, q.size(0),
                               (int)q.size(1), (int)k.size(1), (int)q.size(2), ld_q, ld_k, ld_v, scale, pointer(out), ld_out, s);
    });
}

// No C++ exception leaves the module.
template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return kFn(args);
    } catch (const PythonError&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
        return nullptr;
    }
}
template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<kv_append_mx, 8>("fp4_kv_append_mx"),
    method<qk_norm_rope, 11>("fp4_qk_norm_rope"),
    method<kv_reserve, 7>("fp4_kv_reserve"),
    method<kv_fork, 4>("fp4_kv_fork"),
    method<kv_free, 5>("fp4_kv_free"),
    method<kv_compact<false>, 5>("fp4_kv_compact"),
    method<kv_compact<true>, 6>("fp4_kv_compact_reserved"),
    method<kv_copy_pages, 5>("fp4_kv_copy_pages"),
    method<attn_tree_mx, 10>("fp4_attn_tree_mx"),
    method<attn_prompt, 7>("fp4_attn_prompt"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
