// Python entry points of the operators between the linears and around a batch
// (layer_ops.py and batch_ops.py name and document them): argument checks, outputs and workspaces from torch's
// allocator, then the C ABI of include/nvfp4_w4a16.h on the current stream.
//
// These calls are short (a decode step makes a few hundred of them), and a
// Python body with a ctypes call of twenty arguments took 18 to 30 us of host
// time where the kernels take 3 to 15; the same checks here take 1 to 2 us and
// the call about 6 with its launches.
#include <Python.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <limits>
#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "nvfp4_w4a16.h"

namespace {

PyObject* g_error = nullptr;       // Nvfp4Error(status, message)

struct Refused {
    int status;
    std::string message;
};
struct PythonError {};             // a Python exception is set

[[noreturn]] void refuse(int status, std::string message) { throw Refused{status, std::move(message)}; }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

std::string type_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kFloat: return "torch.float32";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

using Name = const char*;

// The tensor behind `o`, or null for None.
const at::Tensor* tensor_or_none(PyObject* o, Name name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(1, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, Name name) {
    const at::Tensor* t = tensor_or_none(o, name);
    if (!t) refuse(1, std::string(name) + " must be a tensor, got None");
    return *t;
}

int64_t integer(PyObject* o, Name name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(1, std::string(name) + " must be a whole number of 64 bits");
    }
    return v;
}

float real(PyObject* o, Name name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(1, std::string(name) + " must be a number");
    }
    return (float)v;
}

// What a call's tensors share: the device (the current one) and the activation type.
struct Call {
    int dev;
    at::ScalarType act;
    int f16;

    Call(const at::Tensor& t, Name name, bool activation = true) {
        if (!t.is_cuda()) refuse(1, std::string(name) + " must be a CUDA tensor");
        dev = t.get_device();
        const int current = c10::cuda::current_device();
        if (dev != current)
            refuse(1, std::string(name) + " is on cuda:" + std::to_string(dev) + ", the current device is cuda:" + std::to_string(current));
        if (activation) type(t.scalar_type(), name);
    }
    void type(at::ScalarType t, Name name) {
        if (t != at::kBFloat16 && t != at::kHalf)
            refuse(1, std::string(name) + " must be torch.bfloat16 or torch.float16, got " + type_text(t));
        act = t;
        f16 = t == at::kHalf;
    }

    // Device, type and shape; contiguous, or (rows) its last dimension.
    const at::Tensor& check(const at::Tensor& t, Name name, at::ScalarType dt, at::IntArrayRef shape, bool contiguous = true) const {
        if (!t.is_cuda() || t.get_device() != dev) refuse(1, std::string(name) + " must be a tensor on cuda:" + std::to_string(dev));
        if (t.scalar_type() != dt) refuse(1, std::string(name) + " must be " + type_text(dt) + ", got " + type_text(t.scalar_type()));
        if (t.sizes() != shape) refuse(2, std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
        if (contiguous) {
            if (!t.is_contiguous()) refuse(1, std::string(name) + " must be contiguous");
        } else {
            rows(t, name);
        }
        return t;
    }
    void rows(const at::Tensor& t, Name name) const {
        if (t.dim() > 0 && t.size(-1) > 1 && t.stride(-1) != 1) refuse(1, std::string(name) + " must be contiguous in its last dimension");
    }
    // The caller's output, or a new one (straight from the allocator: half the time of a dispatched at::empty).
    at::Tensor output(PyObject* o, Name name, at::ScalarType dt, at::IntArrayRef shape) const {
        if (const at::Tensor* t = tensor_or_none(o, name)) return check(*t, name, dt, shape);
        return at::Tensor(at::detail::empty_cuda(shape, dt, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

void done(nvfp4_status st) {
    if (st != NVFP4_OK) refuse(st, nvfp4_last_error());
}

// Stride of dimension d; a dimension of one element (or none) has no step.
int64_t step(const at::Tensor& t, int d) { return t.size(d) > 1 ? t.stride(d) : 0; }

nvfp4_kv_cache cache_of(const Call& c, PyObject* k_cache, PyObject* v_cache, PyObject* k_scale, PyObject* v_scale) {
    const at::Tensor& k = tensor(k_cache, "k_cache");
    const at::Tensor& v = tensor(v_cache, "v_cache");
    if (k.dim() != 4) refuse(2, "k_cache must be a tensor [pages, heads, page_size, head_dim]");
    const bool e4m3 = k.scalar_type() == at::kFloat8_e4m3fn;
    const auto shape = k.sizes();
    c.check(k, "k_cache", e4m3 ? at::kFloat8_e4m3fn : c.act, shape, false);
    c.check(v, "v_cache", k.scalar_type(), shape, false);
    // A dimension of one element has no step: any stride there stands for that of dense rows.
    int64_t strides[3], dense = shape[3];
    bool same = true;
    for (int i = 2; i >= 0; --i) {
        strides[i] = shape[i] == 1 ? dense : k.stride(i);
        same = same && (shape[i] == 1 || v.stride(i) == k.stride(i));
        dense = strides[i] * shape[i];
    }
    if (!same)
        refuse(1, "k_cache and v_cache must have the same strides, got " + shape_text(k.strides()) + " and " + shape_text(v.strides()));
    const at::Tensor* ks = tensor_or_none(k_scale, "k_scale");
    const at::Tensor* vs = tensor_or_none(v_scale, "v_scale");
    if (e4m3 && (!ks || !vs)) refuse(1, "an E4M3 cache needs k_scale and v_scale");
    if (!e4m3 && (ks || vs)) refuse(1, "k_scale and v_scale go with an E4M3 cache");
    if (e4m3) {
        c.check(*ks, "k_scale", at::kFloat, shape.slice(0, 3));
        c.check(*vs, "v_scale", at::kFloat, shape.slice(0, 3));
    }
    nvfp4_kv_cache d{};
    d.k = k.data_ptr();
    d.v = v.data_ptr();
    d.k_scale = e4m3 ? (float*)ks->data_ptr() : nullptr;
    d.v_scale = e4m3 ? (float*)vs->data_ptr() : nullptr;
    d.num_pages = shape[0]; d.heads = shape[1]; d.page_size = shape[2]; d.head_dim = shape[3];
    d.page_stride = strides[0]; d.head_stride = strides[1]; d.token_stride = strides[2];
    d.type = e4m3 ? NVFP4_CACHE_E4M3 : NVFP4_CACHE_16;
    return d;
}

PyObject* wrapped(at::Tensor t) {
    PyObject* o = THPVariable_Wrap(std::move(t));
    if (!o) throw PythonError{};
    return o;
}

// The tensors as a tuple, the only one as itself.
PyObject* result(std::initializer_list<at::Tensor> ts) {
    if (ts.size() == 1) return wrapped(*ts.begin());
    PyObject* tuple = PyTuple_New((Py_ssize_t)ts.size());
    if (!tuple) throw PythonError{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(tuple);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

// (x, weight, eps, residual, residual_out, out, e4m3, group, scales)
PyObject* rms_norm(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    Call c(x, "x");
    if (x.dim() != 2) refuse(2, "x must be [T, H], got " + shape_text(x.sizes()));
    c.rows(x, "x");
    const int64_t T = x.size(0), H = x.size(1);
    const at::Tensor& w = c.check(tensor(a[1], "weight"), "weight", c.act, {H});
    const float eps = real(a[2], "eps");
    const at::Tensor* residual = tensor_or_none(a[3], "residual");
    at::Tensor added;
    if (residual) {
        c.check(*residual, "residual", c.act, x.sizes(), false);
        added = c.output(a[4], "residual_out", c.act, x.sizes());
    } else if (a[4] != Py_None) {
        refuse(1, "residual_out needs a residual");
    }
    const bool e4m3 = a[6] == Py_True;
    at::Tensor y = c.output(a[5], "out", e4m3 ? at::kFloat8_e4m3fn : c.act, x.sizes()), scales;
    int64_t group = 0;
    if (e4m3) {
        group = integer(a[7], "group");
        if (group < 0 || (group && H % group)) refuse(2, "group=" + std::to_string(group) + " must be 0 or divide H=" + std::to_string(H));
        scales = c.output(a[8], "scales", at::kFloat, {T, group ? H / group : 1});
    }
    done(nvfp4_rms_norm(x.data_ptr(), step(x, 0), residual ? residual->data_ptr() : nullptr, residual ? step(*residual, 0) : 0,
                        w.data_ptr(), T, H, eps, e4m3 ? NVFP4_OUT_E4M3 : NVFP4_OUT_16, group, c.f16, y.data_ptr(),
                        e4m3 ? (float*)scales.data_ptr() : nullptr, residual ? added.data_ptr() : nullptr, c.stream()));
    if (e4m3) return residual ? result({y, scales, added}) : result({y, scales});
    return residual ? result({y, added}) : result({y});
}

// (q, k, v, positions, table, k_cache, v_cache, slots, k_scale, v_scale, sections, interleaved, q_out)
PyObject* rope_cache_write(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0], "q");
    Call c(q, "q");
    if (q.dim() != 3) refuse(2, "q must be [T, Hq, D], got " + shape_text(q.sizes()));
    c.rows(q, "q");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    const nvfp4_kv_cache cache = cache_of(c, a[5], a[6], a[8], a[9]);
    if (cache.head_dim != D) refuse(2, "q has head_dim " + std::to_string(D) + ", the cache " + std::to_string(cache.head_dim));
    const at::Tensor& k = c.check(tensor(a[1], "k"), "k", c.act, {T, cache.heads, D}, false);
    const at::Tensor& v = c.check(tensor(a[2], "v"), "v", c.act, {T, cache.heads, D}, false);
    const at::Tensor& table = tensor(a[4], "table");
    if (table.dim() != 2) refuse(2, "table must be a tensor [rows, rot]");
    c.check(table, "table", at::kFloat, table.sizes());
    const at::Tensor& positions = tensor(a[3], "positions");
    int32_t sections[4];
    int axes = 1;
    if (a[10] == Py_None) {
        if (positions.dim() == 1) c.check(positions, "positions", at::kLong, {T});
        else c.check(positions, "positions", at::kLong, {1, T});
    } else {
        PyObject* seq = PySequence_Fast(a[10], "sections must be a sequence");
        if (!seq) {
            PyErr_Clear();
            refuse(1, "sections must be a list of whole numbers");
        }
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
        bool fine = n >= 1 && n <= 4;
        for (Py_ssize_t i = 0; fine && i < n; ++i) {
            const long s = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
            fine = !(s == -1 && PyErr_Occurred()) && s >= std::numeric_limits<int32_t>::min() && s <= std::numeric_limits<int32_t>::max();
            sections[i] = (int32_t)s;
        }
        PyErr_Clear();
        Py_DECREF(seq);
        if (!fine) refuse(2, "sections must be 1 to 4 whole numbers, one an axis");
        axes = (int)n;
        c.check(positions, "positions", at::kLong, {axes, T});
    }
    const at::Tensor& slots = c.check(tensor(a[7], "slots"), "slots", at::kLong, {T});
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) throw PythonError{};
    at::Tensor q_out = c.output(a[12], "q_out", c.act, q.sizes());
    done(nvfp4_rope_cache_write(q.data_ptr(), step(q, 0), step(q, 1), k.data_ptr(), step(k, 0), step(k, 1), v.data_ptr(), step(v, 0),
                                step(v, 1), T, Hq, (const int64_t*)positions.data_ptr(), axes, a[10] == Py_None ? nullptr : sections,
                                (const float*)table.data_ptr(), table.size(0), table.size(1), interleaved, c.f16,
                                (const int64_t*)slots.data_ptr(), &cache, q_out.data_ptr(), c.stream()));
    return result({q_out});
}

// (k_cache, v_cache, slots, k_scale, v_scale, dtype, k_out, v_out)
PyObject* cache_read(PyObject* const* a) {
    const at::Tensor& k = tensor(a[0], "k_cache");
    Call c(k, "k_cache", false);
    if (a[5] != Py_None) {
        if (!THPDtype_Check(a[5])) refuse(1, "dtype must be torch.bfloat16 or torch.float16");
        c.type(((THPDtype*)a[5])->scalar_type, "dtype");
    } else {
        if (k.scalar_type() == at::kFloat8_e4m3fn) refuse(1, "an E4M3 cache is read as a dtype of torch.bfloat16 or torch.float16");
        c.type(k.scalar_type(), "k_cache");
    }
    const nvfp4_kv_cache cache = cache_of(c, a[0], a[1], a[3], a[4]);
    const at::Tensor& slots = tensor(a[2], "slots");
    if (slots.dim() != 1) refuse(2, "slots must be a tensor [T]");
    c.check(slots, "slots", at::kLong, slots.sizes());
    const int64_t T = slots.size(0);
    at::Tensor ko = c.output(a[6], "k_out", c.act, {T, cache.heads, cache.head_dim});
    at::Tensor vo = c.output(a[7], "v_out", c.act, {T, cache.heads, cache.head_dim});
    done(nvfp4_kv_cache_read(&cache, (const int64_t*)slots.data_ptr(), T, c.f16, ko.data_ptr(), vo.data_ptr(), c.stream()));
    return result({ko, vo});
}

// (q, k_cache, v_cache, block_table, lengths, k_scale, v_scale, softmax_scale, window, out, return_lse, lse, workspace)
PyObject* paged_attention(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0], "q");
    Call c(q, "q");
    if (q.dim() != 3) refuse(2, "q must be [B, Hq, D], got " + shape_text(q.sizes()));
    c.rows(q, "q");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const nvfp4_kv_cache cache = cache_of(c, a[1], a[2], a[5], a[6]);
    if (cache.head_dim != D) refuse(2, "q has head_dim " + std::to_string(D) + ", the cache " + std::to_string(cache.head_dim));
    const at::Tensor& table = tensor(a[3], "block_table");
    if (table.dim() != 2) refuse(2, "block_table must be a tensor [B, width]");
    const int64_t width = table.size(1);
    c.check(table, "block_table", at::kInt, {B, width}, false);
    const at::Tensor& lengths = c.check(tensor(a[4], "lengths"), "lengths", at::kInt, {B});
    const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : real(a[7], "softmax_scale");
    const int64_t window = integer(a[8], "window");
    at::Tensor out = c.output(a[9], "out", c.act, q.sizes()), lse;
    const int with_lse = PyObject_IsTrue(a[10]);
    if (with_lse < 0) throw PythonError{};
    if (with_lse || a[11] != Py_None) lse = c.output(a[11], "lse", at::kFloat, {B, Hq});
    size_t ws_bytes = nvfp4_paged_attention_workspace(B, Hq, cache.heads, D);
    void* ws = nullptr;
    c10::DataPtr held;                                          // given back after the launches, in stream order
    if (const at::Tensor* t = tensor_or_none(a[12], "workspace")) {
        c.check(*t, "workspace", at::kByte, t->sizes());
        ws = t->data_ptr();
        ws_bytes = (size_t)t->numel();
    } else if (ws_bytes) {
        held = c10::cuda::CUDACachingAllocator::get()->allocate(ws_bytes);
        ws = held.get();
    }
    done(nvfp4_paged_attention(q.data_ptr(), step(q, 0), step(q, 1), &cache, (const int32_t*)table.data_ptr(), step(table, 0), width,
                               (const int32_t*)lengths.data_ptr(), B, Hq, scale, window, c.f16, out.data_ptr(),
                               lse.defined() ? (float*)lse.data_ptr() : nullptr, ws, ws_bytes, c.stream()));
    return with_lse ? result({out, lse}) : result({out});
}

// The requests' lengths, block table and stack of free pages of a call.
struct Pool {
    const at::Tensor *lengths, *table, *pages, *count;
    int64_t B, width, page;

    Pool(const Call& c, const at::Tensor& n, PyObject* table_, PyObject* pages_, PyObject* count_, PyObject* page_) {
        if (n.dim() != 1) refuse(2, "lengths must be [B], got " + shape_text(n.sizes()));
        B = n.size(0);
        lengths = &c.check(n, "lengths", at::kInt, {B});
        table = &tensor(table_, "block_table");
        if (table->dim() != 2) refuse(2, "block_table must be a tensor [B, width]");
        width = table->size(1);
        c.check(*table, "block_table", at::kInt, {B, width}, false);
        pages = &tensor(pages_, "free_pages");
        if (pages->dim() != 1) refuse(2, "free_pages must be a tensor [P]");
        c.check(*pages, "free_pages", at::kInt, pages->sizes());
        count = &c.check(tensor(count_, "free_count"), "free_count", at::kInt, {1});
        page = integer(page_, "page_size");
    }
};

// (lengths, new_tokens, block_table, free_pages, free_count, page_size, rows, row_tables, in_place)
PyObject* extend_tables(PyObject* const* a) {
    const at::Tensor& n = tensor(a[0], "lengths");
    Call c(n, "lengths", false);
    const Pool pool(c, n, a[2], a[3], a[4], a[5]);
    const at::Tensor& m = c.check(tensor(a[1], "new_tokens"), "new_tokens", at::kInt, {pool.B});
    const int64_t rows = integer(a[6], "rows");
    if (rows < 0) refuse(1, "rows must not be negative, got " + std::to_string(rows));
    const int tables = PyObject_IsTrue(a[7]), in_place = PyObject_IsTrue(a[8]);
    if (tables < 0 || in_place < 0) throw PythonError{};
    at::Tensor positions = c.output(Py_None, "", at::kLong, {rows}), slots = c.output(Py_None, "", at::kLong, {rows});
    at::Tensor request = c.output(Py_None, "", at::kInt, {rows}), starts = c.output(Py_None, "", at::kInt, {pool.B + 1});
    at::Tensor lengths = in_place ? n : c.output(Py_None, "", at::kInt, {pool.B});
    at::Tensor count = in_place ? *pool.count : c.output(Py_None, "", at::kInt, {1});
    at::Tensor row_tables, row_lengths;
    if (tables) {
        row_tables = c.output(Py_None, "", at::kInt, {rows, pool.width});
        row_lengths = c.output(Py_None, "", at::kInt, {rows});
    }
    done(nvfp4_extend_tables((const int32_t*)n.data_ptr(), (const int32_t*)m.data_ptr(), pool.B, (int32_t*)pool.table->data_ptr(), step(*pool.table, 0),
                             pool.width, (const int32_t*)pool.pages->data_ptr(), pool.pages->numel(), (const int32_t*)pool.count->data_ptr(),
                             pool.page, rows, (int64_t*)positions.data_ptr(), (int64_t*)slots.data_ptr(), (int32_t*)request.data_ptr(),
                             (int32_t*)starts.data_ptr(), (int32_t*)lengths.data_ptr(), (int32_t*)count.data_ptr(),
                             tables ? (int32_t*)row_tables.data_ptr() : nullptr, tables ? (int32_t*)row_lengths.data_ptr() : nullptr, c.stream()));
    if (tables) return result({positions, slots, request, starts, lengths, count, row_tables, row_lengths});
    return result({positions, slots, request, starts, lengths, count});
}

// (lengths, keep, block_table, free_pages, free_count, page_size, in_place)
PyObject* trim_tables(PyObject* const* a) {
    const at::Tensor& n = tensor(a[0], "lengths");
    Call c(n, "lengths", false);
    const Pool pool(c, n, a[2], a[3], a[4], a[5]);
    const at::Tensor& keep = c.check(tensor(a[1], "keep"), "keep", at::kInt, {pool.B});
    const int in_place = PyObject_IsTrue(a[6]);
    if (in_place < 0) throw PythonError{};
    at::Tensor lengths = in_place ? n : c.output(Py_None, "", at::kInt, {pool.B});
    at::Tensor count = in_place ? *pool.count : c.output(Py_None, "", at::kInt, {1});
    done(nvfp4_trim_tables((const int32_t*)n.data_ptr(), (const int32_t*)keep.data_ptr(), pool.B, (const int32_t*)pool.table->data_ptr(),
                           step(*pool.table, 0), pool.width, (int32_t*)pool.pages->data_ptr(), pool.pages->numel(),
                           (const int32_t*)pool.count->data_ptr(), pool.page, (int32_t*)lengths.data_ptr(), (int32_t*)count.data_ptr(), c.stream()));
    return result({lengths, count});
}

// (y, x, a, b, adapters, scales, out, workspace)
PyObject* lora_add(PyObject* const* a) {
    const at::Tensor& y = tensor(a[0], "y");
    Call c(y, "y");
    if (y.dim() != 2) refuse(2, "y must be [T, N], got " + shape_text(y.sizes()));
    c.rows(y, "y");
    const int64_t T = y.size(0), N = y.size(1);
    const at::Tensor &x = tensor(a[1], "x"), &down = tensor(a[2], "a"), &up = tensor(a[3], "b");
    if (down.dim() != 3) refuse(2, "a must be [adapters, r, K], got " + shape_text(down.sizes()));
    const int64_t n = down.size(0), r = down.size(1), K = down.size(2);
    c.check(down, "a", c.act, down.sizes());
    c.check(up, "b", c.act, {n, N, r});
    c.check(x, "x", c.act, {T, K}, false);
    const at::Tensor& ids = c.check(tensor(a[4], "adapters"), "adapters", at::kInt, {T});
    const at::Tensor* scales = tensor_or_none(a[5], "scales");
    if (scales) c.check(*scales, "scales", at::kFloat, {n});
    at::Tensor out = c.output(a[6], "out", c.act, y.sizes());
    size_t ws_bytes = nvfp4_lora_workspace(T, n, r, K);
    void* ws = nullptr;
    c10::DataPtr held;                                          // given back after the launches, in stream order
    if (const at::Tensor* t = tensor_or_none(a[7], "workspace")) {
        c.check(*t, "workspace", at::kByte, t->sizes());
        ws = t->data_ptr();
        ws_bytes = (size_t)t->numel();
    } else if (ws_bytes) {
        held = c10::cuda::CUDACachingAllocator::get()->allocate(ws_bytes);
        ws = held.get();
    }
    done(nvfp4_lora_add(y.data_ptr(), step(y, 0), x.data_ptr(), step(x, 0), down.data_ptr(), up.data_ptr(),
                        scales ? (const float*)scales->data_ptr() : nullptr, (const int32_t*)ids.data_ptr(), T, n, r, K, N, c.f16, out.data_ptr(),
                        ws, ws_bytes, c.stream()));
    return result({out});
}

// (logits, u, temperature, top_k, top_p, min_p, return_logprob, out, logprob)
PyObject* sample(PyObject* const* a) {
    const at::Tensor& logits = tensor(a[0], "logits");
    Call c(logits, "logits", false);
    const auto t = logits.scalar_type();
    if (t != at::kBFloat16 && t != at::kHalf && t != at::kFloat)
        refuse(1, "logits must be torch.bfloat16, torch.float16 or torch.float32, got " + type_text(t));
    if (logits.dim() != 2) refuse(2, "logits must be [B, V], got " + shape_text(logits.sizes()));
    c.rows(logits, "logits");
    const int64_t B = logits.size(0), V = logits.size(1);
    const at::Tensor& u = c.check(tensor(a[1], "u"), "u", at::kFloat, {B});
    nvfp4_sampling how{};
    // A tensor [B], or one number for all rows.
    const auto setting = [&](PyObject* o, Name name, const float** each, float* all) {
        if (THPVariable_Check(o)) *each = (const float*)c.check(THPVariable_Unpack(o), name, at::kFloat, {B}).data_ptr();
        else *all = real(o, name);
    };
    setting(a[2], "temperature", &how.temperature, &how.temperature_all);
    setting(a[4], "top_p", &how.top_p, &how.top_p_all);
    setting(a[5], "min_p", &how.min_p, &how.min_p_all);
    if (THPVariable_Check(a[3])) {
        how.top_k = (const int32_t*)c.check(THPVariable_Unpack(a[3]), "top_k", at::kInt, {B}).data_ptr();
    } else {
        const int64_t k = integer(a[3], "top_k");
        how.top_k_all = (int32_t)std::min<int64_t>(std::max<int64_t>(k, 0), std::numeric_limits<int32_t>::max());
    }
    const int with_logprob = PyObject_IsTrue(a[6]);
    if (with_logprob < 0) throw PythonError{};
    at::Tensor out = c.output(a[7], "out", at::kLong, {B}), logprob;
    if (with_logprob || a[8] != Py_None) logprob = c.output(a[8], "logprob", at::kFloat, {B});
    done(nvfp4_sample(logits.data_ptr(), step(logits, 0), t == at::kBFloat16 ? NVFP4_LOGITS_BF16 : t == at::kHalf ? NVFP4_LOGITS_F16 : NVFP4_LOGITS_F32,
                      B, V, (const float*)u.data_ptr(), &how, (int64_t*)out.data_ptr(), logprob.defined() ? (float*)logprob.data_ptr() : nullptr,
                      c.stream()));
    return with_logprob ? result({out, logprob}) : result({out});
}

// Argument count, and every C++ exception as a Python one.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        PyObject* err = PyObject_CallFunction(g_error, "is", r.status, r.message.c_str());
        if (err) {
            PyErr_SetObject(g_error, err);
            Py_DECREF(err);
        }
    } catch (const PythonError&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* set_error_type(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"set_error_type", set_error_type, METH_O, nullptr},
    ENTRY(rms_norm, 9),
    ENTRY(rope_cache_write, 13),
    ENTRY(cache_read, 8),
    ENTRY(paged_attention, 13),
    ENTRY(extend_tables, 9),
    ENTRY(trim_tables, 7),
    ENTRY(lora_add, 8),
    ENTRY(sample, 9),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nvfp4_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nvfp4_binding(void) { return PyModule_Create(&module); }
