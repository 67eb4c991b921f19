// ops_binding.cpp -- Python binding of include/ar_ops.h as an extension module.
//
// What ctypes does for the rest of the library costs a call of these small
// operators more than their kernels run, so their tensors are checked, their outputs
// allocated and their arguments marshalled here.  ops.py holds the public
// functions, with the defaults and the documentation.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <optional>
#include <string>
#include <utility>
#include <vector>

#include "ar_ops.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;   // ArError

struct Refused {
    std::string why;
};

[[noreturn]] void refuse(const char *what, const std::string &why) { throw Refused{std::string(what) + ": " + why}; }

std::string name_of(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return std::string("torch.") + at::toString(t);
    }
}

std::string name_of(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor &tensor(const char *what, PyObject *o) {
    if (!THPVariable_Check(o)) refuse(what, "not a tensor");
    return THPVariable_Unpack(o);
}

// The device of the tensor that the others go by: the current one.
int device_of(const char *what, const Tensor &t) {
    if (!t.is_cuda()) refuse(what, "not a CUDA tensor");
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device()) refuse(what, "on " + t.device().str() + ", which is not the current device");
    return dev;
}

constexpr at::ScalarType kAny = at::ScalarType::Undefined;

// One tensor on device dev, of this type and rank; dense: contiguous, else its last dimension is.
void check(const char *what, const Tensor &t, int dev, at::ScalarType type, int64_t rank, bool dense) {
    if (!t.is_cuda()) refuse(what, "not a CUDA tensor");
    if (t.get_device() != dev) refuse(what, "on " + t.device().str() + ", not cuda:" + std::to_string(dev));
    if (type != kAny && t.scalar_type() != type) refuse(what, "dtype " + name_of(t.scalar_type()) + ", not " + name_of(type));
    if (t.dim() != rank) refuse(what, std::to_string(t.dim()) + " dimensions, not " + std::to_string(rank));
    if (dense ? !t.is_contiguous() : t.size(-1) > 1 && t.stride(-1) != 1)
        refuse(what, dense ? "not contiguous" : "its last dimension is not contiguous");
}

// A tensor that is written by its strides: an expanded one has several writers to an element.
void check_written(const char *what, const Tensor &t) {
    if (at::has_internal_overlap(t) == at::MemOverlap::Yes) refuse(what, "its elements overlap (an expanded tensor?)");
}

void check_shape(const char *what, const Tensor &t, at::IntArrayRef shape) {
    if (t.sizes() != shape) refuse(what, "shape " + name_of(t.sizes()) + ", not " + name_of(shape));
}

int code_16(const char *what, const Tensor &t) {
    if (t.scalar_type() == at::kHalf) return AR_F16;
    if (t.scalar_type() == at::kBFloat16) return AR_BF16;
    refuse(what, "dtype " + name_of(t.scalar_type()) + " is neither float16 nor bfloat16");
}

int64_t whole(const char *what, PyObject *o, int64_t low, int64_t high) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(what, "not a whole number");
    }
    if (v < low || v > high) refuse(what, std::to_string(v) + " is not within " + std::to_string(low) + " .. " + std::to_string(high));
    return v;
}

double real(const char *what, PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(what, "not a number");
    }
    return v;
}

constexpr int64_t kInt = 0x7fffffff;

Tensor make(at::IntArrayRef shape, at::ScalarType type, const Tensor &like) {
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);      // (without the dispatcher's way there)
}

// n elements of another tensor's memory, from a byte on: cheaper than an allocation of their own.
Tensor part_of(const Tensor &room, at::ScalarType type, int64_t byte, int64_t n) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(room.storage()), room.key_set(),
                                                        c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(byte / (int64_t)c10::elementSize(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
}

ar_stream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// The capture that a stream is part of, by its id; 0: none.
unsigned long long capture_of(ar_stream_t stream) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(stream, &status, &id) != cudaSuccess) {
        (void)cudaGetLastError();      // (the legacy stream beside another's capture: the launch will say so)
        return 0;
    }
    return status == cudaStreamCaptureStatusActive ? id : 0;
}

PyObject *fail(int rc, const char *call) {
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, call);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

PyObject *tuple_of(std::initializer_list<const Tensor *> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const Tensor *t : ts) {
        PyObject *o = t ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
        if (!r || !o) {
            Py_XDECREF(r);
            Py_XDECREF(o);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

struct Pool {
    int64_t pages, heads, dim, page;
};

Pool pool_of(const Tensor &p, int dev) {
    check("pool", p, dev, at::kByte, 4, true);
    const int64_t bytes = p.size(3);
    if ((bytes != 1152 && bytes != 2304 && bytes != 4608) || p.size(1) < 1 || p.size(2) < 1)
        refuse("pool", "shape " + name_of(p.sizes()) + " is not [pages, kv heads, page / 16, 18 * head_dim]");
    return {p.size(0), p.size(1), bytes / 18, p.size(2) * 16};
}

// ------------------------------------------------------------------ operators

// plan(lens, new, table, free_pages, free_used, page, max_tokens, out | None) -> (stream handle, 7 tensors or out)
PyObject *plan(PyObject *const *o) {
    const Tensor &lens = tensor("lens", o[0]), &fresh = tensor("new", o[1]), &table = tensor("table", o[2]), &pages = tensor("free_pages", o[3]),
                 &used = tensor("free_used", o[4]);
    const int dev = device_of("lens", lens);
    check("lens", lens, dev, at::kInt, 1, true);
    const int64_t B = lens.size(0);
    check("new", fresh, dev, at::kInt, 1, true);
    check_shape("new", fresh, {B});
    check("table", table, dev, at::kInt, 2, false);
    if (table.size(0) != B) refuse("table", std::to_string(table.size(0)) + " rows for " + std::to_string(B) + " requests");
    check("free_pages", pages, dev, at::kInt, 1, true);
    check("free_used", used, dev, at::kInt, 1, true);
    check_shape("free_used", used, {1});
    const int64_t page = whole("page", o[5], -kInt, kInt), cap = whole("max_tokens", o[6], INT64_MIN, kInt);
    if (cap < 0) refuse("max_tokens", "is negative");
    static const char *const names[7] = {"out.lens", "out.cu", "out.request", "out.position", "out.free_used", "out.status", "out.slots"};
    const int64_t sizes[7] = {B, B + 1, cap, cap, 1, 1, cap};
    if (o[7] != Py_None && (!PyTuple_Check(o[7]) || PyTuple_GET_SIZE(o[7]) != 7)) refuse("out", "not a KvPlan");
    Tensor out[7], room;
    int64_t at = 8 * cap;        // slots come first
    if (o[7] == Py_None) room = make({cap + B + 2 + cap}, at::kLong, lens);
    for (int i = 0; i < 7; ++i) {
        const at::ScalarType type = i == 6 ? at::kLong : at::kInt;
        if (o[7] == Py_None) {
            out[i] = part_of(room, type, i == 6 ? 0 : at, sizes[i]);
            if (i < 6) at += 4 * sizes[i];
        } else {
            out[i] = tensor(names[i], PyTuple_GET_ITEM(o[7], i));
            check(names[i], out[i], dev, type, 1, true);
            check_shape(names[i], out[i], {sizes[i]});
        }
    }
    ar_kv_plan_args a = {};
    auto p = [](const Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); };
    a.lens = p(lens); a.new_tokens = p(fresh); a.table = p(table); a.free_pages = p(pages); a.free_used = p(used);
    a.lens_out = p(out[0]); a.cu = p(out[1]); a.request = p(out[2]); a.position = p(out[3]); a.free_used_out = p(out[4]);
    a.status = p(out[5]); a.slots = static_cast<int64_t *>(out[6].data_ptr());
    a.table_stride = B > 1 ? table.stride(0) : table.size(1);
    a.free_count = pages.size(0); a.requests = (int32_t)B; a.table_width = (int32_t)table.size(1); a.page = (int32_t)page; a.max_tokens = (int32_t)cap;
    const ar_stream_t stream = stream_of(dev);
    const int rc = ar_kv_plan(&a, stream);
    if (rc) return fail(rc, "ar_kv_plan");
    PyObject *made = o[7] != Py_None ? (Py_INCREF(o[7]), o[7])
                                     : tuple_of({&out[0], &out[1], &out[2], &out[3], &out[4], &out[5], &out[6]});
    return made ? Py_BuildValue("KN", (unsigned long long)(uintptr_t)stream, made) : nullptr;
}

int rows(bool append, const Tensor &k, const Tensor &v, const Tensor &pool, const Pool &dims, const Tensor &slots, int dev) {
    const int64_t n = slots.size(0);
    const int code = code_16("k", k);
    check("k", k, dev, kAny, 3, false);
    check_shape("k", k, {n, dims.heads, dims.dim});
    check("v", v, dev, k.scalar_type(), 3, false);
    check_shape("v", v, {n, dims.heads, dims.dim});
    if (!append) {
        check_written("out", k);
        check_written("out", v);
    }
    ar_kv4_rows_args a = {};
    a.k = k.data_ptr(); a.v = v.data_ptr(); a.pool = pool.data_ptr(); a.slots = static_cast<int64_t *>(slots.data_ptr());
    a.k_token_stride = k.stride(0); a.k_head_stride = k.stride(1); a.v_token_stride = v.stride(0); a.v_head_stride = v.stride(1);
    a.pages = dims.pages; a.tokens = n; a.dtype = code; a.kv_heads = (int32_t)dims.heads; a.head_dim = (int32_t)dims.dim; a.page = (int32_t)dims.page;
    return append ? ar_kv4_append(&a, stream_of(dev)) : ar_kv4_load(&a, stream_of(dev));
}

// append(k, v, pool, slots)
PyObject *append(PyObject *const *o) {
    const Tensor &k = tensor("k", o[0]), &v = tensor("v", o[1]), &pool = tensor("pool", o[2]), &slots = tensor("slots", o[3]);
    const int dev = device_of("pool", pool);
    const Pool dims = pool_of(pool, dev);
    check("slots", slots, dev, at::kLong, 1, true);
    const int rc = rows(true, k, v, pool, dims, slots, dev);
    return rc ? fail(rc, "ar_kv4_append") : (Py_INCREF(Py_None), Py_None);
}

// load(pool, slots, dtype | None, out | None) -> (k, v)
PyObject *load(PyObject *const *o) {
    const Tensor &pool = tensor("pool", o[0]), &slots = tensor("slots", o[1]);
    const int dev = device_of("pool", pool);
    const Pool dims = pool_of(pool, dev);
    check("slots", slots, dev, at::kLong, 1, true);
    if (o[2] != Py_None && !THPDtype_Check(o[2])) refuse("dtype", "not a torch.dtype");
    const at::ScalarType type = o[2] == Py_None ? at::kBFloat16 : reinterpret_cast<THPDtype *>(o[2])->scalar_type;
    Tensor k, v;
    if (o[3] == Py_None) {
        if (type != at::kHalf && type != at::kBFloat16) refuse("k", "dtype " + name_of(type) + " is neither float16 nor bfloat16");
        k = make({slots.size(0), dims.heads, dims.dim}, type, pool);
        v = make({slots.size(0), dims.heads, dims.dim}, type, pool);
    } else {
        if (!PyTuple_Check(o[3]) || PyTuple_GET_SIZE(o[3]) != 2) refuse("out", "not a pair of tensors");
        k = tensor("out", PyTuple_GET_ITEM(o[3], 0));
        v = tensor("out", PyTuple_GET_ITEM(o[3], 1));
        if (o[2] != Py_None && k.scalar_type() != type) refuse("out", "dtype " + name_of(k.scalar_type()) + ", not " + name_of(type));
    }
    const int rc = rows(false, k, v, pool, dims, slots, dev);
    if (rc) return fail(rc, "ar_kv4_load");
    if (o[3] != Py_None) return Py_INCREF(o[3]), o[3];
    return tuple_of({&k, &v});
}

// Workspaces of kv4_attend by device and stream, for calls that are not captured; ops.py makes them and keeps
// them alive.
struct Place {
    int dev;
    ar_stream_t stream;
    void *ws;
};
std::vector<Place> g_places;   // guarded by the interpreter's lock

// attend(q, pool, table, lens, cu | None, max_new | None, window, sinks, scale | None, out | None, lse | None, return_lse, workspace | None)
//   -> out, (out, lse), or None where no workspace was given and the stream has none yet or is being captured
PyObject *attend(PyObject *const *o) {
    const Tensor &q = tensor("q", o[0]), &pool = tensor("pool", o[1]), &table = tensor("table", o[2]), &lens = tensor("lens", o[3]);
    const int dev = device_of("pool", pool);
    const Pool dims = pool_of(pool, dev);
    check("q", q, dev, kAny, 3, false);
    const int64_t T = q.size(0), heads = q.size(1);
    if (q.size(2) != dims.dim) refuse("q", "head_dim " + std::to_string(q.size(2)) + ", the pool's is " + std::to_string(dims.dim));
    if (heads < 1 || heads % dims.heads) refuse("q", std::to_string(heads) + " heads for " + std::to_string(dims.heads) + " kv heads");
    const int code = code_16("q", q);
    check("lens", lens, dev, at::kInt, 1, true);
    const int64_t B = lens.size(0);
    check("table", table, dev, at::kInt, 2, false);
    if (table.size(0) != B) refuse("table", std::to_string(table.size(0)) + " rows for " + std::to_string(B) + " requests");
    const bool many = o[4] != Py_None;
    const int32_t *cu = nullptr;
    if (many) {
        const Tensor &c = tensor("cu", o[4]);
        check("cu", c, dev, at::kInt, 1, true);
        check_shape("cu", c, {B + 1});
        cu = static_cast<int32_t *>(c.data_ptr());
    } else if (T != B) {
        refuse("q", std::to_string(T) + " tokens for " + std::to_string(B) + " requests, and no cu");
    }
    const ar_stream_t stream = stream_of(dev);
    void *ws = nullptr;
    if (o[12] != Py_None) {
        ws = PyLong_AsVoidPtr(o[12]);
    } else {
        if (!capture_of(stream))
            for (const Place &p : g_places)
                if (p.dev == dev && p.stream == stream) ws = p.ws;
        if (!ws) return Py_INCREF(Py_None), Py_None;
    }
    Tensor out, lse;
    if (o[9] == Py_None) {
        out = make(q.sizes(), q.scalar_type(), q);
    } else {
        out = tensor("out", o[9]);
        check("out", out, dev, q.scalar_type(), 3, false);
        check_shape("out", out, q.sizes());
        check_written("out", out);
    }
    if (o[10] != Py_None) {
        lse = tensor("lse", o[10]);
        check("lse", lse, dev, at::kFloat, 2, true);
        check_shape("lse", lse, {T, heads});
    } else if (PyObject_IsTrue(o[11]) == 1) {
        lse = make({T, heads}, at::kFloat, q);
    }
    ar_kv4_attend_args a = {};
    a.q = q.data_ptr(); a.out = out.data_ptr(); a.lse = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr; a.pool = pool.data_ptr();
    a.table = static_cast<int32_t *>(table.data_ptr()); a.lens = static_cast<int32_t *>(lens.data_ptr()); a.cu = cu; a.workspace = ws;
    a.q_token_stride = q.stride(0); a.q_head_stride = q.stride(1); a.out_token_stride = out.stride(0); a.out_head_stride = out.stride(1);
    a.table_stride = B > 1 ? table.stride(0) : table.size(1); a.pages = dims.pages;
    a.dtype = code; a.tokens = (int32_t)T; a.requests = (int32_t)B;
    a.max_new = o[5] != Py_None ? (int32_t)whole("max_new", o[5], -kInt, kInt) : many ? (int32_t)T : 1;
    a.q_heads = (int32_t)heads; a.kv_heads = (int32_t)dims.heads; a.head_dim = (int32_t)dims.dim; a.page = (int32_t)dims.page;
    a.table_width = (int32_t)table.size(1); a.window = (int32_t)whole("window", o[6], -kInt, kInt); a.sinks = (int32_t)whole("sinks", o[7], -kInt, kInt);
    a.scale = o[8] == Py_None ? (float)(1.0 / std::sqrt((double)dims.dim)) : (float)real("scale", o[8]);
    const int rc = ar_kv4_attend(&a, stream);
    if (rc) return fail(rc, "ar_kv4_attend");
    if (!lse.defined()) return o[9] != Py_None ? (Py_INCREF(o[9]), o[9]) : THPVariable_Wrap(out);
    return o[9] == Py_None && o[10] == Py_None ? tuple_of({&out, &lse})
                                               : Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// norm(x, weight, residual | None, eps, group, out | None, scales | None, residual_out | None) -> (out,
// scales, residual_out | None)
PyObject *norm(PyObject *const *o) {
    const Tensor &x = tensor("x", o[0]), &w = tensor("weight", o[1]);
    const int dev = device_of("x", x);
    check("x", x, dev, kAny, 2, false);
    const int code = code_16("x", x);
    const at::ScalarType type = x.scalar_type();
    const int64_t N = x.size(0), d = x.size(1);
    check("weight", w, dev, type, 1, true);
    check_shape("weight", w, {d});
    const int64_t group = whole("group", o[4], 0, d), groups = group ? (d + group - 1) / group : 1;
    ar_add_norm_fp8_args a = {};
    Tensor out, scales, after;
    if (o[2] != Py_None) {
        const Tensor &r = tensor("residual", o[2]);
        check("residual", r, dev, type, 2, false);
        check_shape("residual", r, x.sizes());
        a.residual = r.data_ptr();
        a.residual_stride = r.stride(0);
    }
    if (o[7] != Py_None) {
        after = tensor("residual_out", o[7]);
        check("residual_out", after, dev, type, 2, false);
        check_shape("residual_out", after, x.sizes());
        check_written("residual_out", after);
    } else if (o[2] != Py_None) {      // (an empty residual has no address)
        after = make(x.sizes(), type, x);
    }
    if (o[5] != Py_None) {
        out = tensor("out", o[5]);
        check("out", out, dev, at::kFloat8_e4m3fn, 2, true);
        check_shape("out", out, x.sizes());
    } else {
        out = make(x.sizes(), at::kFloat8_e4m3fn, x);
    }
    if (o[6] != Py_None) {
        scales = tensor("scales", o[6]);
        check("scales", scales, dev, at::kFloat, 2, true);
        check_shape("scales", scales, {N, groups});
    } else {
        scales = make({N, groups}, at::kFloat, x);
    }
    a.x = x.data_ptr(); a.weight = w.data_ptr(); a.out = out.data_ptr(); a.scales = static_cast<float *>(scales.data_ptr());
    a.x_stride = x.stride(0); a.rows = N; a.dtype = code; a.dim = (int32_t)d; a.group = (int32_t)group; a.eps = (float)real("eps", o[3]);
    if (after.defined()) {
        a.residual_out = after.data_ptr();
        a.residual_out_stride = after.stride(0);
    }
    if (d > kInt) refuse("x", "rows too long");
    const int rc = ar_add_norm_fp8(&a, stream_of(dev));
    if (rc) return fail(rc, "ar_add_norm_fp8");
    return tuple_of({&out, &scales, after.defined() ? &after : nullptr});
}

// set_workspace(dev, stream, address): the workspace of a stream from now on
PyObject *set_workspace(PyObject *const *o) {
    const int dev = (int)whole("device", o[0], 0, kInt);
    const ar_stream_t s = static_cast<ar_stream_t>(PyLong_AsVoidPtr(o[1]));
    void *ws = PyLong_AsVoidPtr(o[2]);
    for (Place &p : g_places)
        if (p.dev == dev && p.stream == s) {
            p.ws = ws;
            Py_RETURN_NONE;
        }
    g_places.push_back({dev, s, ws});
    Py_RETURN_NONE;
}

// capture_id(stream): of the capture that the stream is part of, 0 if none
PyObject *capture_id(PyObject *const *o) {
    return PyLong_FromUnsignedLongLong(capture_of(static_cast<ar_stream_t>(PyLong_AsVoidPtr(o[0]))));
}

PyObject *set_error(PyObject *const *o) {
    Py_INCREF(o[0]);
    Py_XDECREF(g_error);
    g_error = o[0];
    Py_RETURN_NONE;
}

// No C++ exception leaves the module.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments wanted, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.why.c_str());
    } catch (const std::exception &) {
        torch::translate_exception_to_python(std::current_exception());   // out of memory among them
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<plan, 8>("plan"), method<append, 4>("append"), method<load, 4>("load"), method<attend, 13>("attend"),
                           method<norm, 8>("norm"), method<set_workspace, 3>("set_workspace"), method<capture_id, 1>("capture_id"),
                           method<set_error, 1>("set_error"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__ops_binding() { return PyModule_Create(&g_module); }
