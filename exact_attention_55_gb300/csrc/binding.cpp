// binding.cpp -- the Python binding of the paged-cache entry points, which a decoding loop
// calls a few times per token and layer: argument checks, output allocation and the C call
// in one native step.  A step of a small batch runs 2-7 us on the GPU; marshalled in Python
// a call took 14-36 us on the host, here it takes a third of that or less.
//
// Only marshalling: the C ABI functions come as addresses from the loaded library (bind),
// and their status is returned as an int for the caller to raise.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/attn.h"

namespace {

using at::Tensor;

struct Refusal {
    PyObject* kind;
    std::string text;
};

[[noreturn]] void type_error(const std::string& text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

decltype(&attn_paged_plan) f_plan;
decltype(&attn_cache_append_bf16) f_append_bf16;
decltype(&attn_cache_append_fp8) f_append_fp8;
decltype(&attn_decode_fp8_paged) f_decode;
decltype(&attn_decode_fp8_workspace_bytes) f_decode_ws;

const Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

const Tensor& cuda_tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        type_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

// A contiguous tensor of exactly this type and shape on `dev`.
const Tensor& exact(PyObject* o, std::initializer_list<int64_t> shape, at::ScalarType dtype, at::Device dev,
                    const char* name)
{
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != dtype || t.device() != dev || !t.is_contiguous() ||
        !t.sizes().equals(at::IntArrayRef(shape))) {
        std::string s = "(";
        for (int64_t n : shape) s += std::to_string(n) + ", ";
        type_error(std::string(name) + " must be a contiguous " + c10::toString(dtype) + " tensor of shape " + s +
                   ") on " + dev.str());
    }
    return t;
}

// Makes a call's device and stream current while it allocates and launches: the given
// stream's handle, or None for the device's current one.  What a call allocates (outputs,
// a workspace that goes back when it returns) belongs to the stream it runs on, so nobody
// on another stream can be given that memory while the call's kernels are in flight.  An output
// of a call on a given stream is recorded for the current one too: its caller may read it there,
// after the usual wait, and drop it.
struct On {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard stream;
    c10::optional<c10::cuda::CUDAStream> callers;      // the current stream, where it is another one
    void* handle;

    On(PyObject* given, at::Device dev)
    {
        if (given == Py_None) {
            device.set_device(dev);
            handle = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
            return;
        }
        handle = PyLong_AsVoidPtr(given);
        if (PyErr_Occurred()) throw Refusal{nullptr, ""};
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(dev.index());
        if (current.stream() != handle) callers = current;
        stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), dev.index()));
    }

    Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, at::Device dev) const
    {
        Tensor t = at::detail::empty_cuda(shape, dtype, dev, c10::nullopt);
        if (callers) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *callers);
        return t;
    }

    // The caller's output, checked, or a new one.
    Tensor output(PyObject* o, std::initializer_list<int64_t> shape, at::ScalarType dtype, at::Device dev,
                  const char* name) const
    {
        if (o != Py_None) return exact(o, shape, dtype, dev, name);
        return empty(at::IntArrayRef(shape), dtype, dev);
    }
};

int int_arg(PyObject* o, const char* name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    if (v < -2147483647LL - 1 || v > 2147483647LL) value_error(std::string(name) + " does not fit an int");
    return (int)v;
}

int size_arg(int64_t n, const char* name)
{
    if (n > 2147483647LL) value_error(std::string(name) + " does not fit an int");
    return (int)n;
}

PyObject* status(attn_status_t st) { return PyLong_FromLong(st); }

template <class Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body body) noexcept
{
    try {
        if (given != wanted) type_error("wrong number of arguments");
        return body();
    } catch (const Refusal& r) {
        if (r.kind) PyErr_SetString(r.kind, r.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error in the binding");
    }
    return nullptr;
}

PyObject* tuple_of(std::initializer_list<Tensor> ts)
{
    PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) throw Refusal{nullptr, ""};
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(out);
            throw Refusal{nullptr, ""};
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

// new_lens, seq_lens, page_table, free_pages, free_count, page_size, num_tokens, six outputs, stream
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 14, [&]() -> PyObject* {
        const Tensor& new_lens = cuda_tensor(a[0], "new_lens");
        const at::Device dev = new_lens.device();
        const int64_t B = new_lens.numel();
        exact(a[0], {B}, at::kInt, dev, "new_lens");
        const Tensor& seq_lens = exact(a[1], {B}, at::kInt, dev, "seq_lens");
        const Tensor& table = tensor(a[2], "page_table");
        if (table.dim() != 2) type_error("page_table must be an int32 [B, max_pages] tensor");
        const int64_t width = table.size(1);
        exact(a[2], {B, width}, at::kInt, dev, "page_table");
        const Tensor& pages = tensor(a[3], "free_pages");
        if (pages.dim() != 1) type_error("free_pages must be an int32 [capacity] tensor");
        exact(a[3], {pages.numel()}, at::kInt, dev, "free_pages");
        const Tensor& count = exact(a[4], {1}, at::kInt, dev, "free_count");
        const int ps = int_arg(a[5], "page_size"), T = int_arg(a[6], "num_tokens");
        if (T < 0) value_error("num_tokens must not be negative");
        const On on(a[13], dev);
        // new outputs share one allocation, each from a 16-byte boundary on
        auto room = [](int64_t bytes) { return (bytes + 15) / 16 * 16; };
        Tensor whole;
        int64_t used = 0;
        auto out = [&](PyObject* given, int64_t count, at::ScalarType dtype, const char* name) {
            if (given != Py_None) return exact(given, {count}, dtype, dev, name);
            if (!whole.defined())
                whole = on.empty({room(8LL * T) + room(4LL * T) + 2 * room(4 * B) + room(4 * B + 4) + 16}, at::kByte, dev);
            const int64_t size = (int64_t)c10::elementSize(dtype);
            Tensor t = at::detail::make_tensor<c10::TensorImpl>(
                c10::Storage(whole.storage()), whole.key_set(), c10::scalarTypeToTypeMeta(dtype));
            t.unsafeGetTensorImpl()->set_storage_offset(used / size);
            t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(&count, 1));
            used += room(count * size);
            return t;
        };
        const Tensor seq_out = out(a[7], B, at::kInt, "seq_lens_out");
        const Tensor count_out = out(a[8], 1, at::kInt, "free_count_out");
        const Tensor cu = out(a[9], B + 1, at::kInt, "cu_new");
        const Tensor slots = out(a[10], T, at::kLong, "slot_map");
        const Tensor pos = out(a[11], T, at::kInt, "positions");
        const Tensor served = out(a[12], B, at::kInt, "served");
        auto ints = [](const Tensor& t) { return static_cast<int*>(t.data_ptr()); };
        const attn_status_t st =
            f_plan(ints(new_lens), ints(seq_lens), ints(table), ints(pages), ints(count), ints(seq_out),
                   ints(count_out), ints(cu), static_cast<long long*>(slots.data_ptr()), ints(pos), ints(served),
                   size_arg(B, "B"), ps, size_arg(width, "max_pages"), size_arg(pages.numel(), "free_pages"), T,
                   on.handle);
        if (st != ATTN_OK) return status(st);
        return tuple_of({seq_out, count_out, cu, slots, pos, served});
    });
}

struct Append {
    at::Device dev;
    int T, H, d, ps, pages;
    long long k_stride, v_stride;
};

bool code_type(at::ScalarType t)
{
    return t == at::kByte || t == at::kFloat8_e4m3fn || t == at::kFloat8_e5m2;
}

void check_cache(const Tensor& t, at::Device dev, bool bits8, const char* name)
{
    if ((bits8 ? !code_type(t.scalar_type()) : t.scalar_type() != at::kBFloat16) || t.device() != dev ||
        t.dim() != 4 || !t.is_contiguous())
        type_error(std::string(name) + " must be a contiguous " + (bits8 ? "8-bit" : "bf16") +
                   " [num_pages, Hkv, page_size, d] tensor on " + dev.str());
}

// k, v, k_cache, v_cache, slot_map
Append append_args(PyObject* const* a, PyObject* slot_map, bool bits8)
{
    const Tensor& k = cuda_tensor(a[0], "k");
    const Tensor& v = tensor(a[1], "v");
    const at::Device dev = k.device();
    for (const Tensor* t : {&k, &v})
        if (t->scalar_type() != at::kBFloat16 || t->device() != dev || t->dim() != 3)
            type_error("k and v must be bf16 [T, Hkv, d] tensors on " + dev.str());
    if (!v.sizes().equals(k.sizes())) value_error("k and v must have the same shape");
    const int64_t T = k.size(0), H = k.size(1), d = k.size(2);
    for (const Tensor* t : {&k, &v})
        if ((d > 1 && t->stride(2) != 1) || (H > 1 && t->stride(1) != d))
            value_error("k and v: the heads of a token must be contiguous");
    const Tensor& kc = tensor(a[2], "k_cache");
    const Tensor& vc = tensor(a[3], "v_cache");
    check_cache(kc, dev, bits8, "k_cache");
    check_cache(vc, dev, bits8, "v_cache");
    if (!vc.sizes().equals(kc.sizes()) || kc.size(1) != H || kc.size(3) != d)
        value_error("the caches must be [num_pages, Hkv, page_size, d] with k's heads and d");
    exact(slot_map, {T}, at::kLong, dev, "slot_map");
    return {dev, size_arg(T, "T"), size_arg(H, "Hkv"), size_arg(d, "d"), size_arg(kc.size(2), "page_size"),
            size_arg(kc.size(0), "num_pages"), T > 1 ? (long long)k.stride(0) : (long long)(H * d),
            T > 1 ? (long long)v.stride(0) : (long long)(H * d)};
}

void* ptr(PyObject* o) { return THPVariable_Unpack(o).data_ptr(); }

// k, v, k_cache, v_cache, slot_map, stream
PyObject* append_bf16(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject* {
        const Append p = append_args(a, a[4], false);
        const On on(a[5], p.dev);
        return status(f_append_bf16(ptr(a[0]), ptr(a[1]), ptr(a[2]), ptr(a[3]), static_cast<long long*>(ptr(a[4])),
                                    p.T, p.H, p.d, p.k_stride, p.v_stride, p.ps, p.pages, on.handle));
    });
}

// Rows per scale block, from the scales' shape; a typed cache has to hold the format's codes.
int block_of(PyObject* kc_, PyObject* vc_, PyObject* ks, PyObject* vs, int format, at::Device dev)
{
    const Tensor& kc = THPVariable_Unpack(kc_);
    const at::ScalarType typed = format == ATTN_FP8_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
    for (const Tensor* t : {&kc, &THPVariable_Unpack(vc_)})
        if (t->scalar_type() != at::kByte && t->scalar_type() != typed)
            type_error(std::string("the cache holds ") + c10::toString(t->scalar_type()) + ", not the format's codes");
    const Tensor& s = tensor(ks, "k_scales");
    if (s.dim() != 3 || s.size(2) < 1)
        type_error("k_scales must be a float32 [num_pages, Hkv, page_size / block] tensor");
    const int64_t nblk = s.size(2);
    exact(ks, {kc.size(0), kc.size(1), nblk}, at::kFloat, dev, "k_scales");
    exact(vs, {kc.size(0), kc.size(1), nblk}, at::kFloat, dev, "v_scales");
    if (kc.size(2) % nblk != 0) value_error("the scales' blocks must divide the page");
    return size_arg(kc.size(2) / nblk, "block");
}

// k, v, k_cache, v_cache, k_scales, v_scales, slot_map, format, stream
PyObject* append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        const Append p = append_args(a, a[6], true);
        const int format = int_arg(a[7], "format");
        const int block = block_of(a[2], a[3], a[4], a[5], format, p.dev);
        const On on(a[8], p.dev);
        return status(f_append_fp8(ptr(a[0]), ptr(a[1]), ptr(a[2]), ptr(a[3]), static_cast<float*>(ptr(a[4])),
                                   static_cast<float*>(ptr(a[5])), static_cast<long long*>(ptr(a[6])), p.T, p.H, p.d,
                                   p.k_stride, p.v_stride, p.ps, p.pages, block, format, on.handle));
    });
}

// q, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, format, scale or None, window,
// workspace, o, lse, stream
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 14, [&]() -> PyObject* {
        const Tensor& q = cuda_tensor(a[0], "q");
        const at::Device dev = q.device();
        if (q.scalar_type() != at::kBFloat16) type_error("q must be bf16");
        if (q.dim() != 4 || !q.is_contiguous()) value_error("q must be a contiguous [B, H, nq, d] tensor");
        const int64_t B = q.size(0), H = q.size(1), nq = q.size(2), d = q.size(3);
        const Tensor& kc = tensor(a[1], "k_cache");
        const Tensor& vc = tensor(a[2], "v_cache");
        check_cache(kc, dev, true, "k_cache");
        check_cache(vc, dev, true, "v_cache");
        if (!vc.sizes().equals(kc.sizes()) || kc.size(3) != d)
            value_error("the caches must be [num_pages, Hkv, page_size, d] with q's d");
        const int format = int_arg(a[7], "format");
        const int block = block_of(a[1], a[2], a[3], a[4], format, dev);
        const Tensor& table = tensor(a[5], "page_table");
        if (table.dim() != 2) type_error("page_table must be an int32 [B, max_pages] tensor");
        exact(a[5], {B, table.size(1)}, at::kInt, dev, "page_table");
        const Tensor& lens = exact(a[6], {B}, at::kInt, dev, "seq_lens");
        float scale = (float)(1.0 / std::sqrt((double)(d > 0 ? d : 1)));
        if (a[8] != Py_None) {
            scale = (float)PyFloat_AsDouble(a[8]);
            if (PyErr_Occurred()) throw Refusal{nullptr, ""};
        }
        const int window = int_arg(a[9], "window");
        const int h = size_arg(H, "H"), hkv = size_arg(kc.size(1), "Hkv"), nqi = size_arg(nq, "nq"), di = size_arg(d, "d");
        const On on(a[13], dev);
        // without a workspace of the caller's: the stream's allocator lends one for the call
        c10::DataPtr lent;
        void* ws = nullptr;
        size_t ws_bytes = 0;
        if (a[10] == Py_None) {
            ws_bytes = f_decode_ws(h, hkv, nqi, di);
            lent = c10::cuda::CUDACachingAllocator::get()->allocate(ws_bytes);
            ws = lent.get();
        } else {
            const Tensor& given = tensor(a[10], "workspace");
            if (given.device() != dev || !given.is_contiguous())
                type_error("workspace must be a contiguous CUDA tensor on " + dev.str());
            ws = given.data_ptr();
            ws_bytes = (size_t)given.nbytes();
        }
        const Tensor o = on.output(a[11], {B, H, nq, d}, at::kBFloat16, dev, "o");
        const Tensor lse = on.output(a[12], {B, H, nq}, at::kFloat, dev, "lse");
        const attn_status_t st = f_decode(
            q.data_ptr(), kc.data_ptr(), vc.data_ptr(), static_cast<float*>(ptr(a[3])), static_cast<float*>(ptr(a[4])),
            static_cast<int*>(table.data_ptr()), static_cast<int*>(lens.data_ptr()), o.data_ptr(),
            static_cast<float*>(lse.data_ptr()), size_arg(B, "B"), h, hkv, nqi, di, size_arg(kc.size(2), "page_size"),
            size_arg(kc.size(0), "num_pages"), size_arg(table.size(1), "max_pages"), block, format, scale, window,
            ws, ws_bytes, on.handle);
        if (st != ATTN_OK) return status(st);
        return tuple_of({o, lse});
    });
}

// The addresses of the five C functions, in the order below.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 5, [&]() -> PyObject* {
        void* f[5];
        for (int i = 0; i < 5; ++i) {
            f[i] = PyLong_AsVoidPtr(a[i]);
            if (PyErr_Occurred()) throw Refusal{nullptr, ""};
        }
        f_plan = reinterpret_cast<decltype(f_plan)>(f[0]);
        f_append_bf16 = reinterpret_cast<decltype(f_append_bf16)>(f[1]);
        f_append_fp8 = reinterpret_cast<decltype(f_append_fp8)>(f[2]);
        f_decode = reinterpret_cast<decltype(f_decode)>(f[3]);
        f_decode_ws = reinterpret_cast<decltype(f_decode_ws)>(f[4]);
        Py_RETURN_NONE;
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),           method<plan>("plan"),
                         method<append_bf16>("append_bf16"), method<append_fp8>("append_fp8"),
                         method<decode>("decode"),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gb300attn_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gb300attn_binding() { return PyModule_Create(&module); }
