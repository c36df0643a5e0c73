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
decltype(&attn_rope_bf16) f_rope;
decltype(&attn_diff_fwd_bf16) f_diff_fwd;
decltype(&attn_diff_fwd_bf16_varlen) f_diff_fwd_varlen;
decltype(&attn_diff_bwd_bf16) f_diff_bwd;
decltype(&attn_diff_bwd_bf16_varlen) f_diff_bwd_varlen;
decltype(&attn_diff_bwd_workspace_bytes) f_diff_bwd_ws;
decltype(&attn_diff_decode_bf16_paged) f_diff_decode;
decltype(&attn_diff_decode_workspace_bytes) f_diff_decode_ws;

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

// ------------------------------------------------------------------ rotary positions

// bf16 rows of q or k: [T, H, d] or [B, H, N, d], elements of a row contiguous.
void check_rows(const Tensor& t, at::Device dev, const char* name)
{
    if (t.scalar_type() != at::kBFloat16 || t.device() != dev || (t.dim() != 3 && t.dim() != 4))
        type_error(std::string(name) + " must be a bf16 [T, H, d] or [B, H, N, d] tensor on " + dev.str());
    if (t.size(-1) > 1 && t.stride(-1) != 1) value_error(std::string(name) + ": a row's elements must be contiguous");
}

// Strides of batch, token and head; that of a single index does not matter.
void row_strides(const Tensor& t, bool written, const char* name, long long* out)
{
    const int dims[3] = {t.dim() == 4 ? 0 : -1, t.dim() == 4 ? 2 : 0, 1};
    for (int i = 0; i < 3; ++i) {
        const bool one = dims[i] < 0 || t.size(dims[i]) <= 1;
        out[i] = one ? 0 : (long long)t.stride(dims[i]);
        if (written && !one && out[i] == 0) value_error(std::string(name) + " has several indices at one place");
    }
}

// q, k or None, positions, inv_freq, axis or None, interleaved, inverse, q_out, k_out, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject* {
        const Tensor& q = cuda_tensor(a[0], "q");
        const at::Device dev = q.device();
        check_rows(q, dev, "q");
        const bool keys = a[1] != Py_None, batched = q.dim() == 4;
        const int64_t B = batched ? q.size(0) : 1, N = q.size(batched ? 2 : 0), d = q.size(-1);
        int64_t hk = 0;
        if (keys) {
            const Tensor& k = tensor(a[1], "k");
            check_rows(k, dev, "k");
            if (k.dim() != q.dim() || (batched && k.size(0) != B) || k.size(batched ? 2 : 0) != N || k.size(-1) != d)
                value_error("k must have q's tokens and d");
            hk = k.size(1);
        }
        const Tensor& pos = tensor(a[2], "positions");
        const int64_t lead = batched ? 2 : 1;
        if (pos.dim() != lead && pos.dim() != lead + 1)
            type_error(std::string("positions must be int32 ") + (batched ? "[B, N] or [axes, B, N]" : "[T] or [axes, T]"));
        const int64_t axes = pos.dim() == lead ? 1 : pos.size(0);
        if (batched && pos.dim() == 3) exact(a[2], {axes, B, N}, at::kInt, dev, "positions");
        else if (batched) exact(a[2], {B, N}, at::kInt, dev, "positions");
        else if (pos.dim() == 2) exact(a[2], {axes, N}, at::kInt, dev, "positions");
        else exact(a[2], {N}, at::kInt, dev, "positions");
        const Tensor& freq = tensor(a[3], "inv_freq");
        if (freq.dim() != 1) type_error("inv_freq must be a float32 [rot / 2] tensor");
        exact(a[3], {freq.numel()}, at::kFloat, dev, "inv_freq");
        const int* axis = nullptr;
        if (a[4] != Py_None)
            axis = static_cast<int*>(exact(a[4], {freq.numel()}, at::kInt, dev, "axis").data_ptr());
        const int interleaved = int_arg(a[5], "interleaved"), inverse = int_arg(a[6], "inverse");
        const On on(a[9], dev);
        auto out = [&](PyObject* given, const Tensor& like, const char* name) {
            if (given == Py_None) return on.empty(like.sizes(), at::kBFloat16, dev);
            const Tensor& t = tensor(given, name);
            check_rows(t, dev, name);
            if (!t.sizes().equals(like.sizes())) value_error(std::string(name) + " must have its input's shape");
            return t;
        };
        long long strides[12] = {};
        const Tensor qo = out(a[7], q, "q_out");
        row_strides(q, false, "q", strides);
        row_strides(qo, true, "q_out", strides + 3);
        Tensor ko;
        if (keys) {
            const Tensor& k = THPVariable_Unpack(a[1]);
            ko = out(a[8], k, "k_out");
            row_strides(k, false, "k", strides + 6);
            row_strides(ko, true, "k_out", strides + 9);
        }
        const attn_status_t st =
            f_rope(q.data_ptr(), keys ? ptr(a[1]) : nullptr, qo.data_ptr(), keys ? ko.data_ptr() : nullptr,
                   static_cast<int*>(pos.data_ptr()), static_cast<float*>(freq.data_ptr()), axis, strides,
                   size_arg(B, "B"), size_arg(N, "N"), size_arg(q.size(1), "Hq"), size_arg(hk, "Hk"), size_arg(d, "d"),
                   size_arg(2 * freq.numel(), "rot"), size_arg(axes, "axes"), interleaved, inverse, on.handle);
        if (st != ATTN_OK) return status(st);
        if (keys) return tuple_of({qo, ko});
        PyObject* first = THPVariable_Wrap(qo);
        if (!first) throw Refusal{nullptr, ""};
        PyObject* pair = PyTuple_Pack(2, first, Py_None);
        Py_DECREF(first);
        if (!pair) throw Refusal{nullptr, ""};
        return pair;
    });
}

// ------------------------------------------------------------------ differential attention

float scale_arg(PyObject* o, int64_t d)
{
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)(d > 0 ? d : 1)));
    const float scale = (float)PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw Refusal{nullptr, ""};
    return scale;
}

// Sizes of q [B, 2H, N, d], k [B, 2Hkv, N, d] and v [B, Hkv, N, 2d], or packed [T, 2H, d], [T, 2Hkv, d] and
// [T, Hkv, 2d] (B = 1, N = T); checked, as lam [H] is.
struct Diff {
    at::Device dev;
    bool packed;
    int64_t B, H, Hkv, N, d;

    at::DimVector shape(int64_t heads, int64_t width) const
    {
        return packed ? at::DimVector{N, heads, width} : at::DimVector{B, heads, N, width};
    }
    at::DimVector lse_shape() const { return packed ? at::DimVector{2 * H, N} : at::DimVector{B, 2 * H, N}; }
};

const Tensor& of_shape(PyObject* o, const at::DimVector& shape, at::ScalarType dtype, at::Device dev, const char* name)
{
    return shape.size() == 4   ? exact(o, {shape[0], shape[1], shape[2], shape[3]}, dtype, dev, name)
           : shape.size() == 3 ? exact(o, {shape[0], shape[1], shape[2]}, dtype, dev, name)
                               : exact(o, {shape[0], shape[1]}, dtype, dev, name);
}

Tensor output_of(const On& on, PyObject* o, const at::DimVector& shape, at::ScalarType dtype, at::Device dev,
                 const char* name)
{
    if (o != Py_None) return of_shape(o, shape, dtype, dev, name);
    return on.empty(shape, dtype, dev);
}

Diff diff_args(PyObject* const* a, bool packed)
{
    const Tensor& q = cuda_tensor(a[0], "q");
    const Tensor& k = tensor(a[1], "k");
    const Tensor& v = tensor(a[2], "v");
    const at::Device dev = q.device();
    const int64_t dims = packed ? 3 : 4;
    for (const Tensor* t : {&q, &k, &v})
        if (t->scalar_type() != at::kBFloat16 || t->device() != dev || t->dim() != dims || !t->is_contiguous())
            type_error(std::string("q, k and v must be contiguous bf16 ") + (packed ? "[T, heads, d]" : "[B, heads, N, d]") +
                       " tensors on " + dev.str());
    Diff s{dev, packed, packed ? 1 : q.size(0), q.size(1) / 2, v.size(1), q.size(packed ? 0 : 2), q.size(-1)};
    if (q.size(1) % 2 != 0 || s.H < 1 || s.Hkv < 1 || s.H % s.Hkv != 0)
        value_error("q must have 2 H heads, H a multiple of v's");
    of_shape(a[1], s.shape(2 * s.Hkv, s.d), at::kBFloat16, dev, "k");
    of_shape(a[2], s.shape(s.Hkv, 2 * s.d), at::kBFloat16, dev, "v");
    exact(a[3], {s.H}, at::kFloat, dev, "lam");
    return s;
}

// cu_seqlens [S + 1] of packed rows.
const Tensor& cu_arg(PyObject* o, at::Device dev)
{
    const Tensor& cu = tensor(o, "cu_seqlens");
    if (cu.dim() != 1 || cu.numel() < 2) type_error("cu_seqlens must be an int32 [S + 1] tensor");
    return exact(o, {cu.numel()}, at::kInt, dev, "cu_seqlens");
}

float* floats(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// q, k, v, lam, cu_seqlens or None, max_seqlen, scale or None, causal, window, save_o2, o, lse, o2, stream
PyObject* diff_fwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 14, [&]() -> PyObject* {
        const bool packed = a[4] != Py_None;
        const Diff s = diff_args(a, packed);
        const float scale = scale_arg(a[6], s.d);
        const int causal = int_arg(a[7], "causal"), window = int_arg(a[8], "window");
        const bool save = int_arg(a[9], "save_o2") != 0 || a[12] != Py_None;
        const Tensor* cu = packed ? &cu_arg(a[4], s.dev) : nullptr;
        const int longest = packed ? int_arg(a[5], "max_seqlen") : 0;
        const On on(a[13], s.dev);
        const Tensor o = output_of(on, a[10], s.shape(s.H, 2 * s.d), at::kBFloat16, s.dev, "o");
        const Tensor lse = output_of(on, a[11], s.lse_shape(), at::kFloat, s.dev, "lse");
        Tensor o2;
        if (save) o2 = output_of(on, a[12], s.shape(s.H, 2 * s.d), at::kBFloat16, s.dev, "o2");
        const int H = size_arg(s.H, "H"), hkv = size_arg(s.Hkv, "Hkv"), N = size_arg(s.N, "N"), d = size_arg(s.d, "d");
        void* second = save ? o2.data_ptr() : nullptr;
        const attn_status_t st =
            packed ? f_diff_fwd_varlen(ptr(a[0]), ptr(a[1]), ptr(a[2]), static_cast<float*>(ptr(a[3])), o.data_ptr(),
                                       floats(lse), second, static_cast<int*>(cu->data_ptr()),
                                       size_arg(cu->numel() - 1, "S"), longest, N, H, hkv, d, scale, causal, window,
                                       on.handle)
                   : f_diff_fwd(ptr(a[0]), ptr(a[1]), ptr(a[2]), static_cast<float*>(ptr(a[3])), o.data_ptr(),
                                floats(lse), second, size_arg(s.B, "B"), H, hkv, N, d, scale, causal, window, on.handle);
        if (st != ATTN_OK) return status(st);
        if (save) return tuple_of({o, lse, o2});
        PyObject* two = tuple_of({o, lse});
        PyObject* out = PyTuple_Pack(3, PyTuple_GET_ITEM(two, 0), PyTuple_GET_ITEM(two, 1), Py_None);
        Py_DECREF(two);
        if (!out) throw Refusal{nullptr, ""};
        return out;
    });
}

// A workspace of the caller's, or one that the stream's allocator lends for the call.
struct Workspace {
    c10::DataPtr lent;
    void* ptr;
    size_t bytes;

    Workspace(PyObject* given, size_t needed, at::Device dev)
    {
        if (given == Py_None) {
            bytes = needed;
            lent = c10::cuda::CUDACachingAllocator::get()->allocate(needed);
            ptr = lent.get();
            return;
        }
        const Tensor& t = tensor(given, "workspace");
        if (t.device() != dev || !t.is_contiguous()) type_error("workspace must be a contiguous CUDA tensor on " + dev.str());
        ptr = t.data_ptr();
        bytes = (size_t)t.nbytes();
    }
};

// q, k, v, lam, o, o2, dout, lse, cu_seqlens or None, max_seqlen, scale or None, causal, window, dq, dk, dv,
// dlam, workspace, stream
PyObject* diff_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 19, [&]() -> PyObject* {
        const bool packed = a[8] != Py_None;
        const Diff s = diff_args(a, packed);
        const at::DimVector out = s.shape(s.H, 2 * s.d);
        of_shape(a[4], out, at::kBFloat16, s.dev, "o");
        of_shape(a[5], out, at::kBFloat16, s.dev, "o2");
        of_shape(a[6], out, at::kBFloat16, s.dev, "dout");
        of_shape(a[7], s.lse_shape(), at::kFloat, s.dev, "lse");
        const Tensor* cu = packed ? &cu_arg(a[8], s.dev) : nullptr;
        const int longest = packed ? int_arg(a[9], "max_seqlen") : 0;
        const float scale = scale_arg(a[10], s.d);
        const int causal = int_arg(a[11], "causal"), window = int_arg(a[12], "window");
        const int B = size_arg(s.B, "B"), H = size_arg(s.H, "H"), hkv = size_arg(s.Hkv, "Hkv");
        const int N = size_arg(s.N, "N"), d = size_arg(s.d, "d");
        const On on(a[18], s.dev);
        const Tensor dq = output_of(on, a[13], s.shape(2 * s.H, s.d), at::kBFloat16, s.dev, "dq");
        const Tensor dk = output_of(on, a[14], s.shape(2 * s.Hkv, s.d), at::kBFloat16, s.dev, "dk");
        const Tensor dv = output_of(on, a[15], s.shape(s.Hkv, 2 * s.d), at::kBFloat16, s.dev, "dv");
        const Tensor dlam = on.output(a[16], {s.H}, at::kFloat, s.dev, "dlam");
        const Workspace ws(a[17], f_diff_bwd_ws(B, H, N), s.dev);
        auto bf = [&](int i) { return ptr(a[i]); };
        float *lam = static_cast<float*>(bf(3)), *lse = static_cast<float*>(bf(7));
        const attn_status_t st =
            packed ? f_diff_bwd_varlen(bf(0), bf(1), bf(2), lam, bf(4), bf(5), bf(6), lse, dq.data_ptr(), dk.data_ptr(),
                                       dv.data_ptr(), floats(dlam), ws.ptr, ws.bytes, static_cast<int*>(cu->data_ptr()),
                                       size_arg(cu->numel() - 1, "S"), longest, N, H, hkv, d, scale, causal, window,
                                       on.handle)
                   : f_diff_bwd(bf(0), bf(1), bf(2), lam, bf(4), bf(5), bf(6), lse, dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), floats(dlam), ws.ptr, ws.bytes, B, H, hkv, N, d, scale, causal, window,
                                on.handle);
        if (st != ATTN_OK) return status(st);
        return tuple_of({dq, dk, dv, dlam});
    });
}

// q, k_cache, v_cache, lam, page_table, seq_lens, scale or None, window, workspace, o, lse, stream
PyObject* diff_decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 12, [&]() -> PyObject* {
        const Tensor& q = cuda_tensor(a[0], "q");
        const at::Device dev = q.device();
        if (q.scalar_type() != at::kBFloat16) type_error("q must be bf16");
        if (q.dim() != 4 || !q.is_contiguous()) value_error("q must be a contiguous [B, 2H, nq, d] tensor");
        const int64_t B = q.size(0), H = q.size(1) / 2, nq = q.size(2), d = q.size(3);
        const Tensor& kc = tensor(a[1], "k_cache");
        const Tensor& vc = tensor(a[2], "v_cache");
        check_cache(kc, dev, false, "k_cache");
        check_cache(vc, dev, false, "v_cache");
        if (!vc.sizes().equals(kc.sizes()) || kc.size(3) != d || kc.size(1) % 2 != 0 || q.size(1) % 2 != 0)
            value_error("q must be [B, 2H, nq, d] and the caches [num_pages, 2Hkv, page_size, d]");
        exact(a[3], {H}, at::kFloat, dev, "lam");
        const Tensor& table = tensor(a[4], "page_table");
        if (table.dim() != 2) type_error("page_table must be an int32 [B, max_pages] tensor");
        exact(a[4], {B, table.size(1)}, at::kInt, dev, "page_table");
        exact(a[5], {B}, at::kInt, dev, "seq_lens");
        const float scale = scale_arg(a[6], d);
        const int window = int_arg(a[7], "window");
        const int h = size_arg(H, "H"), hkv = size_arg(kc.size(1) / 2, "Hkv"), nqi = size_arg(nq, "nq"), di = size_arg(d, "d");
        const On on(a[11], dev);
        const Workspace ws(a[8], a[8] == Py_None ? f_diff_decode_ws(h, hkv, nqi, di) : 0, dev);
        const Tensor o = on.output(a[9], {B, H, nq, 2 * d}, at::kBFloat16, dev, "o");
        const Tensor lse = on.output(a[10], {B, 2 * H, nq}, at::kFloat, dev, "lse");
        const attn_status_t st = f_diff_decode(
            q.data_ptr(), kc.data_ptr(), vc.data_ptr(), static_cast<float*>(ptr(a[3])), static_cast<int*>(ptr(a[4])),
            static_cast<int*>(ptr(a[5])), o.data_ptr(), floats(lse), size_arg(B, "B"), h, hkv, nqi, di,
            size_arg(kc.size(2), "page_size"), size_arg(kc.size(0), "num_pages"), size_arg(table.size(1), "max_pages"),
            scale, window, ws.ptr, ws.bytes, on.handle);
        if (st != ATTN_OK) return status(st);
        return tuple_of({o, lse});
    });
}

// The addresses of the C functions, in the order below.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    constexpr int kCount = 13;
    return guarded(n, kCount, [&]() -> PyObject* {
        void* f[kCount];
        for (int i = 0; i < kCount; ++i) {
            f[i] = PyLong_AsVoidPtr(a[i]);
            if (PyErr_Occurred()) throw Refusal{nullptr, ""};
        }
        f_plan = reinterpret_cast<decltype(f_plan)>(f[0]);
        f_append_bf16 = reinterpret_cast<decltype(f_append_bf16)>(f[1]);
        f_append_fp8 = reinterpret_cast<decltype(f_append_fp8)>(f[2]);
        f_decode = reinterpret_cast<decltype(f_decode)>(f[3]);
        f_decode_ws = reinterpret_cast<decltype(f_decode_ws)>(f[4]);
        f_rope = reinterpret_cast<decltype(f_rope)>(f[5]);
        f_diff_fwd = reinterpret_cast<decltype(f_diff_fwd)>(f[6]);
        f_diff_fwd_varlen = reinterpret_cast<decltype(f_diff_fwd_varlen)>(f[7]);
        f_diff_bwd = reinterpret_cast<decltype(f_diff_bwd)>(f[8]);
        f_diff_bwd_varlen = reinterpret_cast<decltype(f_diff_bwd_varlen)>(f[9]);
        f_diff_bwd_ws = reinterpret_cast<decltype(f_diff_bwd_ws)>(f[10]);
        f_diff_decode = reinterpret_cast<decltype(f_diff_decode)>(f[11]);
        f_diff_decode_ws = reinterpret_cast<decltype(f_diff_decode_ws)>(f[12]);
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
                         method<decode>("decode"),       method<rope>("rope"),
                         method<diff_fwd>("diff_fwd"),   method<diff_bwd>("diff_bwd"),
                         method<diff_decode>("diff_decode"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gb300attn_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gb300attn_binding() { return PyModule_Create(&module); }
