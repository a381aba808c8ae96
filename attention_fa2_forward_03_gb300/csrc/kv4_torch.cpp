// Torch tensors to the C entry points of the 4-bit KV cache (marshalling only).
//
// These calls run once a layer and decoding step, where a step takes a few
// microseconds on the GPU: checking the arguments and allocating the outputs
// in Python took 13 us of an 18 us call. The functions take positional
// arguments; fa2.py gives them names and defaults. They return the outputs, or
// the status of the C call as an int where that is not FA2_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <stdexcept>
#include <string>

#include "fa2.h"

namespace {

using at::Tensor;

// The library's entry points, from the binding that loaded it.
decltype(&fa2_kv4_plan) g_plan;
decltype(&fa2_kv4_append) g_append;
decltype(&fa2_kv4_gather) g_gather;
decltype(&fa2_fwd_kv4) g_fwd;
decltype(&fa2_fwd_kv4_workspace) g_workspace;
PyObject* g_out_of_memory;   // torch.OutOfMemoryError

struct TypeError : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};   // a Python exception is set

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

std::string shape_of(const Tensor& t) {
    std::string s = c10::toString(t.scalar_type()) + std::string(" [");
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] on " + t.device().str();
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeError(std::string(name) + " must be a torch tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    return x;
}

int int32(int64_t x, const char* name) {
    if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
    return static_cast<int>(x);
}

// A contiguous CUDA tensor on `index` of this type; `n` elements unless < 0.
void want(const Tensor& t, const char* name, c10::DeviceIndex index, at::ScalarType type, const char* shape, bool fits) {
    if (!t.is_cuda() || t.get_device() != index)
        refuse(std::string("all tensors must be on one CUDA device, ") + name + " is on " + t.device().str());
    if (t.scalar_type() != type || !fits || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor " + shape + ", got " + shape_of(t));
}

bool is(const Tensor& t, at::IntArrayRef shape) { return t.sizes() == shape; }

fa2_dtype dtype_code(at::ScalarType t) {
    if (t == at::kBFloat16) return FA2_BF16;
    if (t == at::kHalf) return FA2_FP16;
    throw TypeError(std::string("q, k and v must be bf16 or fp16, got ") + c10::toString(t));
}

c10::DeviceIndex device_of(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor, got one on " + t.device().str());
    return t.device().index();
}

// The device and stream of a call: the device's current stream for None, else
// a torch.cuda.Stream or a handle. Both are current while this lives, so what
// is allocated belongs to the stream that writes it.
struct On {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard guard;
    cudaStream_t stream;
    On(PyObject* o, c10::DeviceIndex index) : device(index) {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(index).stream();
            return;
        }
        PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw Raised{};
        void* p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw Raised{};
        stream = static_cast<cudaStream_t>(p);
        // 0, 1 and 2 are CUDA's names for its default streams, not addresses
        guard.reset_stream(reinterpret_cast<uintptr_t>(p) > 2 ? c10::cuda::getStreamFromExternal(stream, index)
                                                              : c10::cuda::getDefaultCUDAStream(index));
    }
};

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex index) {
    return Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, index), std::nullopt));
}

template <typename T>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

// num_pages and page_size of a cache [num_pages, H_kv, 2, page_size * (d/2 + d/16)].
struct Cache {
    int pages, heads, page_size;
    Cache(const Tensor& c, const Tensor& kd, const Tensor& vd, c10::DeviceIndex index, int64_t heads_wanted, int64_t d) {
        const int64_t token = d / 2 + d / 16;
        want(c, "cache", index, at::kByte, "[num_pages, H_kv, 2, page_size*(d/2+d/16)]",
             c.dim() == 4 && (heads_wanted < 0 || c.size(1) == heads_wanted) && c.size(2) == 2 && token > 0 && c.size(3) % token == 0);
        want(kd, "k_descale", index, at::kFloat, "of H_kv elements", kd.numel() == c.size(1));
        want(vd, "v_descale", index, at::kFloat, "of H_kv elements", vd.numel() == c.size(1));
        pages = int32(c.size(0), "num_pages");
        heads = int32(c.size(1), "H_kv");
        page_size = int32(c.size(3) / token, "page_size");
    }
};

PyObject* give(std::initializer_list<const Tensor*> ts) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!out) throw Raised{};
    Py_ssize_t i = 0;
    for (const Tensor* t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(*t));
    return out;
}

// Runs one function with its exceptions turned into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t wanted, F&& f) {
    if (got != wanted) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, got);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised&) {
    } catch (const TypeError& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_out_of_memory ? g_out_of_memory : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// seq_lens, new_lens, block_table, free_pages, free_state, page_size, N,
// seq_lens_out, accepted, slots, free_state_out, stream
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Tensor &lens = tensor(a[0], "seq_lens"), &add = tensor(a[1], "new_lens"), &table = tensor(a[2], "block_table"),
                     &ring = tensor(a[3], "free_pages"), &state = tensor(a[4], "free_state");
        const int page = int32(integer(a[5]), "page_size"), N = int32(integer(a[6]), "N");
        if (lens.dim() != 1 || table.dim() != 2 || ring.dim() != 1)
            refuse("seq_lens must be [B], block_table [B, max_pages], free_pages [num_pages]");
        const c10::DeviceIndex index = device_of(lens, "seq_lens");
        const int64_t B = table.size(0);
        const auto i32 = at::kInt;
        const On on(a[11], index);
        want(lens, "seq_lens", index, i32, "[B]", is(lens, {B}));
        want(add, "new_lens", index, i32, "[B]", is(add, {B}));
        want(table, "block_table", index, i32, "[B, max_pages]", true);
        want(ring, "free_pages", index, i32, "[num_pages]", true);
        want(state, "free_state", index, i32, "[2]", is(state, {2}));
        auto out = [&](PyObject* o, const char* name, const char* says, at::IntArrayRef shape) {
            if (o == Py_None) return fresh(shape, i32, index);
            const Tensor& t = tensor(o, name);
            want(t, name, index, i32, says, is(t, shape));
            return t;
        };
        const Tensor lens_out = out(a[7], "seq_lens_out", "[B]", {B}), accepted = out(a[8], "accepted", "[B]", {B}),
                     slots = out(a[9], "slots", "[B, N]", {B, std::max(N, 0)}),
                     state_out = out(a[10], "free_state_out", "[2]", {2});
        const fa2_status rc = g_plan(ptr<int32_t>(lens), ptr<int32_t>(add), ptr<int32_t>(table), ptr<int32_t>(ring),
                                     ptr<int32_t>(state), ptr<int32_t>(lens_out), ptr<int32_t>(accepted),
                                     ptr<int32_t>(slots), ptr<int32_t>(state_out), int32(B, "B"), N,
                                     int32(table.size(1), "max_pages"), page, int32(ring.size(0), "num_pages"), on.stream);
        if (rc != FA2_OK) return PyLong_FromLong(rc);
        return give({&lens_out, &accepted, &slots, &state_out});
    });
}

// k, v, slots, cache, k_descale, v_descale, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                     &cache = tensor(a[3], "cache"), &kd = tensor(a[4], "k_descale"), &vd = tensor(a[5], "v_descale");
        if (k.dim() != 4 || k.sizes() != v.sizes()) refuse("k and v must be 4-D [B, H_kv, N, d] of one shape");
        if (k.scalar_type() != v.scalar_type()) throw TypeError("k and v must share one dtype");
        const c10::DeviceIndex index = device_of(k, "k");
        if (device_of(v, "v") != index) refuse("k and v must be on one device");
        if (k.stride(3) != 1 || v.stride(3) != 1) refuse("the rows of k and v must be adjacent elements");
        const int64_t B = k.size(0), H = k.size(1), N = k.size(2), d = k.size(3);
        const Cache c(cache, kd, vd, index, H, d);
        want(slots, "slots", index, at::kInt, "[B, N]", is(slots, {B, N}));
        const On on(a[6], index);
        // the stride of an axis of length 1 is never used and may be anything
        auto st = [](const Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; };
        const fa2_status rc = g_append(k.data_ptr(), v.data_ptr(), ptr<int32_t>(slots), cache.data_ptr(), ptr<float>(kd),
                                       ptr<float>(vd), int32(B, "B"), c.heads, int32(N, "N"), int32(d, "d"), st(k, 0),
                                       st(k, 1), st(k, 2), st(v, 0), st(v, 1), st(v, 2), c.page_size, c.pages,
                                       dtype_code(k.scalar_type()), on.stream);
        if (rc != FA2_OK) return PyLong_FromLong(rc);
        return Py_NewRef(a[3]);
    });
}

// cache, block_table, seq_lens, k_descale, v_descale, N, d, starts, dtype, k, v, stream
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Tensor &cache = tensor(a[0], "cache"), &table = tensor(a[1], "block_table"), &lens = tensor(a[2], "seq_lens"),
                     &kd = tensor(a[3], "k_descale"), &vd = tensor(a[4], "v_descale");
        const int N = int32(integer(a[5]), "N"), d = int32(integer(a[6]), "d");
        if (table.dim() != 2 || cache.dim() != 4 || N < 0 || d < 0)
            refuse("block_table must be [B, max_pages], cache [num_pages, H_kv, 2, page_size*(d/2+d/16)], N and d >= 0");
        const c10::DeviceIndex index = device_of(cache, "cache");
        const int64_t B = table.size(0);
        const Cache c(cache, kd, vd, index, -1, d);
        want(table, "block_table", index, at::kInt, "[B, max_pages]", true);
        want(lens, "seq_lens", index, at::kInt, "[B]", is(lens, {B}));
        const int32_t* starts = nullptr;
        if (a[7] != Py_None) {
            const Tensor& s = tensor(a[7], "starts");
            want(s, "starts", index, at::kInt, "[B]", is(s, {B}));
            starts = ptr<int32_t>(s);
        }
        at::ScalarType type = a[9] == Py_None ? at::kBFloat16 : tensor(a[9], "k").scalar_type();
        if (a[8] != Py_None) {
            if (!THPDtype_Check(a[8])) throw TypeError("dtype must be a torch dtype");
            type = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
        }
        const fa2_dtype code = dtype_code(type);
        const On on(a[11], index);
        auto out = [&](PyObject* o, const char* name) {
            const std::array<int64_t, 4> shape = {B, c.heads, N, d};
            if (o == Py_None) return fresh(shape, type, index);
            const Tensor& t = tensor(o, name);
            want(t, name, index, type, "[B, H_kv, N, d]", is(t, shape));
            return t;
        };
        const Tensor k = out(a[9], "k"), v = out(a[10], "v");
        const fa2_status rc = g_gather(cache.data_ptr(), ptr<int32_t>(table), ptr<int32_t>(lens), starts, ptr<float>(kd),
                                       ptr<float>(vd), k.data_ptr(), v.data_ptr(), int32(B, "B"), c.heads, N, d,
                                       int32(table.size(1), "max_pages"), c.page_size, c.pages, code, on.stream);
        if (rc != FA2_OK) return PyLong_FromLong(rc);
        return give({&k, &v});
    });
}

// q, cache, block_table, seq_lens, k_descale, v_descale, o, lse, workspace, scale, causal, stream
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "cache"), &table = tensor(a[2], "block_table"),
                     &lens = tensor(a[3], "seq_lens"), &kd = tensor(a[4], "k_descale"), &vd = tensor(a[5], "v_descale");
        if (q.dim() != 4 || cache.dim() != 4 || table.dim() != 2)
            refuse("q must be [B, H_q, N_q, d], cache 4-D and block_table [B, max_pages]");
        const c10::DeviceIndex index = device_of(q, "q");
        const fa2_dtype code = dtype_code(q.scalar_type());
        const int64_t B = q.size(0), H = q.size(1), N = q.size(2), d = q.size(3);
        want(q, "q", index, q.scalar_type(), "[B, H_q, N_q, d]", true);
        const Cache c(cache, kd, vd, index, -1, d);
        want(table, "block_table", index, at::kInt, "[B, max_pages]", table.size(0) == B);
        want(lens, "seq_lens", index, at::kInt, "[B]", is(lens, {B}));
        const On on(a[11], index);
        Tensor o, lse, ws;
        if (a[6] == Py_None) {
            o = fresh(q.sizes(), q.scalar_type(), index);
        } else {
            o = tensor(a[6], "o");
            want(o, "o", index, q.scalar_type(), "like q", is(o, q.sizes()));
        }
        if (a[7] == Py_None) {
            lse = fresh({B, H, N}, at::kFloat, index);
        } else {
            lse = tensor(a[7], "lse");
            want(lse, "lse", index, at::kFloat, "[B, H_q, N_q]", is(lse, {B, H, N}));
        }
        double scale = 1.0 / std::sqrt(static_cast<double>(d));
        if (a[9] != Py_None) {
            scale = PyFloat_AsDouble(a[9]);
            if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
        }
        const int causal = PyObject_IsTrue(a[10]);
        if (causal < 0) throw Raised{};
        const int b = int32(B, "B"), hq = int32(H, "H_q"), nq = int32(N, "N_q"), dd = int32(d, "d"),
                  pages = int32(table.size(1), "max_pages");
        int64_t bytes = 0;
        if (a[8] != Py_None) {
            ws = tensor(a[8], "workspace");
            if (!ws.is_cuda() || ws.get_device() != index || !ws.is_contiguous())
                refuse("workspace must be a contiguous tensor on q's device");
            bytes = static_cast<int64_t>(ws.nbytes());
        } else if ((bytes = g_workspace(b, hq, c.heads, nq, dd, pages, c.page_size)) > 0) {
            ws = fresh({bytes}, at::kByte, index);   // given back to `on`'s stream behind the call
        }
        const fa2_status rc = g_fwd(q.data_ptr(), cache.data_ptr(), ptr<int32_t>(table), ptr<int32_t>(lens), ptr<float>(kd),
                                    ptr<float>(vd), o.data_ptr(), ptr<float>(lse), ws.defined() ? ws.data_ptr() : nullptr,
                                    bytes, b, hq, c.heads, nq, dd, pages, c.page_size, c.pages,
                                    static_cast<float>(scale), causal, code, on.stream);
        if (rc != FA2_OK) return PyLong_FromLong(rc);
        return give({&o, &lse});
    });
}

// Addresses of the C entry points (plan, append, gather, forward, workspace)
// and torch.OutOfMemoryError.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        void* p[5];
        for (int i = 0; i < 5; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (!p[i]) throw Raised{};
        }
        g_plan = reinterpret_cast<decltype(g_plan)>(p[0]);
        g_append = reinterpret_cast<decltype(g_append)>(p[1]);
        g_gather = reinterpret_cast<decltype(g_gather)>(p[2]);
        g_fwd = reinterpret_cast<decltype(g_fwd)>(p[3]);
        g_workspace = reinterpret_cast<decltype(g_workspace)>(p[4]);
        g_out_of_memory = Py_NewRef(a[5]);
        return Py_NewRef(Py_None);
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(plan), FAST(append), FAST(gather), FAST(fwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4_torch(void) { return PyModule_Create(&module); }
