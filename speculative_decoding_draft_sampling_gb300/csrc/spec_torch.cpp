// spec_torch.cpp -- the cache calls' Python binding: checks tensors, allocates
// outputs with PyTorch and calls the C ABI on the current stream.
//
// The cache calls are made several times a layer and step, and a Python binding
// of one costs more than most of them take on the device (one step's rows
// appended and read back: 26 us of Python and ctypes, 9 us of kernels), so this
// one is C++ against PyTorch's own tensor class.  It computes nothing.
#include <Python.h>

#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstring>
#include <initializer_list>
#include <map>
#include <optional>
#include <string>
#include <utility>

#include "../../include/spec_cache.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;        // SpecError
PyObject* g_attention = nullptr;    // CacheAttention

struct Api {
    decltype(&spec_last_error) last_error;
    decltype(&spec_cache_append) append;
    decltype(&spec_cache_read) read;
    decltype(&spec_cache_attend_workspace_size) attend_ws;
    decltype(&spec_cache_attend) attend;
    decltype(&spec_cache_compact) compact;
    decltype(&spec_cache_reserve) reserve;
    decltype(&spec_cache_release) release;
    decltype(&spec_cache_fork) fork;
} g_api = {};

// a Python exception is set; unwinds to the entry point
struct Raised {};

[[noreturn]] void refuse(const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, buf);
    throw Raised{};
}

void done(spec_status rc, const char* who) {
    if (rc != SPEC_OK) refuse("%s failed (status %d): %s", who, static_cast<int>(rc), g_api.last_error());
}

// CUDA tensors lie where the call works (host tensors are checked for being pinned).
void on_device(PyObject* o, const char* name, c10::Device device) {
    if (!o || !THPVariable_Check(o)) return;
    const Tensor& t = THPVariable_Unpack(o);
    if (t.is_cuda() && t.device() != device)
        refuse("%s is on %s, the call works on %s", name, t.device().str().c_str(), device.str().c_str());
}

// Arguments of a call: positional ones, then keywords, in the order of `names`.
struct Args {
    PyObject* v[16] = {};
    const char* const* const names;
    const int count;

    Args(const char* who, const char* const* names_, int count_, int required, int positional, PyObject* const* args,
         Py_ssize_t nargs, PyObject* kwnames)
        : names(names_), count(count_) {
        if (nargs > positional) {
            PyErr_Format(PyExc_TypeError, "%s() takes at most %d positional arguments (%zd given)", who, positional, nargs);
            throw Raised{};
        }
        for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
        const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < nk; ++k) {
            PyObject* name = PyTuple_GET_ITEM(kwnames, k);
            int at = -1;
            for (int i = 0; i < count; ++i)
                if (PyUnicode_CompareWithASCIIString(name, names[i]) == 0) { at = i; break; }
            if (at < 0 || v[at]) {
                PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", who,
                             at < 0 ? "an unexpected keyword" : "multiple values for", name);
                throw Raised{};
            }
            v[at] = args[nargs + k];
        }
        for (int i = 0; i < count; ++i) {
            if (v[i] == Py_None) v[i] = nullptr;
            if (i < required && !v[i]) {
                PyErr_Format(PyExc_TypeError, "%s() needs the argument '%s'", who, names[i]);
                throw Raised{};
            }
        }
    }
    void all_on(c10::Device device) const {
        for (int i = 0; i < count; ++i) on_device(v[i], names[i], device);
    }
    long long integer(int i, long long fallback) const {
        if (!v[i]) return fallback;
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred()) throw Raised{};
        return x;
    }
    int int32(int i, long long fallback, const char* name) const {
        const long long x = integer(i, fallback);
        if (x < INT32_MIN || x > INT32_MAX) refuse("%s is out of range", name);
        return static_cast<int>(x);
    }
};

int checked(int64_t x, const char* name) {
    if (x > INT32_MAX) refuse("%s is out of range", name);
    return static_cast<int>(x);
}

// A CUDA tensor, or a pinned host tensor that the kernels read (or write) in
// place through its device mapping.
const Tensor& reachable(PyObject* o, const char* name, at::ScalarType type, const char* type_name) {
    if (!o || !THPVariable_Check(o)) refuse("%s must be a CUDA tensor or a pinned host tensor", name);
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() && !(t.device().is_cpu() && t.is_pinned()))
        refuse("%s must be a CUDA tensor or a pinned host tensor", name);
    if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, type_name, c10::toString(t.scalar_type()));
    return t;
}

const Tensor& shaped(PyObject* o, const char* name, at::ScalarType type, const char* type_name,
                     std::initializer_list<int64_t> shape) {
    const Tensor& t = reachable(o, name, type, type_name);
    if (t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) {
        std::string s;
        for (int64_t x : shape) s += (s.empty() ? "" : ", ") + std::to_string(x);
        refuse("%s must be a contiguous [%s] %s tensor", name, s.c_str(), type_name);
    }
    return t;
}

int32_t* ints(PyObject* o, const char* name, std::initializer_list<int64_t> shape) {
    return static_cast<int32_t*>(shaped(o, name, at::kInt, "int32", shape).data_ptr());
}
int32_t* ints_or_null(PyObject* o, const char* name, std::initializer_list<int64_t> shape) {
    return o ? ints(o, name, shape) : nullptr;
}

struct Pool {
    void* data;
    int64_t layer_stride, page_stride, head_stride;
    int layers, pages, heads, page;
    c10::Device device{c10::kCUDA, 0};

    Pool(PyObject* o, int dims, int64_t head_dim) {
        const char* form = dims == 3 ? "[pages, kv_heads, block]" : "[layers, pages, kv_heads, block]";
        if (!o || !THPVariable_Check(o)) refuse("pool must be a uint8 CUDA tensor %s with unit element stride", form);
        const Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.scalar_type() != at::kByte || t.dim() != dims || t.stride(-1) != 1)
            refuse("pool must be a uint8 CUDA tensor %s with unit element stride", form);
        const int64_t block = t.size(-1);
        const int64_t p = head_dim > 0 ? block * 8 / (9 * head_dim) : 0;
        if ((p != 16 && p != 32 && p != 64) || p * head_dim * 9 != block * 8)
            refuse("a block of %lld bytes is no page of head_dim %lld", static_cast<long long>(block),
                   static_cast<long long>(head_dim));
        page = static_cast<int>(p);
        heads = checked(t.size(-2), "kv_heads");
        pages = checked(t.size(-3), "pages");
        head_stride = t.stride(-2);
        page_stride = t.stride(-3);
        layers = dims == 4 ? checked(t.size(0), "layers") : 1;
        layer_stride = dims == 4 ? t.stride(0) : 0;
        data = t.data_ptr();
        device = t.device();
    }
};

struct Table {
    int32_t* data;
    int64_t rows, stride;
    int width;

    Table(PyObject* o, int64_t B) {
        const Tensor& t = reachable(o, "page_table", at::kInt, "int32");
        if (t.dim() != 2 || t.stride(1) != 1 || (B >= 0 && t.size(0) != B))
            refuse("page_table must be [B, M] int32 with unit element stride");
        data = static_cast<int32_t*>(t.data_ptr());
        rows = t.size(0);
        width = checked(t.size(1), "page_table's width");
        stride = rows > 1 ? t.stride(0) : std::max<int64_t>(t.stride(0), width);
    }
};

// The stream that a call runs on: the one given, else the device's current one.  It is
// the current one while the call lasts, so that what the call allocates belongs to it.
class Stream {
    const c10::cuda::OptionalCUDAGuard device_;
    std::optional<c10::cuda::CUDAStreamGuard> on_;
    void* raw_;

  public:
    Stream(PyObject* o, c10::Device device) : device_(device) {
        if (!o) {
            raw_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
            return;
        }
        PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw Raised{};
        raw_ = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!raw_ && PyErr_Occurred()) throw Raised{};
        on_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw_), device.index()));
    }
    operator void*() const { return raw_; }
};

// A call's body, with C++ exceptions turned into Python's.
template <class F>
PyObject* entry(F body) {
    HANDLE_TH_ERRORS
    try {
        return body();
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"k", "v", "pool", "page_table", "start", "count", "status", "stream"};
        const Args a("cache_append", names, 8, 5, 6, args, nargs, kw);
        const Tensor& k = reachable(a.v[0], "k", at::kBFloat16, "bfloat16");
        const Tensor& v = reachable(a.v[1], "v", at::kBFloat16, "bfloat16");
        if (k.dim() != 4 || v.sizes() != k.sizes() || k.stride(3) != 1 || v.stride(3) != 1)
            refuse("k and v must be [B, n, kv_heads, D] with unit element stride");
        const int B = checked(k.size(0), "B"), n = checked(k.size(1), "n"), D = checked(k.size(3), "D");
        const Pool pool(a.v[2], 3, D);
        a.all_on(pool.device);
        if (pool.heads != k.size(2))
            refuse("the pool has %d kv heads, k and v %lld", pool.heads, static_cast<long long>(k.size(2)));
        const Table t(a.v[3], B);
        const int32_t* start = ints(a.v[4], "start", {B});
        const int32_t* count = ints_or_null(a.v[5], "count", {B});
        int32_t* status = ints_or_null(a.v[6], "status", {B});
        const Stream stream(a.v[7], pool.device);
        done(g_api.append(k.data_ptr(), k.stride(0), k.stride(1), k.stride(2), v.data_ptr(), v.stride(0), v.stride(1),
                          v.stride(2), pool.data, pool.page_stride, pool.head_stride, pool.pages, t.data, t.stride,
                          t.width, start, count, B, n, pool.heads, D, pool.page, status, stream),
             "spec_cache_append");
        Py_RETURN_NONE;
    });
}

PyObject* cache_read(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"pool", "page_table", "start", "n", "head_dim", "count", "k", "v", "status", "stream"};
        const Args a("cache_read", names, 10, 5, 6, args, nargs, kw);
        const int n = a.int32(3, 0, "n"), D = a.int32(4, 0, "head_dim");
        const Pool pool(a.v[0], 3, D);
        a.all_on(pool.device);
        const Table t(a.v[1], -1);
        const int B = checked(t.rows, "B");
        if (n < 0) refuse("n must not be negative");
        const int32_t* start = ints(a.v[2], "start", {B});
        const int32_t* count = ints_or_null(a.v[5], "count", {B});
        int32_t* status = ints_or_null(a.v[8], "status", {B});
        const Stream stream(a.v[9], pool.device);
        Tensor out[2];
        for (int i = 0; i < 2; ++i) {
            if (a.v[6 + i])
                out[i] = shaped(a.v[6 + i], names[6 + i], at::kBFloat16, "bfloat16", {B, n, pool.heads, D});
            else
                out[i] = at::empty({B, n, pool.heads, D}, at::TensorOptions(pool.device).dtype(at::kBFloat16));
        }
        done(g_api.read(pool.data, pool.page_stride, pool.head_stride, pool.pages, t.data, t.stride, t.width, start,
                        count, B, n, pool.heads, D, pool.page, out[0].data_ptr(), out[1].data_ptr(), status,
                        stream),
             "spec_cache_read");
        return Py_BuildValue("(NN)", THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
    });
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// cache_attend's workspaces: their control words start at zero and every call
// leaves them so.  Calls on a stream share one, which is replaced when a call needs
// more (its memory is freed in the stream's order).  A capture cannot have that one:
// a graph keeps the address, and may be replayed beside other calls or graphs.  It
// gets its own on each stream, zeroed by the graph, that lives until the graph and
// all that was instantiated from it are gone.
struct Held {
    Tensor ws;
    Held* next;
};
std::atomic<Held*> g_gone{nullptr};             // what the graphs that are gone held

// (called by the CUDA runtime: no CUDA call is allowed here, and freeing may be one)
void CUDART_CB graph_gone(void* p) {
    Held* h = static_cast<Held*>(p);
    h->next = g_gone.load(std::memory_order_relaxed);
    while (!g_gone.compare_exchange_weak(h->next, h, std::memory_order_release, std::memory_order_relaxed)) {}
}

void free_gone() {
    if (!g_gone.load(std::memory_order_relaxed)) return;
    for (Held* h = g_gone.exchange(nullptr, std::memory_order_acquire); h;) {
        Held* next = h->next;
        delete h;
        h = next;
    }
}

void runtime(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return;
    cudaGetLastError();
    refuse("cache_attend: %s: %s", what, cudaGetErrorString(e));
}

// (the stream is the current one)
Tensor attend_workspace(size_t bytes, c10::Device device, void* stream) {
    struct Captured {
        unsigned long long id;
        Tensor ws;
    };
    using Key = std::pair<int, void*>;
    static auto* eager = new std::map<Key, Tensor>;             // (both outlive the interpreter's end)
    static auto* captured = new std::map<Key, Captured>;
    const auto st = static_cast<cudaStream_t>(stream);
    const Key key{device.index(), stream};
    const auto is_enough = [&](const Tensor& t) { return t.defined() && static_cast<size_t>(t.numel()) >= bytes; };
    free_gone();

    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    cudaGraph_t graph = nullptr;
    const cudaGraphNode_t* nodes = nullptr;
    const cudaGraphEdgeData* edges = nullptr;
    size_t count = 0;
    runtime(cudaStreamGetCaptureInfo(st, &status, &id, &graph, &nodes, &edges, &count), "the stream's capture");
    const bool capturing = status == cudaStreamCaptureStatusActive;
    Captured* mine = capturing ? &(*captured)[key] : nullptr;
    Tensor& kept = capturing ? mine->ws : (*eager)[key];
    if (is_enough(kept) && (!capturing || mine->id == id)) return kept;

    const Tensor fresh = at::empty({static_cast<int64_t>(bytes)}, at::TensorOptions(device).dtype(at::kByte));
    fresh.narrow(0, 0, SPEC_CACHE_WS_CONTROL).zero_();
    if (capturing) {
        auto* h = new Held{fresh, nullptr};
        cudaUserObject_t object;
        const cudaError_t made = cudaUserObjectCreate(&object, h, graph_gone, 1, cudaUserObjectNoDestructorSync);
        if (made != cudaSuccess) delete h;
        runtime(made, "the graph's workspace");
        const cudaError_t kept_by = cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove);
        if (kept_by != cudaSuccess) cudaUserObjectRelease(object, 1);
        runtime(kept_by, "the graph's workspace");
        mine->id = id;
    }
    kept = fresh;
    return fresh;
}

PyObject* cache_attend(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"q", "pool", "page_table", "ctx_len", "num_rows", "anc_mask", "depth", "window",
                                            "sinks", "scale", "out", "lse", "want_lse", "status", "ws", "stream"};
        const Args a("cache_attend", names, 16, 4, 5, args, nargs, kw);
        const Tensor& q = reachable(a.v[0], "q", at::kBFloat16, "bfloat16");
        if (q.dim() != 4 || q.stride(3) != 1) refuse("q must be [B, n, q_heads, D] with unit element stride");
        const int B = checked(q.size(0), "B"), n = checked(q.size(1), "n"), hq = checked(q.size(2), "q_heads"),
                  D = checked(q.size(3), "D");
        const Pool pool(a.v[1], 3, D);
        a.all_on(pool.device);
        const Table t(a.v[2], B);
        const int32_t* ctx = ints(a.v[3], "ctx_len", {B});
        const int32_t* rows = ints_or_null(a.v[4], "num_rows", {B});
        const void* mask = a.v[5] ? shaped(a.v[5], "anc_mask", at::kLong, "int64", {B, n, (n + 63) / 64}).data_ptr() : nullptr;
        const int32_t* depth = ints_or_null(a.v[6], "depth", {B, n});
        const int window = a.int32(7, 0, "window"), sinks = a.int32(8, 0, "sinks");
        float scale = D > 0 ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : 1.0f;
        if (a.v[9]) {
            const double x = PyFloat_AsDouble(a.v[9]);
            if (x == -1.0 && PyErr_Occurred()) throw Raised{};
            scale = static_cast<float>(x);
        }
        int32_t* status = ints_or_null(a.v[13], "status", {B});
        const Stream stream(a.v[15], pool.device);
        Tensor out = a.v[10] ? shaped(a.v[10], "out", at::kBFloat16, "bfloat16", {B, n, hq, D})
                             : at::empty({B, n, hq, D}, at::TensorOptions(pool.device).dtype(at::kBFloat16));
        Tensor lse;
        if (a.v[11]) lse = shaped(a.v[11], "lse", at::kFloat, "float32", {B, n, hq});
        else if (a.v[12] && PyObject_IsTrue(a.v[12]) > 0)
            lse = at::empty({B, n, hq}, at::TensorOptions(pool.device).dtype(at::kFloat));
        Tensor ws;
        if (a.v[14]) {
            ws = reachable(a.v[14], "ws", at::kByte, "uint8");
            if (!ws.is_contiguous()) refuse("ws must be contiguous");
        } else if (const size_t need = g_api.attend_ws(B, n, hq, pool.heads, D)) {
            ws = attend_workspace(need, pool.device, stream);
        }
        done(g_api.attend(q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), pool.data, pool.page_stride,
                          pool.head_stride, pool.pages, t.data, t.stride, t.width, ctx, rows,
                          static_cast<const uint64_t*>(mask), depth, window, sinks, scale, B, n, hq, pool.heads, D,
                          pool.page, out.data_ptr(), lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                          status, ws.defined() ? ws.data_ptr() : nullptr,
                          ws.defined() ? static_cast<size_t>(ws.numel()) : 0, stream),
             "spec_cache_attend");
        PyObject* parts[3];
        const Tensor* from[3] = {&out, &lse, &ws};
        for (int i = 0; i < 3; ++i) parts[i] = from[i]->defined() ? THPVariable_Wrap(*from[i]) : Py_NewRef(Py_None);
        PyObject* r = PyObject_Vectorcall(g_attention, parts, 3, nullptr);
        for (PyObject* p : parts) Py_XDECREF(p);
        return r;
    });
}

// ---------------------------------------------------------------------------
// compaction and pages
// ---------------------------------------------------------------------------
PyObject* cache_compact(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"pool", "page_table", "ctx_len", "path_nodes", "num_accepted", "head_dim", "status", "stream"};
        const Args a("cache_compact", names, 8, 6, 6, args, nargs, kw);
        const int D = a.int32(5, 0, "head_dim");
        const Pool pool(a.v[0], 4, D);
        a.all_on(pool.device);
        const Table t(a.v[1], -1);
        const int B = checked(t.rows, "B");
        const Tensor& path = reachable(a.v[3], "path_nodes", at::kInt, "int32");
        if (path.dim() != 2 || path.size(0) != B || !path.is_contiguous())
            refuse("path_nodes must be a contiguous [B, path_width] int32 tensor");
        const int32_t* ctx = ints(a.v[2], "ctx_len", {B});
        const int32_t* accepted = ints(a.v[4], "num_accepted", {B});
        int32_t* status = ints_or_null(a.v[6], "status", {B});
        const Stream stream(a.v[7], pool.device);
        done(g_api.compact(pool.data, pool.layers, pool.layer_stride, pool.page_stride, pool.head_stride, pool.pages,
                           t.data, t.stride, t.width, ctx, static_cast<const int32_t*>(path.data_ptr()),
                           checked(path.size(1), "path_width"), accepted, B, pool.heads, D, pool.page, status,
                           stream),
             "spec_cache_compact");
        Py_RETURN_NONE;
    });
}

// The fields of a PageState.
struct Pages {
    PyObject* owned[5] = {};
    Table* table = nullptr;
    int32_t *held, *ref, *free_list, *num_free;
    int count, R;
    c10::Device device{c10::kCUDA, 0};

    explicit Pages(PyObject* o) {
        static const char* const names[] = {"page_table", "num_held", "ref", "free_list", "num_free"};
        static PyObject* interned[5] = {};
        try {
            for (int i = 0; i < 5; ++i) {
                if (!interned[i]) interned[i] = PyUnicode_InternFromString(names[i]);
                owned[i] = PyObject_GetAttr(o, interned[i]);
                if (!owned[i]) throw Raised{};
            }
            const Tensor& r = reachable(owned[2], "ref", at::kInt, "int32");
            if (!r.is_cuda()) refuse("ref must be device memory");
            device = r.device();
            for (int i = 0; i < 5; ++i) on_device(owned[i], names[i], device);
            table = new Table(owned[0], -1);
            R = checked(table->rows, "requests");
            const int64_t n = r.dim() == 1 ? r.size(0) : -1;
            ref = ints(owned[2], "ref", {n});
            held = ints(owned[1], "num_held", {R});
            free_list = ints(owned[3], "free_list", {n});
            num_free = ints(owned[4], "num_free", {1});
            count = checked(n, "pages");
        } catch (...) {
            release();
            throw;
        }
    }
    ~Pages() { release(); }
    Pages(const Pages&) = delete;
    Pages& operator=(const Pages&) = delete;
    void release() {
        for (PyObject*& p : owned) Py_CLEAR(p);
        delete table;
        table = nullptr;
    }
};

PyObject* grow_or_shrink(const char* who, decltype(&spec_cache_reserve) call, const char* c_name, PyObject* const* args,
                         Py_ssize_t nargs, PyObject* kw) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"pages", "length", "page_size", "status", "stream"};
        const Args a(who, names, 5, 3, 3, args, nargs, kw);
        const Pages s(a.v[0]);
        a.all_on(s.device);
        const int32_t* length = ints(a.v[1], "length", {s.R});
        int32_t* status = ints_or_null(a.v[3], "status", {s.R});
        const Stream stream(a.v[4], s.device);
        done(call(s.table->data, s.table->stride, s.table->width, s.held, s.ref, s.free_list, s.num_free, s.count,
                  length, s.R, a.int32(2, 0, "page_size"), status, stream),
             c_name);
        Py_RETURN_NONE;
    });
}
PyObject* cache_reserve(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return grow_or_shrink("cache_reserve", g_api.reserve, "spec_cache_reserve", args, nargs, kw);
}
PyObject* cache_release(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return grow_or_shrink("cache_release", g_api.release, "spec_cache_release", args, nargs, kw);
}

PyObject* cache_fork(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"pool", "pages", "src", "dst", "length", "head_dim", "new_page", "status", "stream"};
        const Args a("cache_fork", names, 9, 6, 6, args, nargs, kw);
        const int D = a.int32(5, 0, "head_dim");
        const Pool pool(a.v[0], 4, D);
        a.all_on(pool.device);
        const Pages s(a.v[1]);
        if (s.device != pool.device)
            refuse("the state is on %s, the pool on %s", s.device.str().c_str(), pool.device.str().c_str());
        if (s.count != pool.pages) refuse("the state has %d pages, the pool %d", s.count, pool.pages);
        const Tensor& first = reachable(a.v[2], "src", at::kInt, "int32");
        const int F = checked(first.dim() == 1 ? first.size(0) : -1, "forks");
        const int32_t* src = ints(a.v[2], "src", {F});
        const int32_t* dst = ints(a.v[3], "dst", {F});
        const int32_t* length = ints(a.v[4], "length", {s.R});
        int32_t* status = ints_or_null(a.v[7], "status", {F});
        const Stream stream(a.v[8], pool.device);
        const Tensor fresh = a.v[6] ? shaped(a.v[6], "new_page", at::kInt, "int32", {F})
                                    : at::empty({F}, at::TensorOptions(pool.device).dtype(at::kInt));
        done(g_api.fork(pool.data, pool.layers, pool.layer_stride, pool.page_stride, pool.head_stride, s.table->data,
                        s.table->stride, s.table->width, s.held, s.ref, s.free_list, s.num_free, s.count, src, dst,
                        length, s.R, F, pool.heads, D, pool.page, static_cast<int32_t*>(fresh.data_ptr()), status,
                        stream),
             "spec_cache_fork");
        return THPVariable_Wrap(fresh);
    });
}

// setup(SpecError, CacheAttention, addresses of the C functions in Api's order)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    constexpr Py_ssize_t kFns = sizeof(Api) / sizeof(void*);
    if (nargs != 2 + kFns) {
        PyErr_SetString(PyExc_TypeError, "setup() takes two classes and the C functions");
        return nullptr;
    }
    void* p[kFns];
    for (Py_ssize_t i = 0; i < kFns; ++i) {
        p[i] = PyLong_AsVoidPtr(args[2 + i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup() got a null function");
            return nullptr;
        }
    }
    Py_INCREF(args[0]);
    Py_XSETREF(g_error, args[0]);
    Py_INCREF(args[1]);
    Py_XSETREF(g_attention, args[1]);
    memcpy(&g_api, p, sizeof g_api);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fn(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)); }

PyMethodDef g_methods[] = {
    {"setup", fn(setup), METH_FASTCALL, nullptr},
    {"cache_append", fn(cache_append), METH_FASTCALL | METH_KEYWORDS,
     "cache_append(k, v, pool, page_table, start, count=None, *, status=None, stream=None)\n\n"
     "Write k, v [B, n, kv_heads, D] bf16 (any strides, unit element stride) into the cache in\n"
     "4 bits: row (b, i), i < count[b] (default n), at position start[b] + i.  Groups of 32\n"
     "values share a scale."},
    {"cache_read", fn(cache_read), METH_FASTCALL | METH_KEYWORDS,
     "cache_read(pool, page_table, start, n, head_dim, count=None, *, k=None, v=None, status=None, stream=None)\n\n"
     "Rows of the cache as bf16 values, exactly what the codes stand for: (k, v), each\n"
     "[B, n, kv_heads, D]; rows i >= count[b] are 0."},
    {"cache_attend", fn(cache_attend), METH_FASTCALL | METH_KEYWORDS,
     "cache_attend(q, pool, page_table, ctx_len, num_rows=None, *, anc_mask=None, depth=None, window=0, sinks=0,\n"
     "             scale=None, out=None, lse=None, want_lse=False, status=None, ws=None, stream=None)\n\n"
     "Attention of drafted rows q [B, n, q_heads, D] bf16 over the cache; returns a\n"
     "CacheAttention (out, lse, ws).\n\n"
     "Request b's cache holds ctx_len[b] context positions and behind them its num_rows[b]\n"
     "(default n) drafted rows, written by cache_append.  A row sees the context and, of the\n"
     "drafted rows, those in its anc_mask (int64 [B, n, ceil(n/64)], as tree_build writes it),\n"
     "or without a mask the rows up to itself.  Its position is ctx_len[b] + depth[b, i]\n"
     "(default i); with window > 0 it sees only keys of position p with p_i - p < window or\n"
     "p < sinks.  scale defaults to 1/sqrt(D).  Rows that see nothing are 0, their lse -inf;\n"
     "lse (natural log) is written when given or asked for.  Without a ws, calls on a stream\n"
     "share one and a captured graph has its own.  A ws of one's own starts zeroed, serves one\n"
     "stream, and outlives the graphs that were captured with it."},
    {"cache_compact", fn(cache_compact), METH_FASTCALL | METH_KEYWORDS,
     "cache_compact(pool, page_table, ctx_len, path_nodes, num_accepted, head_dim, *, status=None, stream=None)\n\n"
     "Keep an accepted path's rows: position ctx_len[b] + path_nodes[b, j] moves to\n"
     "ctx_len[b] + j, j = 0..num_accepted[b], in every layer of pool\n"
     "[layers, pages, kv_heads, block].  In place."},
    {"cache_reserve", fn(cache_reserve), METH_FASTCALL | METH_KEYWORDS,
     "cache_reserve(pages, length, page_size, *, status=None, stream=None)\n\n"
     "Give each request the pages it lacks for length[r] tokens, off the top of the stack,\n"
     "requests in order; one that they do not suffice for gets none (ST_NO_PAGE)."},
    {"cache_release", fn(cache_release), METH_FASTCALL | METH_KEYWORDS,
     "cache_release(pages, length, page_size, *, status=None, stream=None)\n\n"
     "Each request keeps the pages of length[r] tokens (0: none); pages that nothing holds any\n"
     "more are free.  A request cut back to a length inside a page that a fork made shared must\n"
     "not be written to (ST_SHARED_PAGE): fork it at that length and release it instead."},
    {"cache_fork", fn(cache_fork), METH_FASTCALL | METH_KEYWORDS,
     "cache_fork(pool, pages, src, dst, length, head_dim, *, new_page=None, status=None, stream=None)\n\n"
     "Request dst[f] (holding nothing) becomes a copy of request src[f] at length[src[f]]\n"
     "tokens: full pages are shared, the last partial one is copied in every layer of pool\n"
     "[layers, pages, kv_heads, block].  Returns new_page [F]: the page of its own that each\n"
     "got, or -1."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_spec_torch", "Binding of the cache calls.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__spec_torch(void) { return PyModule_Create(&g_module); }
