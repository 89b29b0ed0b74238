// Argument marshalling of the paged-attention entry points (CPython extension
// `_marshal`): tensors to the C ABI of include/kda.h, and nothing else.
//
// These calls take a few microseconds on the GPU, and a chain of them is bound by the
// host: looking at ten tensors from Python and passing 25 values through ctypes costs 6
// to 18 us a call, from here under one.  The module links to PyTorch only; the
// library's functions are handed to it by address when the library is loaded.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <string>
#include <utility>

#include "kda.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The library's entry points, in the order of kNames.
struct Library {
    decltype(&kda_page_plan) page_plan;
    decltype(&kda_qk_norm_rope) rope;
    decltype(&kda_qk_norm_rope_append) append;
    decltype(&kda_qk_norm_rope_bwd) rope_bwd;
    decltype(&kda_qk_norm_rope_bwd_workspace_size) rope_bwd_size;
    decltype(&kda_paged_decode) decode;
    decltype(&kda_paged_decode_workspace_size) decode_size;
} lib;
const char* const kNames[] = {"kda_page_plan", "kda_qk_norm_rope", "kda_qk_norm_rope_append",
                              "kda_qk_norm_rope_bwd", "kda_qk_norm_rope_bwd_workspace_size",
                              "kda_paged_decode", "kda_paged_decode_workspace_size"};

// A Python exception is set; unwinds to the entry point.
struct Raised {};

template <typename... A> [[noreturn]] void raise(PyObject* type, const char* format, A... args)
{
    PyErr_Format(type, format, args...);
    throw Raised();
}

std::string dtype_name(ScalarType t)
{
    switch (t) {
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Double: return "torch.float64";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        default: return std::string("torch ") + c10::toString(t);
    }
}

const Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

void need_dtype(const Tensor& t, const char* name, ScalarType dtype)
{
    if (t.scalar_type() != dtype)
        raise(PyExc_TypeError, "%s must be %s, not %s", name, dtype_name(dtype).c_str(),
              dtype_name(t.scalar_type()).c_str());
}
void need_cuda(const Tensor& t, const char* name)
{
    if (!t.is_cuda())
        raise(PyExc_RuntimeError, "%s must be a CUDA tensor (the library has no CPU path)", name);
}
int32_t code(ScalarType t)
{
    if (t == ScalarType::Float) return KDA_F32;
    if (t == ScalarType::BFloat16) return KDA_BF16;
    raise(PyExc_TypeError, "unsupported dtype %s", dtype_name(t).c_str());
}

// Device pointer of a contiguous tensor of `dtype` (and of n elements, unless negative).
template <typename T = void>
T* pointer(const Tensor& t, const char* name, ScalarType dtype, int64_t n = -1)
{
    need_dtype(t, name, dtype);
    if (n >= 0 && t.numel() != n)
        raise(PyExc_ValueError, "%s must have %lld elements, not %lld", name, (long long)n,
              (long long)t.numel());
    need_cuda(t, name);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T*>(t.data_ptr());
}
template <typename T> T* pointer_or_null(PyObject* o, const char* name, ScalarType dtype, int64_t n = -1)
{
    return o == Py_None ? nullptr : pointer<T>(tensor(o, name), name, dtype, n);
}
// A status word or a workspace: any contiguous CUDA tensor.
template <typename T> T* any_pointer(PyObject* o, const char* name)
{
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, name);
    need_cuda(t, name);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T*>(t.data_ptr());
}

void need_shape(const Tensor& t, const char* name, int64_t a, int64_t b, int64_t c)
{
    if (t.dim() != 3 || t.size(0) != a || t.size(1) != b || t.size(2) != c)
        raise(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld)", name, (long long)a,
              (long long)b, (long long)c);
}
void* dense(const Tensor& t, const char* name, ScalarType dtype, int64_t a, int64_t b, int64_t c)
{
    need_shape(t, name, a, b, c);
    return pointer<void>(t, name, dtype);
}

// [T, H, D] whose heads are dense within a token.
struct Rows {
    const void* p;
    int64_t stride;
};
Rows rows(const Tensor& t, const char* name, ScalarType dtype, int64_t T, int64_t H, int64_t D)
{
    need_dtype(t, name, dtype);
    need_shape(t, name, T, H, D);
    need_cuda(t, name);
    if ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1))
        raise(PyExc_ValueError, "%s: the heads of a token must be dense (strides %lld, %lld, %lld)",
              name, (long long)t.stride(0), (long long)t.stride(1), (long long)t.stride(2));
    return {t.data_ptr(), T > 1 ? t.stride(0) : H * D};
}

int32_t as_i32(int64_t x, const char* name)
{
    if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, "%s is out of range", name);
    return (int32_t)x;
}
int64_t integer(PyObject* o, const char* name)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, "%s must be an integer", name);
    }
    return x;
}
float number(PyObject* o, const char* name)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, "%s must be a number", name);
    }
    return (float)x;
}
int32_t flag(PyObject* o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Raised();
    return x;
}

// The stream of a call: the current one of the tensors' device, or the one given.  While this
// lives the device and the stream are the current ones: the library asks the device its
// sizes and launches there, and what the call allocates belongs to the stream that
// writes it: the memory waits for that stream's calls, and a captured stream's is its graph's.
class Stream {
    static c10::cuda::CUDAStream find(PyObject* o, const Tensor& t)
    {
        const c10::DeviceIndex dev = t.device().index();
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev);
        PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw Raised();
        void* p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw Raised();
        return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), dev);
    }
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard current;

public:
    const c10::cuda::CUDAStream s;
    Stream(PyObject* o, const Tensor& t) : s(find(o, t))
    {
        if (c10::cuda::current_device() != t.device().index()) device.set_device(t.device());
        if (o != Py_None) current.reset_stream(s);
    }
    kda_stream_t handle() const { return reinterpret_cast<kda_stream_t>(s.stream()); }
};

at::TensorOptions like(const Tensor& t, ScalarType dtype)
{
    return at::TensorOptions().device(t.device()).dtype(dtype);
}
Tensor output(PyObject* given, const char* name, at::IntArrayRef shape, const Tensor& t, ScalarType dtype)
{
    return given == Py_None ? at::empty(shape, like(t, dtype)) : tensor(given, name);
}
ScalarType dtype_or(PyObject* o, ScalarType otherwise)
{
    if (o == Py_None) return otherwise;
    if (!THPDtype_Check(o)) raise(PyExc_TypeError, "a dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// Whether the call's stream, which need not be the current one, is being captured.
bool captures(const Stream& stream)
{
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    C10_CUDA_CHECK(cudaStreamIsCapturing(stream.s.stream(), &st));
    return st != cudaStreamCaptureStatusNone;
}

// The workspace of a call that was given none: one buffer per stream, kept and grown,
// since calls on one stream are ordered.  A captured call gets one of its graph's own.
struct Workspace {
    Tensor keep;
    void* p = nullptr;
    int64_t bytes = 0;
};
Workspace workspace(PyObject* given, int64_t bytes, const Tensor& t, const Stream& stream)
{
    Workspace w;
    if (given != Py_None) {
        w.p = any_pointer<void>(given, "workspace");
        w.bytes = (int64_t)tensor(given, "workspace").nbytes();
        return w;
    }
    w.bytes = bytes;
    const auto bytes_like = like(t, ScalarType::Byte);
    if (captures(stream)) {
        w.keep = at::empty({bytes}, bytes_like);
    } else {
        // never destroyed: the allocator may be gone first when the process ends
        static auto* kept = new std::map<std::pair<int, cudaStream_t>, Tensor>;
        Tensor& mine = (*kept)[{t.device().index(), stream.s.stream()}];
        if (!mine.defined() || mine.numel() < bytes) mine = at::empty({bytes}, bytes_like);
        w.keep = mine;
    }
    w.p = w.keep.data_ptr();
    return w;
}

// Sizes depend on the device and the arguments alone; asked once each.
template <typename F> int64_t size_of(F ask, const int64_t (&key)[4], std::map<std::array<int64_t, 4>, int64_t>& known)
{
    const std::array<int64_t, 4> k = {key[0], key[1], key[2], key[3]};
    const auto it = known.find(k);
    if (it != known.end()) return it->second;
    int64_t bytes = 0;
    if (ask(&bytes) != KDA_OK) return 0;       // the call itself refuses and says why
    if (known.size() > 4096) known.clear();
    known[k] = bytes;
    return bytes;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap_or_none(const Tensor& t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
// New references to a tuple; on a failed element the whole is dropped.
template <size_t N> PyObject* tuple(PyObject* const (&items)[N])
{
    PyObject* t = PyTuple_New(N);
    bool ok = t != nullptr;
    for (size_t i = 0; i < N; ++i) {
        ok = ok && items[i] != nullptr;
        if (t) PyTuple_SET_ITEM(t, i, items[i]);
        else Py_XDECREF(items[i]);
    }
    if (!ok) {
        Py_XDECREF(t);
        return nullptr;
    }
    return t;
}

// A call's CUDA tensors are on one device, which Stream makes the current one.
void need_one_device(PyObject* const* a, Py_ssize_t n)
{
    int first = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPVariable_Check(a[i])) continue;
        const at::Device d = THPVariable_Unpack(a[i]).device();
        if (!d.is_cuda()) continue;            // refused by name, with what it should be
        if (first < 0) first = d.index();
        if (d.index() != first)
            raise(PyExc_ValueError, "all tensors of a call must be on one device, not cuda:%d and cuda:%d",
                  first, (int)d.index());
    }
}

// What every entry does: its arguments counted, Python errors and C++ exceptions caught.
// A refusal by the library comes back as its status, an int.
template <typename F> PyObject* entry(PyObject* const* a, Py_ssize_t got, Py_ssize_t want, F body)
{
    HANDLE_TH_ERRORS
    if (got != want) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    if (!lib.page_plan) {
        PyErr_SetString(PyExc_RuntimeError, "the KDA library is not loaded");
        return nullptr;
    }
    try {
        need_one_device(a, got);
        return body();
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
PyObject* status(kda_status st) { return PyLong_FromLong(st); }

PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return entry(a, n, 13, [&]() -> PyObject* {
        const Tensor &cached = tensor(a[0], "cached_lens"), &cu = tensor(a[1], "cu_seqlens"),
                     &table = tensor(a[2], "block_table"), &free = tensor(a[3], "free_pages");
        const int64_t N = cached.numel(), T = integer(a[5], "num_tokens");
        if (table.dim() != 2 || table.size(0) != N)
            raise(PyExc_ValueError, "block_table must have shape [%lld, max_pages]", (long long)N);
        const auto i32 = ScalarType::Int;
        const int32_t* c = pointer<int32_t>(cached, "cached_lens", i32);
        const Stream s(a[12], cached);
        const Tensor lens = output(a[7], "seq_lens", {N}, cached, i32),
                     pos = output(a[8], "positions", {T}, cached, i32),
                     slots = output(a[9], "slots", {T}, cached, ScalarType::Long),
                     end = output(a[10], "free_end", {1}, cached, i32);
        const kda_status st = lib.page_plan(
            c, pointer<int32_t>(cu, "cu_seqlens", i32, N + 1), as_i32(N, "the number of requests"), T,
            as_i32(integer(a[4], "page_size"), "page_size"), pointer<int32_t>(table, "block_table", i32),
            as_i32(table.size(1), "max_pages"), pointer<int32_t>(free, "free_pages", i32),
            as_i32(free.numel(), "the number of free pages"),
            pointer_or_null<int32_t>(a[6], "free_start", i32, 1),
            pointer<int32_t>(lens, "seq_lens", i32, N), pointer<int32_t>(pos, "positions", i32, T),
            pointer<int64_t>(slots, "slots", ScalarType::Long, T),
            pointer<int32_t>(end, "free_end", i32, 1), any_pointer<int32_t>(a[11], "status"),
            s.handle());
        if (st != KDA_OK) return status(st);
        return tuple({wrap(lens), wrap(pos), wrap(slots), wrap(end)});
    });
}

// positions, inv_freq, q_weight, k_weight, eps, qk_norm, interleaved, rope_scale: a[0 .. 7].
struct Rope {
    const int32_t* positions;
    const float* inv_freq;
    int32_t rot;
    const float *qw, *kw;
    float eps;
    int32_t norm, inter;
    float scale;
    Rope(PyObject* const* a, int64_t T, int64_t D)
    {
        positions = pointer<int32_t>(tensor(a[0], "positions"), "positions", ScalarType::Int, T);
        const int64_t pairs = a[1] == Py_None ? 0 : tensor(a[1], "inv_freq").numel();
        inv_freq = pointer_or_null<float>(a[1], "inv_freq", ScalarType::Float);
        rot = as_i32(2 * pairs, "the rotated channels");
        qw = pointer_or_null<float>(a[2], "q_weight", ScalarType::Float, D);
        kw = pointer_or_null<float>(a[3], "k_weight", ScalarType::Float, D);
        eps = number(a[4], "eps");
        norm = flag(a[5]);
        inter = flag(a[6]);
        scale = number(a[7], "rope_scale");
    }
};

// q [T, Hq, D] and the heads of k.
struct Heads {
    int64_t T;
    int32_t Hq, Hk, D;
    Heads(const Tensor& q, const Tensor& k)
    {
        if (q.dim() != 3) raise(PyExc_ValueError, "q must have shape [T, Hq, D]");
        if (k.dim() != 3) raise(PyExc_ValueError, "k must have shape [T, Hk, D]");
        T = q.size(0);
        Hq = as_i32(q.size(1), "the number of heads");
        Hk = as_i32(k.size(1), "the number of heads");
        D = as_i32(q.size(2), "the head dimension");
        need_dtype(k, "k", q.scalar_type());
    }
};

PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return entry(a, n, 14, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
        const auto dt = q.scalar_type();
        const Heads h(q, k);
        const Rows qr = rows(q, "q", dt, h.T, h.Hq, h.D), kr = rows(k, "k", dt, h.T, h.Hk, h.D);
        const Rope r(a + 2, h.T, h.D);
        const Stream s(a[13], q);
        const Tensor qo = output(a[10], "q_out", {h.T, h.Hq, h.D}, q, dtype_or(a[12], dt));
        const auto odt = qo.scalar_type();
        const Tensor ko = output(a[11], "k_out", {h.T, h.Hk, h.D}, q, odt);
        const kda_status st = lib.rope(
            qr.p, qr.stride, kr.p, kr.stride, code(dt), r.positions, r.inv_freq, r.rot, r.inter, r.scale,
            r.qw, r.kw, r.eps, r.norm, h.T, h.Hq, h.Hk, h.D, dense(qo, "q_out", odt, h.T, h.Hq, h.D),
            dense(ko, "k_out", odt, h.T, h.Hk, h.D), code(odt), s.handle());
        if (st != KDA_OK) return status(st);
        return tuple({wrap(qo), wrap(ko)});
    });
}

// The caches' shape [num_pages, Hk, page_size, D].
void need_caches(const Tensor& kc, const Tensor& vc, int64_t Hk, int64_t D)
{
    if (kc.dim() != 4 || (Hk >= 0 && kc.size(1) != Hk) || kc.size(3) != D)
        raise(PyExc_ValueError, "k_cache must have shape [num_pages, %s%lld, page_size, %lld]",
              Hk < 0 ? "Hk, not " : "", (long long)(Hk < 0 ? kc.dim() : Hk), (long long)D);
    if (vc.sizes() != kc.sizes() || vc.scalar_type() != kc.scalar_type())
        raise(PyExc_ValueError, "v_cache must have the shape and dtype of k_cache");
}

PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return entry(a, n, 17, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
                     &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache");
        const auto dt = q.scalar_type(), cdt = kc.scalar_type();
        const Heads h(q, k);
        need_caches(kc, vc, h.Hk, h.D);
        const Rows qr = rows(q, "q", dt, h.T, h.Hq, h.D), kr = rows(k, "k", dt, h.T, h.Hk, h.D),
                   vr = rows(v, "v", dt, h.T, h.Hk, h.D);
        const Rope r(a + 6, h.T, h.D);
        const Stream s(a[16], q);
        const Tensor qo = output(a[14], "q_out", {h.T, h.Hq, h.D}, q, cdt);
        const kda_status st = lib.append(
            qr.p, qr.stride, kr.p, kr.stride, vr.p, vr.stride, code(dt), r.positions,
            pointer<int64_t>(tensor(a[3], "slots"), "slots", ScalarType::Long, h.T), r.inv_freq, r.rot,
            r.inter, r.scale, r.qw, r.kw, r.eps, r.norm, h.T, h.Hq, h.Hk, h.D,
            dense(qo, "q_out", cdt, h.T, h.Hq, h.D), pointer(kc, "k_cache", cdt),
            pointer(vc, "v_cache", cdt), code(cdt), as_i32(kc.size(0), "the number of pages"),
            as_i32(kc.size(2), "page_size"), any_pointer<int32_t>(a[15], "status"),
            s.handle());
        if (st != KDA_OK) return status(st);
        return wrap(qo);
    });
}

PyObject* norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return entry(a, n, 17, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &dq = tensor(a[2], "dq_out"),
                     &dk = tensor(a[3], "dk_out");
        const auto dt = q.scalar_type(), ydt = dq.scalar_type();
        const Heads h(q, k);
        const Rows qr = rows(q, "q", dt, h.T, h.Hq, h.D), kr = rows(k, "k", dt, h.T, h.Hk, h.D);
        const Rope r(a + 4, h.T, h.D);
        const Stream s(a[16], q);
        const Tensor qg = output(a[12], "q_grad", {h.T, h.Hq, h.D}, q, dtype_or(a[14], ScalarType::Float));
        const auto gdt = qg.scalar_type();
        const Tensor kg = output(a[13], "k_grad", {h.T, h.Hk, h.D}, q, gdt);
        Tensor wq, wk;
        if (r.norm && r.qw) wq = at::empty({h.D}, like(q, ScalarType::Float));
        if (r.norm && r.kw) wk = at::empty({h.D}, like(q, ScalarType::Float));
        Workspace w;
        if (wq.defined() || wk.defined() || a[15] != Py_None) {
            static auto* known = new std::map<std::array<int64_t, 4>, int64_t>;
            const int64_t bytes = size_of(
                [&](int64_t* b) { return lib.rope_bwd_size(h.T, h.Hq, h.Hk, h.D, b); },
                {q.device().index(), h.D, 0, 0}, *known);
            w = workspace(a[15], bytes, q, s);
        }
        const kda_status st = lib.rope_bwd(
            qr.p, qr.stride, kr.p, kr.stride, code(dt), dense(dq, "dq_out", ydt, h.T, h.Hq, h.D),
            dense(dk, "dk_out", ydt, h.T, h.Hk, h.D), code(ydt), r.positions, r.inv_freq, r.rot, r.inter,
            r.scale, r.qw, r.kw, r.eps, r.norm, h.T, h.Hq, h.Hk, h.D,
            dense(qg, "q_grad", gdt, h.T, h.Hq, h.D), dense(kg, "k_grad", gdt, h.T, h.Hk, h.D), code(gdt),
            wq.defined() ? wq.data_ptr<float>() : nullptr, wk.defined() ? wk.data_ptr<float>() : nullptr,
            w.p, w.bytes, s.handle());
        if (st != KDA_OK) return status(st);
        return tuple({wrap(qg), wrap(kg), wrap_or_none(wq), wrap_or_none(wk)});
    });
}

PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return entry(a, n, 13, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                     &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
        if (q.dim() != 3) raise(PyExc_ValueError, "q must have shape [N, Hq, D]");
        const int64_t N = q.size(0);
        const int32_t Hq = as_i32(q.size(1), "the number of heads"), D = as_i32(q.size(2), "the head dimension");
        need_caches(kc, vc, -1, D);
        const int32_t Hk = as_i32(kc.size(1), "the number of heads");
        if (table.dim() != 2 || table.size(0) != N)
            raise(PyExc_ValueError, "block_table must have shape [%lld, max_pages]", (long long)N);
        const auto dt = kc.scalar_type(), f32 = ScalarType::Float;
        const void* qp = pointer(q, "q", dt);
        const Stream s(a[12], q);
        const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : number(a[5], "scale");
        const Tensor out = output(a[6], "out", {N, Hq, D}, q, dtype_or(a[7], dt));
        const auto odt = out.scalar_type();
        Tensor lse;
        if (a[8] != Py_None) lse = tensor(a[8], "lse");
        else if (flag(a[9])) lse = at::empty({N, Hq}, like(q, f32));
        static auto* known = new std::map<std::array<int64_t, 4>, int64_t>;
        const int64_t bytes = a[11] != Py_None ? 0 : size_of(
            [&](int64_t* b) { return lib.decode_size(as_i32(N, "the number of requests"), Hq, Hk, D, b); },
            {q.device().index(), ((int64_t)Hq << 32) | (uint32_t)Hk, D, N}, *known);
        const Workspace w = workspace(a[11], bytes, q, s);
        const kda_status st = lib.decode(
            qp, pointer(kc, "k_cache", dt), pointer(vc, "v_cache", dt), code(dt),
            pointer<int32_t>(table, "block_table", ScalarType::Int),
            pointer<int32_t>(lens, "seq_lens", ScalarType::Int, N), as_i32(N, "the number of requests"), Hq,
            Hk, D, as_i32(kc.size(0), "the number of pages"), as_i32(kc.size(2), "page_size"),
            as_i32(table.size(1), "max_pages"), scale, dense(out, "out", odt, N, Hq, D), code(odt),
            lse.defined() ? pointer<float>(lse, "lse", f32, N * Hq) : nullptr, w.p, w.bytes,
            any_pointer<int32_t>(a[10], "status"), s.handle());
        if (st != KDA_OK) return status(st);
        return tuple({wrap(out), wrap_or_none(lse)});
    });
}

// bind(names -> addresses): the loaded library's functions.
PyObject* bind(PyObject*, PyObject* addresses)
{
    void* at[sizeof(kNames) / sizeof(*kNames)];
    for (size_t i = 0; i < sizeof(kNames) / sizeof(*kNames); ++i) {
        PyObject* o = PyDict_GetItemString(addresses, kNames[i]);
        at[i] = o ? PyLong_AsVoidPtr(o) : nullptr;
        if (!at[i]) return PyErr_Format(PyExc_KeyError, "%s", kNames[i]);
    }
    static_assert(sizeof(lib) == sizeof(at), "one address per entry point");
    memcpy(&lib, at, sizeof(lib));
    Py_RETURN_NONE;
}

template <typename F> PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef kMethods[] = {{"bind", bind, METH_O, nullptr},
                          {"page_plan", fast(page_plan), METH_FASTCALL, nullptr},
                          {"norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
                          {"append", fast(append), METH_FASTCALL, nullptr},
                          {"norm_rope_bwd", fast(norm_rope_bwd), METH_FASTCALL, nullptr},
                          {"paged_decode", fast(paged_decode), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
