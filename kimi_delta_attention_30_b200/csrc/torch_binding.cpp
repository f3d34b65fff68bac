// Marshalling of torch tensors into the C ABI for the calls that take microseconds on the
// GPU (linear attention with one decay a head, query/key norm with rotation): argument
// checks, output and scratch allocation, current stream.  Nothing is computed here.  The
// same checks in Python cost 6 to 28 us a call, more than a decode step's kernel.
//
// Functions take positional arguments only (the package's functions of the same names pass
// them).  `stream` is None (the device's current stream) or (handle, stream_id, device index,
// device type) of another stream of the same device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>
#include <vector>

#include "kda.h"

// What this module is compiled for (build.py reads it before the module is loaded).
extern "C" __attribute__((used, visibility("default"))) const char kda_binding_built_for[] =
    "kda binding built for [" KDA_BUILT_FOR "]";

namespace {

PyObject* g_error = nullptr;   // KdaError
PyObject* g_memory = nullptr;  // torch.OutOfMemoryError

struct BadValue : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Status {
    int code;
    const char* what;
};
struct PythonError {};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char* dtype_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return c10::toString(t);
    }
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) throw BadValue(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

void on_device(const char* name, const at::Tensor& t, int dev) {
    if (!t.is_cuda()) throw BadValue(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
    if (t.get_device() != dev)
        throw BadValue(std::string(name) + " is on " + t.device().str() + ", the call runs on cuda:" + std::to_string(dev));
}

void of_type(const char* name, const at::Tensor& t, at::ScalarType dt) {
    if (t.scalar_type() != dt)
        throw BadValue(std::string(name) + " has dtype " + dtype_text(t.scalar_type()) + ", expected " + dtype_text(dt));
}

void of_shape(const char* name, const at::Tensor& t, at::IntArrayRef shape) {
    if (t.sizes() != shape)
        throw BadValue(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
}

// A contiguous tensor of this device, type and shape.
void* dense(const char* name, const at::Tensor& t, int dev, at::ScalarType dt, at::IntArrayRef shape) {
    on_device(name, t, dev);
    of_type(name, t, dt);
    of_shape(name, t, shape);
    if (!t.is_contiguous()) throw BadValue(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void* dense(const char* name, PyObject* o, int dev, at::ScalarType dt, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : dense(name, tensor(name, o), dev, dt, shape);
}

kda_dtype type_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    if (t.scalar_type() == at::kFloat) return KDA_F32;
    throw BadValue(std::string("unsupported dtype ") + dtype_text(t.scalar_type()));
}

int device_of(const char* name, const at::Tensor& t) {
    type_of(t);
    if (!t.is_cuda()) throw BadValue(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
    return t.get_device();
}

// The device and stream of one call, and the tensors it allocates.  Memory comes from the pool
// of the call's own stream: a block of the current stream's pool may still be in use by what is
// queued there, which another stream does not wait for.
struct Call {
    c10::cuda::OptionalCUDAGuard guard;
    c10::cuda::OptionalCUDAStreamGuard on;
    int dev;
    void* raw;
    std::optional<c10::Stream> home;   // the current stream, where the call runs on another
    std::vector<at::Tensor> made;

    Call(int device, PyObject* stream) : dev(device) {
        guard.set_index((c10::DeviceIndex)device);
        const auto cur = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device);
        raw = cur.stream();
        if (stream != Py_None) {
            unsigned long long handle;
            long long id, index, type;
            if (!PyArg_ParseTuple(stream, "KLLL", &handle, &id, &index, &type)) throw PythonError();
            if (index != device)
                throw BadValue("stream belongs to cuda:" + std::to_string(index) + ", the call runs on cuda:" +
                               std::to_string(device));
            if ((void*)handle != raw) {
                raw = (void*)handle;
                home = cur.unwrap();
                on.reset_stream(c10::Stream::unpack3(id, (c10::DeviceIndex)index, (c10::DeviceType)type));
            }
        }
    }
    at::Tensor scratch(at::IntArrayRef shape, at::ScalarType dt) {
        return at::detail::empty_cuda(shape, dt, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType dt) {   // a result
        at::Tensor t = scratch(shape, dt);
        if (home) made.push_back(t);
        return t;
    }
    // results are the caller's from here on, whose stream is not the one they were allocated for
    void done(int status, const char* what) {
        if (home)
            for (const at::Tensor& t : made) t.record_stream(*home);
        if (status != KDA_OK) throw Status{status, what};
    }
};

// Scratch: the given workspace (any dtype, contiguous), or a new one of `need` bytes.
struct Scratch {
    at::Tensor own;
    void* ptr;
    size_t bytes;
    template <typename Need>
    Scratch(Call& c, PyObject* given, Need need) {
        if (given == Py_None) {
            const size_t n = need();
            own = c.scratch({(int64_t)(n > 256 ? n : 256)}, at::kByte);
            ptr = own.data_ptr();
            bytes = (size_t)own.numel();
        } else {
            const at::Tensor& t = tensor("workspace", given);
            on_device("workspace", t, c.dev);
            if (!t.is_contiguous()) throw BadValue("workspace must be contiguous");
            ptr = t.data_ptr();
            bytes = t.nbytes();
        }
    }
};

bool truth(PyObject* o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw PythonError();
    return t != 0;
}

std::vector<int32_t> offsets(PyObject* cu) {   // a list or tuple of ints
    std::vector<int32_t> v;
    if (cu == Py_None) return v;
    PyObject* seq = PySequence_Fast(cu, "cu_seqlens must be a sequence of ints");
    if (!seq) throw PythonError();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    v.resize((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const long long x = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
        if (x == -1 && PyErr_Occurred()) {
            Py_DECREF(seq);
            throw PythonError();
        }
        v[(size_t)i] = x < INT32_MIN || x > INT32_MAX ? -1 : (int32_t)x;   // -1: refused as an offset
    }
    Py_DECREF(seq);
    if (v.empty()) throw BadValue("cu_seqlens must hold at least one offset");
    return v;
}

int small(const char* name, int64_t n) {
    if (n > INT32_MAX) throw BadValue(std::string(name) + " is too large");
    return (int)n;
}

// What the chunk calls share.
struct Linear {
    const at::Tensor &q, &k, &v, &la;
    int dev;
    at::ScalarType dt;
    kda_dtype type;
    kda_decay decay;
    int B, T, H, dk, dv;
    void *pq, *pk, *pv, *pla;
    std::vector<int32_t> cu;
    int64_t N;

    Linear(PyObject* const* a, PyObject* seqlens)
        : q(tensor("q", a[0])), k(tensor("k", a[1])), v(tensor("v", a[2])), la(tensor("log_alpha", a[3])) {
        dev = device_of("q", q);
        type = type_of(q);
        dt = q.scalar_type();
        if (q.dim() != 4 || v.dim() != 4) throw BadValue("q and v must have 4 dimensions [B, T, H, d]");
        B = small("B", q.size(0)); T = small("T", q.size(1)); H = small("H", q.size(2)); dk = small("dk", q.size(3));
        dv = small("dv", v.size(3));
        pq = dense("q", q, dev, dt, q.sizes());
        pk = dense("k", k, dev, dt, q.sizes());
        pv = dense("v", v, dev, dt, {B, T, H, dv});
        if (la.dim() == 1) {
            decay = KDA_DECAY_HEAD;
            pla = dense("log_alpha", la, dev, at::kFloat, {H});
        } else {
            decay = KDA_DECAY_TOKEN;
            pla = dense("log_alpha", la, dev, dt, {B, T, H});
        }
        cu = offsets(seqlens);
        N = cu.empty() ? B : (int64_t)cu.size() - 1;
    }
    const int32_t* cu_ptr() const { return cu.empty() ? nullptr : cu.data(); }
    int n_seqs() const { return cu.empty() ? 0 : (int)N; }
};

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// A tensor of the caller's that the call writes: its version counter goes up, so that autograd
// notices if it had been saved for a backward pass.
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The caller's output tensor, or a new one.
at::Tensor output(Call& c, const char* name, PyObject* given, at::ScalarType dt, at::IntArrayRef shape) {
    if (given == Py_None) return c.make(shape, dt);
    const at::Tensor& t = tensor(name, given);
    dense(name, t, c.dev, dt, shape);
    written(t);
    return t;
}

PyObject* pack(std::initializer_list<at::Tensor> ts) {
    PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) throw PythonError();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, wrap(t));
    return out;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// (q, k, v, log_alpha, init_state, cu_seqlens, output_final_state, o, final_state, workspace, stream)
PyObject* linear_chunk_fwd(PyObject* const* a) {
    const Linear L(a, a[5]);
    const int64_t st[4] = {L.N, L.H, L.dk, L.dv};
    void* init = dense("init_state", a[4], L.dev, at::kFloat, st);
    Call c(L.dev, a[10]);
    const at::Tensor o = output(c, "o", a[7], L.dt, L.v.sizes());
    at::Tensor fs;
    if (a[8] != Py_None || truth(a[6])) fs = output(c, "final_state", a[8], at::kFloat, st);
    const Scratch w(c, a[9], [&] {
        return kda_linear_chunk_fwd_workspace_size(L.B, L.T, L.H, L.dk, L.dv, L.type, L.cu_ptr(), L.n_seqs());
    });
    c.done(kda_linear_chunk_fwd(L.pq, L.pk, L.pv, L.pla, L.decay, L.type, (const float*)init, L.cu_ptr(), L.n_seqs(), L.B,
                                L.T, L.H, L.dk, L.dv, o.data_ptr(), (float*)ptr(fs), w.ptr, w.bytes, c.raw),
           "kda_linear_chunk_fwd");
    return pack({o, fs});
}

// (q, k, v, log_alpha, d_o, init_state, d_final_state, cu_seqlens, need_d_init_state, dq, dk, dv, dlog_alpha,
//  d_init_state, given, workspace, stream); given: the five outputs are the caller's (None: not wanted)
PyObject* linear_chunk_bwd(PyObject* const* a) {
    const Linear L(a, a[7]);
    const int64_t st[4] = {L.N, L.H, L.dk, L.dv};
    void* pdo = dense("d_o", tensor("d_o", a[4]), L.dev, L.dt, L.v.sizes());
    void* init = dense("init_state", a[5], L.dev, at::kFloat, st);
    void* pdf = dense("d_final_state", a[6], L.dev, at::kFloat, st);
    Call c(L.dev, a[16]);
    const bool given = truth(a[14]);
    at::Tensor dq, dk, dv, dla, ds;
    if (!given || a[9] != Py_None) dq = output(c, "dq", a[9], L.dt, L.q.sizes());
    if (!given || a[10] != Py_None) dk = output(c, "dk", a[10], L.dt, L.k.sizes());
    if (!given || a[11] != Py_None) dv = output(c, "dv", a[11], L.dt, L.v.sizes());
    if (given ? a[12] != Py_None : L.decay == KDA_DECAY_TOKEN)
        dla = output(c, "dlog_alpha", a[12], L.la.scalar_type(), L.la.sizes());
    if (given ? a[13] != Py_None : truth(a[8])) ds = output(c, "d_init_state", a[13], at::kFloat, st);
    const Scratch w(c, a[15], [&] {
        return kda_linear_chunk_bwd_workspace_size(L.B, L.T, L.H, L.dk, L.dv, L.type, L.cu_ptr(), L.n_seqs());
    });
    c.done(kda_linear_chunk_bwd(L.pq, L.pk, L.pv, L.pla, L.decay, L.type, (const float*)init, L.cu_ptr(), L.n_seqs(), L.B,
                                L.T, L.H, L.dk, L.dv, pdo, (const float*)pdf, ptr(dq), ptr(dk), ptr(dv), ptr(dla),
                                (float*)ptr(ds), w.ptr, w.bytes, c.raw),
           "kda_linear_chunk_bwd");
    return pack({dq, dk, dv, dla, ds});
}

// (q, k, v, log_alpha, state, o, stream)
PyObject* linear_decode_step(PyObject* const* a) {
    const at::Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]), &la = tensor("log_alpha", a[3]);
    const int dev = device_of("q", q);
    const at::ScalarType dt = q.scalar_type();
    if (q.dim() != 3 || v.dim() != 3) throw BadValue("q and v must have 3 dimensions [N, H, d]");
    const int64_t N = q.size(0), H = q.size(1), dk = q.size(2), dv = v.size(2);
    void *pq = dense("q", q, dev, dt, q.sizes()), *pk = dense("k", k, dev, dt, q.sizes()),
         *pv = dense("v", v, dev, dt, {N, H, dv});
    const bool per_head = la.dim() == 1;
    void* pla = per_head ? dense("log_alpha", la, dev, at::kFloat, {H}) : dense("log_alpha", la, dev, dt, {N, H});
    const at::Tensor& state = tensor("state", a[4]);
    void* ps = dense("state", state, dev, at::kFloat, {N, H, dk, dv});
    Call c(dev, a[6]);
    written(state);
    const at::Tensor o = output(c, "o", a[5], dt, v.sizes());
    c.done(kda_linear_decode_step(pq, pk, pv, pla, per_head ? KDA_DECAY_HEAD : KDA_DECAY_TOKEN, type_of(q), (float*)ps,
                                  small("N", N), small("H", H), small("dk", dk), small("dv", dv), o.data_ptr(), c.raw),
           "kda_linear_decode_step");
    return wrap(o);
}

// [..., H, d] as kda_rows: any strides that let the leading dimensions be walked with one step
kda_rows rows(const char* name, const at::Tensor& t, int dev, at::ScalarType dt) {
    on_device(name, t, dev);
    of_type(name, t, dt);
    const int64_t n = t.dim();
    if (n < 2) throw BadValue(std::string(name) + " must have shape [..., H, d]");
    const int64_t H = t.size(n - 2), d = t.size(n - 1);
    if (t.is_contiguous()) return kda_rows{t.data_ptr(), H * d, d};
    if (t.stride(n - 1) != 1 && d > 1) throw BadValue(std::string(name) + " must be contiguous in its last dimension");
    if (t.numel() == 0) return kda_rows{nullptr, 0, 0};
    int64_t token = 0, walked = 0;   // the innermost stride of more than one step, and its steps
    for (int64_t i = n - 3; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (walked == 0) {
            token = t.stride(i);
            walked = t.size(i);
        } else {
            if (t.stride(i) != token * walked)
                throw BadValue(std::string(name) + "'s token dimensions must be walkable with one stride");
            walked *= t.size(i);
        }
    }
    // a stride that no step is made along is taken as that of packed heads
    const int64_t head = H > 1 ? t.stride(n - 2) : d;
    return kda_rows{t.data_ptr(), walked ? token : H * head, head};
}

struct NormRope {
    const at::Tensor &q, &k;
    int dev;
    at::ScalarType dt, wdt;
    kda_rows rq, rk;
    long long T;
    int Hq, Hk, d, rot = 0;
    void *wq = nullptr, *wk = nullptr, *pos = nullptr, *freq = nullptr;
    float eps;
    int interleaved;

    // (q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)
    explicit NormRope(PyObject* const* a) : q(tensor("q", a[0])), k(tensor("k", a[1])) {
        dev = device_of("q", q);
        dt = wdt = q.scalar_type();
        rq = rows("q", q, dev, dt);
        rk = rows("k", k, dev, dt);
        const auto lead = q.sizes().slice(0, q.dim() - 2);
        Hq = small("Hq", q.size(-2)); Hk = small("Hk", k.size(-2)); d = small("d", q.size(-1));
        if (k.dim() != q.dim() || k.sizes().slice(0, k.dim() - 2) != lead || k.size(-1) != d) {
            std::vector<int64_t> want(lead.begin(), lead.end());
            want.push_back(Hk);
            want.push_back(d);
            of_shape("k", k, want);
        }
        T = 1;
        for (const int64_t n : lead) T *= n;
        for (const int i : {3, 2})
            if (a[i] != Py_None) wdt = tensor("weight", a[i]).scalar_type();
        if (wdt != at::kBFloat16 && wdt != at::kFloat)
            throw BadValue(std::string("unsupported weight dtype ") + dtype_text(wdt));
        wq = dense("q_weight", a[2], dev, wdt, {d});
        wk = dense("k_weight", a[3], dev, wdt, {d});
        if (a[5] != Py_None) {
            const at::Tensor& f = tensor("inv_freq", a[5]);
            if (f.dim() != 1) throw BadValue("inv_freq must have one dimension [rot / 2]");
            freq = dense("inv_freq", f, dev, at::kFloat, f.sizes());
            rot = 2 * small("rot", f.size(0));
            if (a[4] == Py_None) throw BadValue("positions are required with inv_freq");
            pos = dense("positions", a[4], dev, at::kInt, lead);
        } else if (a[4] != Py_None) {
            throw BadValue("inv_freq is required with positions");
        }
        const double e = PyFloat_AsDouble(a[6]);
        if (e == -1.0 && PyErr_Occurred()) throw PythonError();
        eps = (float)e;
        interleaved = truth(a[7]);
    }
    kda_dtype wtype() const { return wdt == at::kFloat ? KDA_F32 : KDA_BF16; }
    kda_rows out_rows(const char* name, const at::Tensor& t, const at::Tensor& like) const {
        of_shape(name, t, like.sizes());
        return rows(name, t, dev, dt);
    }
    at::Tensor out(Call& c, const char* name, PyObject* given, const at::Tensor& like) const {
        if (given == Py_None) return c.make(like.sizes(), dt);
        const at::Tensor& t = tensor(name, given);
        written(t);
        return t;
    }
};

// (the eight above, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject* const* a) {
    const NormRope A(a);
    Call c(A.dev, a[10]);
    const at::Tensor qo = A.out(c, "q_out", a[8], A.q), ko = A.out(c, "k_out", a[9], A.k);
    const kda_rows oq = A.out_rows("q_out", qo, A.q), ok = A.out_rows("k_out", ko, A.k);
    c.done(kda_qk_norm_rope(&A.rq, &A.rk, A.wq, A.wk, A.wtype(), (const int32_t*)A.pos, (const float*)A.freq, type_of(A.q),
                            A.T, A.Hq, A.Hk, A.d, A.rot, A.eps, A.interleaved, &oq, &ok, c.raw),
           "kda_qk_norm_rope");
    return pack({qo, ko});
}

// (the eight above, d_q_out, d_k_out, need_weight_grads, dq, dk, dq_weight, dk_weight, given, workspace, stream)
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
    const NormRope A(a);
    const kda_rows gq = A.out_rows("d_q_out", tensor("d_q_out", a[8]), A.q),
                   gk = A.out_rows("d_k_out", tensor("d_k_out", a[9]), A.k);
    Call c(A.dev, a[17]);
    const bool given = truth(a[15]), weights = truth(a[10]);
    if (given && (a[11] == Py_None || a[12] == Py_None)) throw BadValue("grads must hold dq and dk");
    const at::Tensor dq = A.out(c, "dq", a[11], A.q), dk = A.out(c, "dk", a[12], A.k);
    at::Tensor dwq, dwk;
    if (given ? a[13] != Py_None : weights && A.wq) dwq = output(c, "dq_weight", a[13], A.wdt, {A.d});
    if (given ? a[14] != Py_None : weights && A.wk) dwk = output(c, "dk_weight", a[14], A.wdt, {A.d});
    const kda_rows oq = A.out_rows("dq", dq, A.q), ok = A.out_rows("dk", dk, A.k);
    const Scratch w(c, a[16], [&] { return kda_qk_norm_rope_bwd_workspace_size(A.T, A.Hq, A.Hk, A.d, A.rot); });
    c.done(kda_qk_norm_rope_bwd(&A.rq, &A.rk, A.wq, A.wk, A.wtype(), (const int32_t*)A.pos, (const float*)A.freq,
                                type_of(A.q), A.T, A.Hq, A.Hk, A.d, A.rot, A.eps, A.interleaved, &gq, &gk, &oq, &ok,
                                ptr(dwq), ptr(dwk), w.ptr, w.bytes, c.raw),
           "kda_qk_norm_rope_bwd");
    return pack({dq, dk, dwq, dwk});
}

// No C++ exception passes into Python: ValueError, KdaError, or RuntimeError from torch.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const BadValue& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Status& s) {
        PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", s.code, s.what) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, s.what);
        }
    } catch (const PythonError&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_memory ? g_memory : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* set_errors(PyObject*, PyObject* args) {   // (KdaError, torch.OutOfMemoryError)
    PyObject *error, *memory;
    if (!PyArg_ParseTuple(args, "OO", &error, &memory)) return nullptr;
    Py_XSETREF(g_error, Py_NewRef(error));
    Py_XSETREF(g_memory, Py_NewRef(memory));
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return PyMethodDef{name, (PyCFunction)(void (*)(void))&entry<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<linear_chunk_fwd, 11>("linear_chunk_fwd"),
    method<linear_chunk_bwd, 17>("linear_chunk_bwd"),
    method<linear_decode_step, 7>("linear_decode_step"),
    method<qk_norm_rope, 11>("qk_norm_rope"),
    method<qk_norm_rope_bwd, 18>("qk_norm_rope_bwd"),
    {"set_errors", set_errors, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&g_module); }
