// Argument checks of the int8-cache, rotary, windowed and tree bindings, in native code.
//
// pkv.py's wrappers for these calls hand their tensors here: shapes, types, devices and layouts are checked,
// raw pointers taken and the C entry point called; the status goes back to the wrapper.  A decode step's calls run
// for a few microseconds on the GPU, and checking their ten or so tensors attribute by attribute in Python takes
// longer than that (store of 64 rows: 10.4 us a call with the checks in Python, 3.4 us of them the C call).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>

#include "../../include/pkv.h"

namespace {

// A refused argument: the Python error is set.
struct Refused {
};

[[noreturn]] void refuse(const char *what, const char *why)
{
    PyErr_Format(PyExc_ValueError, "%s %s", what, why);
    throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(name, "must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(name, "must be a CUDA tensor");
    return t;
}

// The device of a call: that of its first tensor, which has to be the current one (the library launches there).
struct Device {
    int index;
    explicit Device(PyObject *first, const char *name)
    {
        index = tensor(first, name).device().index();
        if (index != c10::cuda::current_device()) refuse(name, "is not on the current CUDA device");
    }

    const at::Tensor &typed(PyObject *o, at::ScalarType type, int dims, const char *name) const
    {
        const at::Tensor &t = tensor(o, name);
        if (t.scalar_type() != type) {
            PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, c10::toString(type),
                         c10::toString(t.scalar_type()));
            throw Refused();
        }
        if (t.device().index() != index) refuse(name, "is on another device than the call's other tensors");
        if (dims >= 0 && t.dim() != dims) {
            PyErr_Format(PyExc_ValueError, "%s must have %d dims, got %d", name, dims, int(t.dim()));
            throw Refused();
        }
        return t;
    }

    const at::Tensor &dense(PyObject *o, at::ScalarType type, int dims, const char *name) const
    {
        const at::Tensor &t = typed(o, type, dims, name);
        if (!t.is_contiguous()) refuse(name, "must be contiguous");
        return t;
    }

    int32_t *ints(PyObject *o, int dims, int64_t count, const char *name, const char *what) const
    {
        const at::Tensor &t = dense(o, at::kInt, dims, name);
        if (count >= 0 && t.numel() != count) refuse(what, "shape mismatch");
        return static_cast<int32_t *>(t.data_ptr());
    }

    int32_t *err(PyObject *o) const { return o == Py_None ? nullptr : ints(o, -1, -1, "err_word", "err_word"); }

    pkv_stream_t stream(PyObject *o) const
    {
        if (o == Py_None)
            return reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream());
        PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw Refused();
        void *p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw Refused();
        return static_cast<pkv_stream_t>(p);
    }
};

// bf16 rows [T][H, D], dense within a row, any distance between rows.
struct Rows {
    uint16_t *p;
    int64_t stride, T, H, D;
    Rows(const Device &dev, PyObject *o, const char *name)
    {
        const at::Tensor &t = dev.typed(o, at::kBFloat16, 3, name);
        T = t.size(0);
        H = t.size(1);
        D = t.size(2);
        if ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D)) refuse(name, "needs dense heads within a row");
        stride = T > 1 ? t.stride(0) : H * D;
        p = static_cast<uint16_t *>(t.data_ptr());
    }
    bool same(const Rows &o) const { return T == o.T && H == o.H && D == o.D; }
};

struct I8Cache {
    int8_t *k, *v;
    float *scales;
    int64_t NB, bs, H, D;
    I8Cache(const Device &dev, PyObject *ko, PyObject *vo, PyObject *so, const char *what)
    {
        const at::Tensor &kt = dev.dense(ko, at::kChar, 4, "k_cache");
        const at::Tensor &vt = dev.dense(vo, at::kChar, 4, "v_cache");
        const at::Tensor &st = dev.dense(so, at::kFloat, 4, "scales");
        NB = kt.size(0);
        bs = kt.size(1);
        H = kt.size(2);
        D = kt.size(3);
        if (vt.sizes() != kt.sizes() || st.size(0) != NB || st.size(1) != bs / PKV_I8_BLOCK || st.size(2) != H ||
            st.size(3) != 2)
            refuse(what, "shape mismatch");
        k = static_cast<int8_t *>(kt.data_ptr());
        v = static_cast<int8_t *>(vt.data_ptr());
        scales = static_cast<float *>(st.data_ptr());
    }
};

long integer(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

// A size or count as the C entry points take it; one that does not fit is out of their bounds anyway.
int32_t i32(int64_t v, const char *what)
{
    if (v < INT32_MIN || v > INT32_MAX) refuse(what, "is out of range");
    return int32_t(v);
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}

int truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v;
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&call)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
        return nullptr;
    }
    try {
        return PyLong_FromLong(long(call()));
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (k, v, k_cache, v_cache, scales, block_tables, context_lens, cu_seqlens, new_per_seq, err_word, stream)
PyObject *kv_store_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const char *what = "kv_store_i8:";
        const Device dev(a[0], "k");
        const Rows k(dev, a[0], "k"), v(dev, a[1], "v");
        const I8Cache c(dev, a[2], a[3], a[4], what);
        const at::Tensor &bt = dev.dense(a[5], at::kInt, 2, "block_tables");
        const int64_t B = bt.size(0);
        const long per = integer(a[8]);
        const int32_t *lens = dev.ints(a[6], -1, B, "context_lens", what);
        if (!k.same(v) || k.H != c.H || k.D != c.D || (a[7] == Py_None && per <= 0)) refuse(what, "shape mismatch");
        const int32_t *cu = a[7] == Py_None ? nullptr : dev.ints(a[7], -1, B + 1, "cu_seqlens", what);
        return pkv_kv_store_i8(k.p, v.p, k.stride, v.stride, static_cast<const int32_t *>(bt.data_ptr()),
                               i32(bt.size(1), what), cu, lens, i32(B, what), i32(k.T, what), i32(per, "new_per_seq"),
                               c.k, c.v, c.scales, i32(c.NB, what), i32(c.bs, what), i32(c.H, what), i32(c.D, what),
                               dev.err(a[9]), dev.stream(a[10]));
    });
}

// What the two attention calls share: q, the cache, tables, lengths, out and workspace, checked.
struct Attend {
    Device dev;
    I8Cache c;
    const at::Tensor &q, &bt, &out, &ws;
    int64_t rows, Hq, B, mb;
    int32_t mx;
    Attend(PyObject *qo, PyObject *ko, PyObject *vo, PyObject *so, PyObject *bto, PyObject *outo, PyObject *wso,
           PyObject *mxo, const char *what)
        : dev(qo, "q"), c(dev, ko, vo, so, what), q(dev.dense(qo, at::kBFloat16, 3, "q")),
          bt(dev.dense(bto, at::kInt, 2, "block_tables")), out(dev.dense(outo, at::kBFloat16, 3, "out")),
          ws(dev.dense(wso, at::kByte, -1, "workspace"))
    {
        rows = q.size(0);
        Hq = q.size(1);
        B = bt.size(0);
        mb = bt.size(1);
        if (q.size(2) != c.D || out.sizes() != q.sizes()) refuse(what, "shape mismatch");
        // lengths beyond the table are rejected anyway
        mx = mxo == Py_None ? int32_t(std::min<int64_t>(mb * c.bs, INT32_MAX)) : i32(integer(mxo), "max_context_len");
    }
};

// (q, k_cache, v_cache, scales, block_tables, context_lens, scale, out, workspace, max_context_len, num_workers,
//  err_word, stream)
PyObject *paged_decode_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const char *what = "paged_decode_i8:";
        const Attend t(a[0], a[1], a[2], a[3], a[4], a[7], a[8], a[9], what);
        const int32_t *lens = t.dev.ints(a[5], -1, t.B, "context_lens", what);
        if (t.rows != t.B) refuse(what, "shape mismatch");
        return pkv_paged_decode_i8(static_cast<const uint16_t *>(t.q.data_ptr()), t.c.k, t.c.v, t.c.scales,
                                   static_cast<const int32_t *>(t.bt.data_ptr()), i32(t.mb, what), lens,
                                   i32(t.B, what), i32(t.Hq, what), i32(t.c.H, what), i32(t.c.D, what),
                                   i32(t.c.bs, what), i32(t.c.NB, what), t.mx, float(real(a[6])),
                                   static_cast<uint16_t *>(t.out.data_ptr()), t.ws.data_ptr(), size_t(t.ws.numel()),
                                   i32(integer(a[10]), "num_workers"), t.dev.err(a[11]), t.dev.stream(a[12]));
    });
}

// (q, k_cache, v_cache, scales, block_tables, cu_seqlens_q, context_lens, scale, out, workspace, max_context_len,
//  num_workers, err_word, stream, new_per_seq)
PyObject *paged_attention_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 15, [&] {
        const char *what = "paged_attention_i8:";
        const Attend t(a[0], a[1], a[2], a[3], a[4], a[8], a[9], a[10], what);
        const int32_t *lens = t.dev.ints(a[6], -1, t.B, "context_lens", what);
        const long per = integer(a[14]);
        if (a[5] == Py_None && per <= 0) refuse(what, "shape mismatch");
        const int32_t *cu = a[5] == Py_None ? nullptr : t.dev.ints(a[5], -1, t.B + 1, "cu_seqlens_q", what);
        return pkv_paged_attention_i8(static_cast<const uint16_t *>(t.q.data_ptr()), t.c.k, t.c.v, t.c.scales,
                                      static_cast<const int32_t *>(t.bt.data_ptr()), i32(t.mb, what), cu, lens,
                                      i32(t.B, what), i32(t.rows, what), i32(t.Hq, what), i32(t.c.H, what),
                                      i32(t.c.D, what), i32(t.c.bs, what), i32(t.c.NB, what), t.mx, float(real(a[7])),
                                      static_cast<uint16_t *>(t.out.data_ptr()), i32(per, "new_per_seq"),
                                      t.ws.data_ptr(), size_t(t.ws.numel()), i32(integer(a[11]), "num_workers"),
                                      t.dev.err(a[12]), t.dev.stream(a[13]));
    });
}

// (k_cache, v_cache, scales, pairs, err_word, stream)
PyObject *copy_blocks_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const char *what = "copy_blocks_i8:";
        const Device dev(a[0], "k_cache");
        const I8Cache c(dev, a[0], a[1], a[2], what);
        const at::Tensor &pairs = dev.dense(a[3], at::kInt, 2, "pairs");
        if (pairs.size(1) != 2) refuse(what, "shape mismatch");
        return pkv_copy_blocks_i8(c.k, c.v, c.scales, static_cast<const int32_t *>(pairs.data_ptr()),
                                  i32(pairs.size(0), what), i32(c.NB, what), i32(c.bs, what), i32(c.H, what),
                                  i32(c.D, what), dev.err(a[4]), dev.stream(a[5]));
    });
}

// What the two rotary calls share: rows of q, k and q_out, positions and frequencies.
struct Rotary {
    Device dev;
    Rows q, k, q_out;
    const int32_t *pos, *freq_axis;
    const float *inv;
    int32_t axes, half;
    Rotary(PyObject *qo, PyObject *ko, PyObject *po, PyObject *io, PyObject *oo, PyObject *ao, const char *what)
        : dev(qo, "q"), q(dev, qo, "q"), k(dev, ko, "k"), q_out(dev, oo, "q_out")
    {
        const at::Tensor &p = dev.dense(po, at::kInt, -1, "positions");
        const at::Tensor &f = dev.dense(io, at::kFloat, 1, "inv_freq");
        half = i32(f.numel(), what);
        const bool flat = p.dim() == 1;
        if ((!flat && p.dim() != 2) || p.size(flat ? 0 : 1) != q.T || k.T != q.T || k.D != q.D || !q.same(q_out) ||
            half > (1 << 20))
            refuse(what, "shape mismatch");
        axes = flat ? 1 : i32(p.size(0), what);
        pos = static_cast<const int32_t *>(p.data_ptr());
        inv = static_cast<const float *>(f.data_ptr());
        freq_axis = ao == Py_None ? nullptr : dev.ints(ao, 1, half, "freq_axis", what);
    }
};

// (q, k, positions, inv_freq, q_out, k_out, freq_axis, interleaved, err_word, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const char *what = "rope:";
        const Rotary r(a[0], a[1], a[2], a[3], a[4], a[6], what);
        const Rows k_out(r.dev, a[5], "k_out");
        if (!k_out.same(r.k)) refuse(what, "shape mismatch");
        return pkv_rope(r.q.p, r.q.stride, r.k.p, r.k.stride, r.pos, r.axes, r.inv, r.freq_axis, i32(r.q.T, what),
                        i32(r.q.H, what), i32(r.k.H, what), i32(r.q.D, what), 2 * r.half, truth(a[7]),
                        r.q_out.p, r.q_out.stride, k_out.p, k_out.stride, r.dev.err(a[8]), r.dev.stream(a[9]));
    });
}

// (q, k, v, positions, inv_freq, slot_mapping, q_out, k_cache, v_cache, freq_axis, interleaved, err_word, stream)
PyObject *rope_store(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const char *what = "rope_store:";
        const Rotary r(a[0], a[1], a[3], a[4], a[6], a[9], what);
        const Rows v(r.dev, a[2], "v");
        const int32_t *slots = r.dev.ints(a[5], -1, r.q.T, "slot_mapping", what);
        const at::Tensor &kc = r.dev.dense(a[7], at::kBFloat16, 4, "k_cache");
        const at::Tensor &vc = r.dev.dense(a[8], at::kBFloat16, 4, "v_cache");
        if (!v.same(r.k) || kc.size(2) != r.k.H || kc.size(3) != r.k.D || vc.sizes() != kc.sizes())
            refuse(what, "shape mismatch");
        return pkv_rope_store(r.q.p, r.q.stride, r.k.p, r.k.stride, v.p, v.stride, r.pos, r.axes, r.inv, r.freq_axis,
                              slots, i32(r.q.T, what), i32(r.q.H, what), i32(r.k.H, what), i32(r.q.D, what),
                              2 * r.half, truth(a[10]), r.q_out.p, r.q_out.stride,
                              static_cast<uint16_t *>(kc.data_ptr()), static_cast<uint16_t *>(vc.data_ptr()),
                              i32(kc.size(0), what), i32(kc.size(1), what), r.dev.err(a[11]), r.dev.stream(a[12]));
    });
}

// A float32 [head_dim] weight, or None.
const float *weight(const Device &dev, PyObject *o, int64_t D, const char *name, const char *what)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = dev.dense(o, at::kFloat, 1, name);
    if (t.numel() != D) refuse(what, "shape mismatch");
    return static_cast<const float *>(t.data_ptr());
}

// (q, k, q_weight, k_weight, eps, positions, inv_freq, q_out, k_out, freq_axis, interleaved, err_word, stream)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const char *what = "qk_norm_rope:";
        const Rotary r(a[0], a[1], a[5], a[6], a[7], a[9], what);
        const Rows k_out(r.dev, a[8], "k_out");
        if (!k_out.same(r.k)) refuse(what, "shape mismatch");
        return pkv_qk_norm_rope(r.q.p, r.q.stride, r.k.p, r.k.stride, weight(r.dev, a[2], r.q.D, "q_weight", what),
                                weight(r.dev, a[3], r.q.D, "k_weight", what), float(real(a[4])), r.pos, r.axes, r.inv,
                                r.freq_axis, i32(r.q.T, what), i32(r.q.H, what), i32(r.k.H, what), i32(r.q.D, what),
                                2 * r.half, truth(a[10]), r.q_out.p, r.q_out.stride, k_out.p, k_out.stride,
                                r.dev.err(a[11]), r.dev.stream(a[12]));
    });
}

// (q, k, v, q_weight, k_weight, eps, positions, inv_freq, slot_mapping, q_out, k_cache, v_cache, freq_axis,
//  interleaved, err_word, stream)
PyObject *qk_norm_rope_store(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 16, [&] {
        const char *what = "qk_norm_rope_store:";
        const Rotary r(a[0], a[1], a[6], a[7], a[9], a[12], what);
        const Rows v(r.dev, a[2], "v");
        const int32_t *slots = r.dev.ints(a[8], -1, r.q.T, "slot_mapping", what);
        const at::Tensor &kc = r.dev.dense(a[10], at::kBFloat16, 4, "k_cache");
        const at::Tensor &vc = r.dev.dense(a[11], at::kBFloat16, 4, "v_cache");
        if (!v.same(r.k) || kc.size(2) != r.k.H || kc.size(3) != r.k.D || vc.sizes() != kc.sizes())
            refuse(what, "shape mismatch");
        return pkv_qk_norm_rope_store(
            r.q.p, r.q.stride, r.k.p, r.k.stride, v.p, v.stride, weight(r.dev, a[3], r.q.D, "q_weight", what),
            weight(r.dev, a[4], r.q.D, "k_weight", what), float(real(a[5])), r.pos, r.axes, r.inv, r.freq_axis, slots,
            i32(r.q.T, what), i32(r.q.H, what), i32(r.k.H, what), i32(r.q.D, what), 2 * r.half, truth(a[13]),
            r.q_out.p, r.q_out.stride, static_cast<uint16_t *>(kc.data_ptr()), static_cast<uint16_t *>(vc.data_ptr()),
            i32(kc.size(0), what), i32(kc.size(1), what), r.dev.err(a[14]), r.dev.stream(a[15]));
    });
}

// A cache of any type: bf16 (scales None), E4M3 (float32 scales [kv heads] of K and of V) or int8 (scales, None).
struct AnyCache {
    at::ScalarType type;
    const void *k, *v;
    const float *s0 = nullptr, *s1 = nullptr;
    int64_t NB, bs, H, D;
    AnyCache(const Device &dev, PyObject *ko, PyObject *vo, PyObject *so, PyObject *to, const char *what)
    {
        type = so == Py_None ? at::kBFloat16 : to == Py_None ? at::kChar : at::kByte;
        const at::Tensor &kt = dev.dense(ko, type, 4, "k_cache");
        const at::Tensor &vt = dev.dense(vo, type, 4, "v_cache");
        NB = kt.size(0);
        bs = kt.size(1);
        H = kt.size(2);
        D = kt.size(3);
        if (vt.sizes() != kt.sizes()) refuse(what, "shape mismatch");
        k = kt.data_ptr();
        v = vt.data_ptr();
        if (type == at::kChar) {
            const at::Tensor &st = dev.dense(so, at::kFloat, 4, "scales");
            if (st.size(0) != NB || st.size(1) != bs / PKV_I8_BLOCK || st.size(2) != H || st.size(3) != 2)
                refuse(what, "shape mismatch");
            s0 = static_cast<const float *>(st.data_ptr());
        } else if (type == at::kByte) {
            s0 = weight(dev, so, H, "k_scale", what);
            s1 = weight(dev, to, H, "v_scale", what);
        }
    }
    template <typename T>
    const T *keys() const { return static_cast<const T *>(k); }
    template <typename T>
    const T *values() const { return static_cast<const T *>(v); }
};

// What the windowed and tree calls share.
struct MaskedAttend {
    Device dev;
    AnyCache c;
    const at::Tensor &q, &bt, &out, &ws;
    const int32_t *tables;
    const uint16_t *qp;
    uint16_t *outp;
    int64_t rows, Hq, B, mb;
    int32_t mx;
    MaskedAttend(PyObject *qo, PyObject *ko, PyObject *vo, PyObject *so, PyObject *to, PyObject *bto, PyObject *outo,
                 PyObject *wso, PyObject *mxo, const char *what)
        : dev(qo, "q"), c(dev, ko, vo, so, to, what), q(dev.dense(qo, at::kBFloat16, 3, "q")),
          bt(dev.dense(bto, at::kInt, 2, "block_tables")), out(dev.dense(outo, at::kBFloat16, 3, "out")),
          ws(dev.dense(wso, at::kByte, -1, "workspace"))
    {
        rows = q.size(0);
        Hq = q.size(1);
        B = bt.size(0);
        mb = bt.size(1);
        if (q.size(2) != c.D || out.sizes() != q.sizes()) refuse(what, "shape mismatch");
        // lengths beyond the table are rejected anyway, and those beyond 2^30 by the call
        mx = mxo == Py_None ? int32_t(std::min<int64_t>(mb * c.bs, 1 << 30)) : i32(integer(mxo), "max_context_len");
        tables = static_cast<const int32_t *>(bt.data_ptr());
        qp = static_cast<const uint16_t *>(q.data_ptr());
        outp = static_cast<uint16_t *>(out.data_ptr());
    }
};

// (q, k_cache, v_cache, scales or k_scale or None, v_scale or None, block_tables, context_lens, scale, window, sinks,
//  out, workspace, max_context_len, num_workers, err_word, stream)
PyObject *paged_decode_window(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 16, [&] {
        const char *what = "paged_decode_window:";
        const MaskedAttend t(a[0], a[1], a[2], a[3], a[4], a[5], a[10], a[11], a[12], what);
        const int32_t *lens = t.dev.ints(a[6], -1, t.B, "context_lens", what);
        if (t.rows != t.B) refuse(what, "shape mismatch");
        auto call = [&](auto fn, auto... cache) {
            return fn(t.qp, cache..., t.tables, i32(t.mb, what), lens, i32(t.B, what), i32(t.Hq, what),
                      i32(t.c.H, what), i32(t.c.D, what), i32(t.c.bs, what), i32(t.c.NB, what), t.mx,
                      float(real(a[7])), i32(integer(a[8]), "window"), i32(integer(a[9]), "sinks"), t.outp,
                      t.ws.data_ptr(), size_t(t.ws.numel()), i32(integer(a[13]), "num_workers"), t.dev.err(a[14]),
                      t.dev.stream(a[15]));
        };
        if (t.c.type == at::kChar)
            return call(pkv_paged_decode_window_i8, t.c.keys<int8_t>(), t.c.values<int8_t>(), t.c.s0);
        if (t.c.type == at::kByte)
            return call(pkv_paged_decode_window_fp8, t.c.keys<uint8_t>(), t.c.values<uint8_t>(), t.c.s0, t.c.s1);
        return call(pkv_paged_decode_window, t.c.keys<uint16_t>(), t.c.values<uint16_t>());
    });
}

// (q, k_cache, v_cache, scales or None, block_tables, cu_seqlens_q, context_lens, tree_mask or None, window, sinks,
//  scale, out, workspace, max_context_len, num_workers, err_word, stream, new_per_seq)
PyObject *paged_attention_mask(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 18, [&] {
        const bool tree = a[7] != Py_None;
        const char *what = tree ? "paged_attention_tree:" : "paged_attention_window:";
        const MaskedAttend t(a[0], a[1], a[2], a[3], Py_None, a[4], a[11], a[12], a[13], what);
        const int32_t *lens = t.dev.ints(a[6], -1, t.B, "context_lens", what);
        const long per = integer(a[17]);
        if (a[5] == Py_None && per <= 0) refuse(what, "shape mismatch");
        const int32_t *cu = a[5] == Py_None ? nullptr : t.dev.ints(a[5], -1, t.B + 1, "cu_seqlens_q", what);
        const int32_t *bits = nullptr;
        int64_t words = 0;
        if (tree) {
            const at::Tensor &m = t.dev.dense(a[7], at::kInt, 2, "tree_mask");
            if (m.size(0) != t.rows) refuse(what, "shape mismatch");
            bits = static_cast<const int32_t *>(m.data_ptr());
            words = m.size(1);
        }
        const int32_t m0 = tree ? 0 : i32(integer(a[8]), "window"), m1 = tree ? 0 : i32(integer(a[9]), "sinks");
        auto call = [&](auto fn, auto x, auto y, auto... cache) {
            return fn(t.qp, cache..., t.tables, i32(t.mb, what), cu, lens, i32(t.B, what), i32(t.rows, what),
                      i32(t.Hq, what), i32(t.c.H, what), i32(t.c.D, what), i32(t.c.bs, what), i32(t.c.NB, what), t.mx,
                      float(real(a[10])), x, y, t.outp, i32(per, "new_per_seq"), t.ws.data_ptr(),
                      size_t(t.ws.numel()), i32(integer(a[14]), "num_workers"), t.dev.err(a[15]),
                      t.dev.stream(a[16]));
        };
        const int8_t *k8 = t.c.keys<int8_t>(), *v8 = t.c.values<int8_t>();
        const uint16_t *k16 = t.c.keys<uint16_t>(), *v16 = t.c.values<uint16_t>();
        if (tree)
            return t.c.type == at::kChar
                       ? call(pkv_paged_attention_tree_i8, bits, i32(words, what), k8, v8, t.c.s0)
                       : call(pkv_paged_attention_tree, bits, i32(words, what), k16, v16);
        return t.c.type == at::kChar ? call(pkv_paged_attention_window_i8, m0, m1, k8, v8, t.c.s0)
                                     : call(pkv_paged_attention_window, m0, m1, k16, v16);
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(kv_store_i8),    FAST(paged_decode_i8), FAST(paged_attention_i8),
                         FAST(copy_blocks_i8), FAST(rope),            FAST(rope_store),
                         FAST(qk_norm_rope),   FAST(qk_norm_rope_store), FAST(paged_decode_window),
                         FAST(paged_attention_mask),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch this was compiled against (pkv.py refuses another one).
PyMODINIT_FUNC PyInit__pkv_torch(void)
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
