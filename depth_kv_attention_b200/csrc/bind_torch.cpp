// Python binding of the paged-cache entry points on torch tensors: argument
// checks, output and workspace allocation, and the C call, in one step. A decode
// step calls these per layer on a few kilobytes; through ctypes the marshalling
// of their 40 arguments took 20 us a call, four times the launch.
//
// The functions take positional arguments only (the package's functions of the
// same names hold the signatures and documentation) and return the result, or a
// non-zero status code as an int. A wrong argument raises ValueError; torch's
// errors (an allocation that fails) come as torch's own types.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <stdexcept>
#include <string>

#include "../../include/moda.h"

namespace {

using at::Tensor;

[[noreturn]] void bad(const char* where, const char* what) { throw std::invalid_argument(std::string(where) + ": " + what); }

// A tensor argument; nullptr for None where that is allowed.
const Tensor* tensor(PyObject* o, const char* where, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad(where, "a tensor expected");
    return &THPVariable_Unpack(o);
}
long long integer(PyObject* o, const char* where) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        bad(where, "an integer expected");
    }
    return v;
}
int size32(int64_t v, const char* where) {
    if (v < 0 || v > 0x7fffffffLL) bad(where, "a size past 32 bits");
    return (int)v;
}
void* addr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

struct Cache {
    int N, B, Hq, Hkv, d, pages, page, blocks;
    moda_dtype dt;
};

// Shapes, types and places of what both operators share. `tok` [N, H, d]: the
// packed tokens (k, or q); `dense`: further tensors that have to be contiguous.
Cache check_cache(const char* where, const Tensor& tok, const Tensor& kp, const Tensor& vp, const Tensor* ks,
                  const Tensor* vs, const Tensor& table, const Tensor& cu, const Tensor& ctx, const Tensor* kd,
                  const Tensor* vd, std::initializer_list<const Tensor*> dense) {
    if (tok.dim() != 3 || kp.dim() != 4 || vp.dim() != 4 || table.dim() != 2 || cu.dim() != 1 || ctx.dim() != 1)
        bad(where, "packed tokens [N,H,d], pages [num_pages,Hkv,page_size,d], a block table [B,max_blocks], cu_q [B+1] and ctx_lens [B] expected");
    Cache c;
    c.N = size32(tok.size(0), where);
    c.Hq = size32(tok.size(1), where);
    c.d = size32(tok.size(2), where);
    c.pages = size32(kp.size(0), where);
    c.Hkv = size32(kp.size(1), where);
    c.page = size32(kp.size(2), where);
    c.B = size32(table.size(0), where);
    c.blocks = size32(table.size(1), where);
    if (kp.size(3) != c.d || vp.sizes() != kp.sizes() || cu.size(0) != c.B + 1LL || ctx.size(0) != c.B)
        bad(where, "shapes of pages, cu_q [B+1] or ctx_lens [B] do not match");
    if (table.scalar_type() != at::kInt || cu.scalar_type() != at::kInt || ctx.scalar_type() != at::kInt)
        bad(where, "int32 cu_q, ctx_lens and block_table expected");
    const auto type = tok.scalar_type();
    if (type == at::kBFloat16) c.dt = MODA_BF16;
    else if (type == at::kFloat) c.dt = MODA_F32;
    else bad(where, "bf16 or fp32 expected");
    const auto held = ks ? at::kChar : type;
    if (kp.scalar_type() != held || vp.scalar_type() != held)
        bad(where, ks ? "int8 pages expected" : "pages of the tokens' type expected");
    if (ks)
        for (const Tensor* t : {ks, vs})
            if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(0) != c.pages || t->size(1) != c.Hkv)
                bad(where, "fp32 scales [num_pages,Hkv] expected");
    if (!kd != !vd) bad(where, "kd and vd come together");
    if (kd && (kd->dim() != 4 || kd->size(0) != c.N || kd->size(2) != c.Hkv || kd->size(3) != c.d ||
               kd->sizes() != vd->sizes() || kd->scalar_type() != type || vd->scalar_type() != type))
        bad(where, "kd, vd [N,Ld,Hkv,d] of the tokens' type expected");
    if (!tok.is_cuda()) bad(where, "MoDA tensors must be CUDA tensors");
    const int dev = tok.get_device();
    auto place = [&](const Tensor* t) {
        if (t && (!t->is_cuda() || t->get_device() != dev || !t->is_contiguous()))
            bad(where, "contiguous tensors on one CUDA device expected");
    };
    for (const Tensor* t : {&kp, &vp, &table, &cu, &ctx, ks, vs, kd, vd}) place(t);
    for (const Tensor* t : dense) place(t);
    return c;
}

// Elements from token to token of t [N, H, d] with dense heads (a dimension of
// one element may carry any stride).
long long token_stride(const char* where, const Tensor& t, int dev) {
    if (!t.is_cuda() || t.get_device() != dev || (t.size(2) > 1 && t.stride(2) != 1) ||
        (t.size(1) > 1 && t.stride(1) != t.size(2)))
        bad(where, "dense heads on one device expected (any stride from token to token)");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

// The stream a call runs on: `o` is its handle, or None for the current one.
c10::cuda::CUDAStream stream_of(PyObject* o, int dev, const char* where) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
    return c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(integer(o, where)), (c10::DeviceIndex)dev);
}

template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {  // as torch's own functions: torch.OutOfMemoryError and the like
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// (q, k, v, k_pages, v_pages, k_scale, v_scale, block_table, cu_q, ctx_lens, rope, interleaved, q_out, kd, vd, slot, stream)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 17) throw std::invalid_argument("paged_append: 17 arguments expected");
        const bool q8 = a[5] != Py_None;
        const char* where = q8 ? "moda_paged_append_q8" : "moda_paged_append";
        const Tensor *q = tensor(a[0], where, true), *k = tensor(a[1], where), *v = tensor(a[2], where);
        const Tensor *kp = tensor(a[3], where), *vp = tensor(a[4], where);
        const Tensor *ks = q8 ? tensor(a[5], where) : nullptr, *vs = q8 ? tensor(a[6], where) : nullptr;
        const Tensor *table = tensor(a[7], where), *cu = tensor(a[8], where), *ctx = tensor(a[9], where);
        const Tensor *rope = tensor(a[10], where, true), *qo = tensor(a[12], where, true);
        const Tensor *kd = tensor(a[13], where, true), *vd = tensor(a[14], where, true);
        const int inter = PyObject_IsTrue(a[11]);
        if (inter < 0) {
            PyErr_Clear();
            bad(where, "a truth value expected as interleaved");
        }
        const long long slot = integer(a[15], where);
        if (slot < 0 || slot > 0x7fffffffLL) bad(where, "slot must lie in [0, slots of kd)");
        Cache c = check_cache(where, *k, *kp, *vp, ks, vs, *table, *cu, *ctx, kd, vd, {rope, qo});
        if (c.Hq != c.Hkv || v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type())
            bad(where, "k, v [N,Hkv,d] of one type expected");
        if (q) {
            if (q->dim() != 3 || q->size(0) != c.N || q->size(2) != c.d || q->scalar_type() != k->scalar_type())
                bad(where, "q [N,Hq,d] of the type of k expected");
            c.Hq = size32(q->size(1), where);
            if (qo && (qo->sizes() != q->sizes() || qo->scalar_type() != q->scalar_type())) bad(where, "q_out like q expected");
        } else if (qo) {
            bad(where, "q_out without q");
        }
        if (rope && (rope->scalar_type() != at::kFloat || rope->dim() != 2)) bad(where, "fp32 rope [positions, rot_dim] expected");
        const int dev = k->get_device();
        const long long sq = q ? token_stride(where, *q, dev) : 0, sk = token_stride(where, *k, dev), sv = token_stride(where, *v, dev);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[16], dev, where);
        const c10::cuda::CUDAStreamGuard on(stream);  // what is made here comes from the pool of the stream that writes it
        Tensor made;
        if (q && !qo) {
            made = at::empty({c.N, c.Hq, c.d}, q->options());
            qo = &made;
        }
        moda_status st = MODA_OK;
        if (c.N > 0) {
            void* s = stream.stream();
            const int rl = rope ? size32(rope->size(0), where) : 0, rot = rope ? size32(rope->size(1), where) : 0;
            const int Ld = kd ? size32(kd->size(1), where) : 0;
            auto i32 = [](const Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); };
            st = q8 ? moda_paged_append_q8(addr(q), addr(k), addr(v), sq, sk, sv, static_cast<const float*>(addr(rope)), rl, rot,
                                           inter, i32(cu), i32(ctx), i32(table), c.N, c.B, c.Hq, c.Hkv, c.d, c.pages, c.page,
                                           c.blocks, c.dt, static_cast<int8_t*>(addr(kp)), static_cast<int8_t*>(addr(vp)),
                                           static_cast<float*>(addr(ks)), static_cast<float*>(addr(vs)), addr(qo), addr(kd),
                                           addr(vd), Ld, (int)slot, s)
                    : moda_paged_append(addr(q), addr(k), addr(v), sq, sk, sv, static_cast<const float*>(addr(rope)), rl, rot, inter,
                                        i32(cu), i32(ctx), i32(table), c.N, c.B, c.Hq, c.Hkv, c.d, c.pages, c.page, c.blocks, c.dt,
                                        addr(kp), addr(vp), addr(qo), addr(kd), addr(vd), Ld, (int)slot, s);
        }
        if (st != MODA_OK) return PyLong_FromLong(st);
        if (made.defined()) return THPVariable_Wrap(std::move(made));
        PyObject* res = q ? a[12] : Py_None;
        Py_INCREF(res);
        return res;
    });
}

// (q, k_pages, v_pages, k_scale, v_scale, block_table, cu_q, ctx_lens, max_q, kd, vd, Ld, scale, out, lse, workspace, impl, stream)
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 18) throw std::invalid_argument("fwd_paged: 18 arguments expected");
        const bool q8 = a[3] != Py_None;
        const char* where = q8 ? "moda_fwd_paged_q8" : "moda_fwd_paged";
        const Tensor *q = tensor(a[0], where), *kp = tensor(a[1], where), *vp = tensor(a[2], where);
        const Tensor *ks = q8 ? tensor(a[3], where) : nullptr, *vs = q8 ? tensor(a[4], where) : nullptr;
        const Tensor *table = tensor(a[5], where), *cu = tensor(a[6], where), *ctx = tensor(a[7], where);
        const Tensor *kd = tensor(a[9], where, true), *vd = tensor(a[10], where, true);
        const Tensor *out = tensor(a[13], where, true), *lse = tensor(a[14], where, true), *ws = tensor(a[15], where, true);
        const Cache c = check_cache(where, *q, *kp, *vp, ks, vs, *table, *cu, *ctx, kd, vd, {q, out, lse, ws});
        const int max_q = size32(integer(a[8], where), where);
        const int cap = kd ? size32(kd->size(1), where) : 0;
        const long long Ld = a[11] == Py_None ? cap : integer(a[11], where);
        if (Ld < 0 || Ld > cap) bad(where, "Ld must lie in [0, slots of kd]");
        double scale = 1.0 / std::sqrt((double)c.d);
        if (a[12] != Py_None) {
            scale = PyFloat_AsDouble(a[12]);
            if (scale == -1.0 && PyErr_Occurred()) {
                PyErr_Clear();
                bad(where, "a number expected as scale");
            }
        }
        if (out && (out->sizes() != q->sizes() || out->scalar_type() != q->scalar_type())) bad(where, "out like q expected");
        if (lse && (lse->dim() != 2 || lse->size(0) != c.N || lse->size(1) != c.Hq || lse->scalar_type() != at::kFloat))
            bad(where, "fp32 lse [N,Hq] expected");
        const int dev = q->get_device();
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[17], dev, where);
        const c10::cuda::CUDAStreamGuard on(stream);  // what is made here comes from the pool of the stream that writes it
        Tensor made_out, made_lse, made_ws;
        if (!out) {
            made_out = at::empty(q->sizes(), q->options());
            out = &made_out;
        }
        if (!lse) {
            made_lse = at::empty({c.N, c.Hq}, q->options().dtype(at::kFloat));
            lse = &made_lse;
        }
        moda_status st = MODA_OK;
        if (c.N > 0) {
            const moda_impl impl = (moda_impl)integer(a[16], where);
            auto make_ws = [&](int copy) {
                const size_t need = moda_fwd_paged_workspace_bytes_ex(c.N, c.B, max_q, c.Hq, c.Hkv, c.d, c.pages, c.page,
                                                                      c.blocks, c.dt, copy, impl);
                if (!need) return;
                made_ws = at::empty({(int64_t)need}, q->options().dtype(at::kByte));
                ws = &made_ws;
            };
            if (!ws) {
                try {
                    make_ws(q8);
                } catch (const c10::OutOfMemoryError&) {
                    if (!q8) throw;
                    make_ws(0);  // without the bf16 copy of 8-bit pages
                }
            }
            const size_t have = ws ? ws->nbytes() : 0;
            void* s = stream.stream();
            auto i32 = [](const Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); };
            const void *kda = Ld ? addr(kd) : nullptr, *vda = Ld ? addr(vd) : nullptr;
            float* lp = static_cast<float*>(addr(lse));
            st = q8 ? moda_fwd_paged_q8_ex(addr(q), static_cast<const int8_t*>(addr(kp)), static_cast<const int8_t*>(addr(vp)),
                                           static_cast<const float*>(addr(ks)), static_cast<const float*>(addr(vs)), kda, vda,
                                           i32(cu), i32(ctx), i32(table), c.N, c.B, max_q, c.Hq, c.Hkv, c.d, (int)Ld, cap,
                                           c.pages, c.page, c.blocks, c.dt, (float)scale, addr(out), lp, addr(ws), have, s,
                                           impl)
                    : moda_fwd_paged(addr(q), addr(kp), addr(vp), kda, vda, i32(cu), i32(ctx), i32(table), c.N, c.B, max_q, c.Hq,
                                     c.Hkv, c.d, (int)Ld, cap, c.pages, c.page, c.blocks, c.dt, (float)scale, addr(out), lp,
                                     addr(ws), have, s, impl);
        }
        if (st != MODA_OK) return PyLong_FromLong(st);
        PyObject* res = PyTuple_New(2);
        if (!res) return nullptr;
        for (int i = 0; i < 2; ++i) {
            Tensor& made = i ? made_lse : made_out;
            PyObject* o;
            if (made.defined()) {
                o = THPVariable_Wrap(std::move(made));
            } else {
                o = a[13 + i];
                Py_INCREF(o);
            }
            PyTuple_SET_ITEM(res, i, o);
        }
        return res;
    });
}

PyMethodDef kMethods[] = {
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_append)), METH_FASTCALL, nullptr},
    {"fwd_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fwd_paged)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_moda_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__moda_torch(void) {
    PyObject* m = PyModule_Create(&kModule);
    // the torch that this was compiled against: tensors of another one may be laid out differently
    if (m && PyModule_AddStringConstant(m, "torch_version", MODA_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
