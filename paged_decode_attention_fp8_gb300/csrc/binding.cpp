// Native marshalling of the per-step operators for Python: rotary_apply,
// paged_kv_append, paged_cache_read, paged_gqa_decode_fp4,
// paged_cross_attention, paged_gqa_decode_shared and attention_merge.
//
// A decode step calls these once per layer and their kernels take a few
// microseconds, so the host's share counts: the same checks in Python with a
// ctypes call of 25-40 arguments took 16-33 us on the Grace host, here 3-6.
// Like the Python side, this file checks types, shapes and devices, makes the
// outputs that are not given, and hands raw pointers and the current stream to
// the C ABI; there is no computation here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "fp8mla.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_status_error = nullptr;  // FP8MLAError(status, where)

struct BadValue {
  std::string what;
};
[[noreturn]] void bad(std::string what) { throw BadValue{std::move(what)}; }

struct BadStatus {
  int status;
  const char* where;
};
void check(fp8mla_status_t s, const char* where) {
  if (s != FP8MLA_OK) throw BadStatus{static_cast<int>(s), where};
}

const Tensor* maybe(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& given(PyObject* o, const char* name) {
  const Tensor* t = maybe(o, name);
  if (t == nullptr) bad(std::string(name) + " must be a tensor");
  return *t;
}
struct PyFailure {};  // a Python exception is set
long long integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PyFailure{};
  return x;
}
int small(PyObject* o, const char* name) {
  const long long x = integer(o);
  if (x < INT32_MIN || x > INT32_MAX) bad(std::string(name) + " is out of range");
  return static_cast<int>(x);
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PyFailure{};
  return x != 0;
}

// The calls record nothing for autograd: a tensor whose gradient would be lost is refused.
void need_no_grad(std::initializer_list<const Tensor*> tensors) {
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : tensors)
    if (t != nullptr && t->requires_grad())
      bad("a tensor requires a gradient, which this call does not carry: detach it, or call under torch.no_grad()");
}
// After the call: autograd must not take what it saved of these tensors for their present values.
void written(std::initializer_list<const Tensor*> tensors) {
  for (const Tensor* t : tensors)
    if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

void* ptr(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
template <typename P>
P* ptr_as(const Tensor* t) {
  return static_cast<P*>(ptr(t));
}
fp8mla_stream_t stream_of(const c10::Device& d) {
  return reinterpret_cast<fp8mla_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}
// A dimension's stride; that of a single element means nothing and may be anything.
int64_t stride_of(const Tensor* t, int d) { return t == nullptr || t->size(d) <= 1 ? 0 : t->stride(d); }
int dim32(int64_t x, const char* name) {
  if (x > INT32_MAX) bad(std::string(name) + " is too large");
  return static_cast<int>(x);
}

// Rows [n, heads, head_dim] whose heads are contiguous.
void need_heads(const Tensor& x, const char* name, ScalarType type, const c10::Device& dev, int64_t n,
                int64_t head_dim = -1) {
  if (x.device() != dev || x.scalar_type() != type || x.dim() != 3 || x.size(0) != n)
    bad(std::string(name) + " must be " + c10::toString(type) + " [" + std::to_string(n) + ", heads, head_dim] on " +
        dev.str());
  if (head_dim >= 0 && x.size(2) != head_dim)
    bad(std::string(name) + " must have head_dim " + std::to_string(head_dim));
  if (x.size(2) > 1 && x.stride(2) != 1) bad(std::string(name) + ": the dims of a head must be contiguous");
}

// The same for an output.  (Rows that share memory in other ways than these are refused by the library.)
void need_heads_out(const Tensor& x, const char* name, c10::IntArrayRef shape, ScalarType type,
                    const c10::Device& dev) {
  need_heads(x, name, type, dev, shape[0], shape[2]);
  if (x.sizes() != shape) bad(std::string(name) + " must have its input's shape");
  if ((x.size(0) > 1 && x.stride(0) == 0) || (x.size(1) > 1 && x.stride(1) == 0))
    bad(std::string(name) + ": its rows overlap");
}

// int32 or int64 [n]; returns whether they are 64 bits wide.
int need_positions(const Tensor& p, const c10::Device& dev, int64_t n) {
  if (p.device() != dev || p.dim() != 1 || p.size(0) != n || !p.is_contiguous())
    bad("positions must be contiguous [" + std::to_string(n) + "] on " + dev.str());
  if (p.scalar_type() == ScalarType::Int) return 0;
  if (p.scalar_type() != ScalarType::Long) bad("positions must be int32 or int64");
  return 1;
}
void need_table(const Tensor& t, const c10::Device& dev) {
  if (t.device() != dev || t.scalar_type() != ScalarType::Float || t.dim() != 3 || t.size(2) != 2 ||
      !t.is_contiguous())
    bad("table must be contiguous float32 [n_positions, rot / 2, 2] on " + dev.str());
}
void need_int32(const Tensor& t, const char* name, const c10::Device& dev, int64_t n) {
  if (t.device() != dev || t.scalar_type() != ScalarType::Int || t.dim() != 1 || (n >= 0 && t.size(0) != n) ||
      !t.is_contiguous())
    bad(std::string(name) + " must be contiguous int32 [" + (n >= 0 ? std::to_string(n) : "n") + "] on " + dev.str());
}
void need_like(const Tensor& out, const char* name, c10::IntArrayRef shape, ScalarType type, const c10::Device& dev) {
  if (out.device() != dev || out.scalar_type() != type || out.sizes() != shape || !out.is_contiguous())
    bad(std::string(name) + " must be contiguous " + c10::toString(type) + " of the expected shape on " + dev.str());
}
Tensor make(c10::IntArrayRef shape, ScalarType type, const c10::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
PyObject* wrap(const Tensor* t, PyObject* given) {  // the caller's own object where there is one
  if (given != nullptr && given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(*t);
}

fp8mla_kv_dtype_t kv_code(const Tensor& cache, const Tensor* block_scales) {
  const ScalarType t = cache.scalar_type();
  if (block_scales != nullptr)  // block scales mark a 4-bit cache
    return t == ScalarType::Byte || t == ScalarType::Float4_e2m1fn_x2 ? FP8MLA_KV_E2M1 : FP8MLA_KV_OTHER;
  switch (t) {
    case ScalarType::Byte:
    case ScalarType::Float8_e4m3fn: return FP8MLA_KV_E4M3;
    case ScalarType::Float8_e4m3fnuz: return FP8MLA_KV_E4M3FNUZ;
    case ScalarType::Float8_e5m2:
    case ScalarType::Float8_e5m2fnuz: return FP8MLA_KV_E5M2;
    default: return FP8MLA_KV_OTHER;
  }
}

// A cache [num_blocks, h_kv, page, bytes a row]; the dense MLA form [num_pages, page, d] is one head.
struct CacheShape {
  int64_t blocks, h_kv, page, wide;
  bool operator==(const CacheShape& o) const {
    return blocks == o.blocks && h_kv == o.h_kv && page == o.page && wide == o.wide;
  }
};
CacheShape cache_shape(const Tensor& c, const char* name, const c10::Device& dev) {
  if (c.device() != dev || !c.is_contiguous() || (c.dim() != 3 && c.dim() != 4))
    bad(std::string(name) + " must be contiguous [num_blocks, h_kv, page, ...] on " + dev.str());
  if (c.dim() == 3) return {c.size(0), 1, c.size(1), c.size(2)};
  return {c.size(0), c.size(1), c.size(2), c.size(3)};
}
void need_scales(const char* name, const CacheShape& s, int64_t hd, fp8mla_kv_dtype_t code, const Tensor* scale,
                 const Tensor* rows, const Tensor* blocks, const c10::Device& dev) {
  const std::string who(name);
  if (code == FP8MLA_KV_E2M1) {
    if (scale == nullptr || blocks == nullptr || rows != nullptr)
      bad(who + ": a 4-bit cache takes one scale and its block scales");
    const ScalarType t = blocks->scalar_type();
    if (blocks->device() != dev || (t != ScalarType::Byte && t != ScalarType::Float8_e4m3fn) ||
        !blocks->is_contiguous() || blocks->dim() < 1 || blocks->size(-1) != hd / 16 ||
        blocks->numel() != s.blocks * s.h_kv * s.page * (hd / 16))
      bad(who + ": block scales must be contiguous E4M3 [num_blocks, h_kv, page, head_dim / 16]");
  } else if ((scale == nullptr) == (rows == nullptr)) {
    bad(who + ": give one scale or one per row");
  }
  if (scale != nullptr &&
      (scale->device() != dev || scale->scalar_type() != ScalarType::Float || scale->numel() != 1))
    bad(who + ": the scale must be one float32 on " + dev.str());
  if (rows != nullptr && (rows->device() != dev || rows->scalar_type() != ScalarType::Float ||
                          !rows->is_contiguous() || rows->dim() < 1 || rows->size(-1) != s.page ||
                          rows->numel() != s.blocks * s.h_kv * s.page))
    bad(who + ": row scales must be contiguous float32 [num_blocks, h_kv, page]");
}

// Runs f, with its exceptions turned into Python's.
template <typename F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const BadStatus& e) {
    PyObject* x = g_status_error == nullptr ? nullptr : PyObject_CallFunction(g_status_error, "is", e.status, e.where);
    if (x != nullptr) {
      PyErr_SetObject(g_status_error, x);
      Py_DECREF(x);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, e.where);
    }
  } catch (const PyFailure&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

bool count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
  return false;
}

// (q, k, positions, table, interleaved, rot_offset, inverse, q_out, k_out) -> (q_out, k_out)
PyObject* py_rotary_apply(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& q = given(a[0], "q");
    const Tensor* k = maybe(a[1], "k");
    const Tensor& pos = given(a[2], "positions");
    const Tensor& table = given(a[3], "table");
    const Tensor *q_out = maybe(a[7], "q_out"), *k_out = maybe(a[8], "k_out");
    need_no_grad({&q, k, &table, q_out, k_out});
    const ScalarType type = q.scalar_type();
    if (!q.is_cuda() || (type != ScalarType::BFloat16 && type != ScalarType::Half && type != ScalarType::Float))
      bad("q must be a CUDA tensor of bfloat16, float16 or float32");
    const c10::Device dev = q.device();
    const int64_t n = q.dim() > 0 ? q.size(0) : 0;
    need_heads(q, "q", type, dev, n);
    const int64_t hd = q.size(2);
    if (k != nullptr) need_heads(*k, "k", type, dev, n, hd);
    const int wide = need_positions(pos, dev, n);
    need_table(table, dev);
    if (k_out != nullptr && k == nullptr) bad("k_out without k");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor q_new, k_new;  // nothing else will have written their rows of padding
    int layout = truth(a[4]) ? FP8MLA_ROTARY_INTERLEAVED : 0;
    if (q_out == nullptr) layout |= FP8MLA_ROTARY_ZERO_Q;
    if (k_out == nullptr) layout |= FP8MLA_ROTARY_ZERO_K;
    if (q_out == nullptr) {
      q_new = make(q.sizes(), type, dev);
      q_out = &q_new;
    } else {
      need_heads_out(*q_out, "q_out", q.sizes(), type, dev);
    }
    if (k != nullptr) {
      if (k_out == nullptr) {
        k_new = make(k->sizes(), type, dev);
        k_out = &k_new;
      } else {
        need_heads_out(*k_out, "k_out", k->sizes(), type, dev);
      }
    }
    const fp8mla_dtype_t code =
        type == ScalarType::BFloat16 ? FP8MLA_BF16 : (type == ScalarType::Half ? FP8MLA_F16 : FP8MLA_F32);
    check(rotary_apply(q.data_ptr(), stride_of(&q, 0), stride_of(&q, 1), q_out->data_ptr(), stride_of(q_out, 0),
                       stride_of(q_out, 1), dim32(q.size(1), "h_q"), ptr(k), stride_of(k, 0), stride_of(k, 1),
                       ptr(k_out), stride_of(k_out, 0), stride_of(k_out, 1),
                       k == nullptr ? 0 : dim32(k->size(1), "h_k"), code, pos.data_ptr(), wide,
                       ptr_as<const float>(&table), table.size(0), dim32(n, "n_tokens"), dim32(hd, "head_dim"),
                       dim32(2 * table.size(1), "rot"), small(a[5], "rot_offset"), layout, truth(a[6]) ? 1 : 0,
                       stream_of(dev)),
          "rotary_apply");
    written({q_out, k_out});
    PyObject* qo = wrap(q_out, a[7]);
    PyObject* ko = k == nullptr ? Py_NewRef(Py_None) : wrap(k_out, a[8]);
    if (qo == nullptr || ko == nullptr) {
      Py_XDECREF(qo);
      Py_XDECREF(ko);
      return nullptr;
    }
    PyObject* r = PyTuple_Pack(2, qo, ko);
    Py_DECREF(qo);
    Py_DECREF(ko);
    return r;
  });
}

// (k, v, slot_mapping, k_cache, v_cache, positions, table, interleaved, rot_offset, k_scale, v_scale, k_row_scales,
//  v_row_scales, k_block_scales, v_block_scales, q, q_out) -> q_out or None
PyObject* py_kv_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& k0 = given(a[0], "k");
    const Tensor* v0 = maybe(a[1], "v");
    const Tensor& slots = given(a[2], "slot_mapping");
    const Tensor& kc = given(a[3], "k_cache");
    const Tensor* vc = maybe(a[4], "v_cache");
    const Tensor* pos = maybe(a[5], "positions");
    const Tensor* table = maybe(a[6], "table");
    const Tensor *ks = maybe(a[9], "k_scale"), *vs = maybe(a[10], "v_scale");
    const Tensor *kr = maybe(a[11], "k_row_scales"), *vr = maybe(a[12], "v_row_scales");
    const Tensor *kb = maybe(a[13], "k_block_scales"), *vb = maybe(a[14], "v_block_scales");
    const Tensor* q = maybe(a[15], "q");
    const Tensor* q_out = maybe(a[16], "q_out");
    need_no_grad({&k0, v0, &kc, vc, table, ks, vs, kr, vr, kb, vb, q, q_out});
    if (!k0.is_cuda() || k0.scalar_type() != ScalarType::BFloat16) bad("k must be a CUDA bf16 tensor");
    const c10::Device dev = k0.device();
    const Tensor k = k0.dim() == 2 ? k0.unsqueeze(1) : k0;
    const int64_t n = k.dim() > 0 ? k.size(0) : 0;
    need_heads(k, "k", ScalarType::BFloat16, dev, n);
    const int64_t h_kv = k.size(1), hd = k.size(2);
    const fp8mla_kv_dtype_t code = kv_code(kc, kb);
    const CacheShape shape = cache_shape(kc, "k_cache", dev);
    if (shape.h_kv != h_kv || shape.wide != (code == FP8MLA_KV_E2M1 ? hd / 2 : hd))
      bad("k and k_cache shapes disagree");
    need_scales("k", shape, hd, code, ks, kr, kb, dev);
    need_int32(slots, "slot_mapping", dev, n);
    if ((v0 == nullptr) != (vc == nullptr)) bad("v and v_cache go together");
    Tensor v;
    if (v0 != nullptr) {
      v = v0->dim() == 2 ? v0->unsqueeze(1) : *v0;
      need_heads(v, "v", ScalarType::BFloat16, dev, n, hd);
      if (v.size(1) != h_kv || !(cache_shape(*vc, "v_cache", dev) == shape) || kv_code(*vc, vb) != code)
        bad("v and v_cache must match k and k_cache");
      need_scales("v", shape, hd, code, vs, vr, vb, dev);
    } else if (vs != nullptr || vr != nullptr || vb != nullptr) {
      bad("scales for v without v");
    }
    int wide = 0;
    if (table == nullptr && pos != nullptr) bad("positions without a table");
    if (table != nullptr) {
      if (pos == nullptr) bad("a table needs positions");
      wide = need_positions(*pos, dev, n);
      need_table(*table, dev);
    }
    Tensor q_new;  // nothing else will have written its rows of padding
    const int layout =
        (truth(a[7]) ? FP8MLA_ROTARY_INTERLEAVED : 0) | (q_out == nullptr ? FP8MLA_ROTARY_ZERO_Q : 0);
    const c10::cuda::CUDAGuard guard(dev);
    if (q != nullptr) {
      if (table == nullptr) bad("q is rotated by a table: give one");
      need_heads(*q, "q", ScalarType::BFloat16, dev, n, hd);
      if (q_out == nullptr) {
        q_new = make(q->sizes(), ScalarType::BFloat16, dev);
        q_out = &q_new;
      } else {
        need_like(*q_out, "q_out", q->sizes(), ScalarType::BFloat16, dev);
      }
    } else if (q_out != nullptr) {
      bad("q_out without q");
    }
    const bool has_v = v0 != nullptr;
    const Tensor* pv = has_v ? &v : nullptr;
    check(paged_kv_append(k.data_ptr(), stride_of(&k, 0), stride_of(&k, 1), ptr(pv), stride_of(pv, 0),
                          stride_of(pv, 1), ptr_as<const int32_t>(&slots),
                          dim32(n, "n_tokens"), dim32(h_kv, "h_kv"), dim32(hd, "head_dim"), dim32(shape.page, "page"),
                          dim32(shape.blocks, "num_blocks"), code, kc.data_ptr(), ptr(vc), ptr_as<const float>(ks),
                          ptr_as<const float>(vs), ptr_as<float>(kr), ptr_as<float>(vr), ptr(kb), ptr(vb),
                          table != nullptr ? pos->data_ptr() : nullptr, wide, ptr_as<const float>(table),
                          table != nullptr ? table->size(0) : 0,
                          table != nullptr ? dim32(2 * table->size(1), "rot") : 0, small(a[8], "rot_offset"),
                          layout, ptr(q), stride_of(q, 0), stride_of(q, 1), ptr(q_out),
                          q != nullptr ? dim32(q->size(1), "h_q") : 0, stream_of(dev)),
          "paged_kv_append");
    written({&kc, vc, kr, vr, kb, vb, q_out});
    if (q == nullptr) return Py_NewRef(Py_None);
    return wrap(q_out, a[16]);
  });
}

// (cache, slots, scale, row_scales, block_scales, out) -> out
PyObject* py_cache_read(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& cache = given(a[0], "cache");
    const Tensor& slots = given(a[1], "slots");
    const Tensor *scale = maybe(a[2], "scale"), *rows = maybe(a[3], "row_scales");
    const Tensor* blocks = maybe(a[4], "block_scales");
    const Tensor* out = maybe(a[5], "out");
    need_no_grad({&cache, scale, rows, blocks, out});
    if (!cache.is_cuda()) bad("cache must be a CUDA tensor");
    const c10::Device dev = cache.device();
    const fp8mla_kv_dtype_t code = kv_code(cache, blocks);
    const CacheShape s = cache_shape(cache, "cache", dev);
    const int64_t hd = code == FP8MLA_KV_E2M1 ? 2 * s.wide : s.wide;
    need_scales("cache", s, hd, code, scale, rows, blocks, dev);
    need_int32(slots, "slots", dev, -1);
    const int64_t n = slots.size(0);
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t shape[3] = {n, s.h_kv, hd};
    Tensor made;
    if (out == nullptr) {
      made = make(shape, ScalarType::BFloat16, dev);
      out = &made;
    } else {
      need_like(*out, "out", shape, ScalarType::BFloat16, dev);
    }
    check(paged_cache_read(cache.data_ptr(), code, ptr_as<const float>(scale), ptr_as<const float>(rows), ptr(blocks),
                           ptr_as<const int32_t>(&slots), dim32(n, "n"), dim32(s.h_kv, "h_kv"), dim32(hd, "head_dim"),
                           dim32(s.page, "page"), dim32(s.blocks, "num_blocks"), out->data_ptr(), stream_of(dev)),
          "paged_cache_read");
    written({out});
    return wrap(out, a[5]);
  });
}

// (q, k_cache, v_cache, k_block_scales, v_block_scales, block_table, seqlens, k_scale, v_scale, softmax_scale,
//  spec_mask, window, sinks, num_splits, out, lse, workspace) -> (out, lse)
PyObject* py_decode_fp4(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& q = given(a[0], "q");
    const Tensor &kc = given(a[1], "k_cache"), &vc = given(a[2], "v_cache");
    const Tensor *kb = maybe(a[3], "k_block_scales"), *vb = maybe(a[4], "v_block_scales");
    const Tensor& bt = given(a[5], "block_table");
    const Tensor& sl = given(a[6], "seqlens");
    const Tensor *ks = maybe(a[7], "k_scale"), *vs = maybe(a[8], "v_scale");
    const Tensor *mask = maybe(a[10], "spec_mask"), *sinks = maybe(a[12], "sinks");
    const Tensor *out = maybe(a[14], "out"), *lse = maybe(a[15], "lse"), *ws = maybe(a[16], "workspace");
    need_no_grad({&q, &kc, &vc, kb, vb, ks, vs, sinks, out, lse});
    if (!q.is_cuda() || q.scalar_type() != ScalarType::BFloat16 || (q.dim() != 3 && q.dim() != 4) ||
        !q.is_contiguous())
      bad("q must be a contiguous CUDA bf16 tensor [bs, q_len, h_q, hd] or [bs, h_q, hd]");
    const c10::Device dev = q.device();
    const int64_t bs = q.size(0), h_q = q.size(-2), hd = q.size(-1), q_len = q.dim() == 4 ? q.size(1) : 1;
    const CacheShape s = cache_shape(kc, "k_cache", dev);
    if (kc.dim() != 4 || vc.sizes() != kc.sizes() || vc.scalar_type() != kc.scalar_type() || vc.device() != dev ||
        !vc.is_contiguous())
      bad("k_cache and v_cache must match");
    if (kc.scalar_type() != ScalarType::Byte && kc.scalar_type() != ScalarType::Float4_e2m1fn_x2)
      throw BadStatus{FP8MLA_ERR_UNSUPPORTED_DTYPE, "paged_gqa_decode_fp4"};
    if (s.wide * 2 != hd) bad("head_dim mismatch");
    need_scales("k", s, hd, FP8MLA_KV_E2M1, ks, nullptr, kb, dev);
    need_scales("v", s, hd, FP8MLA_KV_E2M1, vs, nullptr, vb, dev);
    if (bt.device() != dev || bt.scalar_type() != ScalarType::Int || bt.dim() != 2 || bt.size(0) != bs ||
        !bt.is_contiguous())
      bad("block_table must be contiguous int32 [bs, max_blocks] on " + dev.str());
    need_int32(sl, "seqlens", dev, bs);
    if (mask != nullptr &&
        (mask->device() != dev || mask->scalar_type() != ScalarType::Byte || mask->dim() != 3 ||
         mask->size(0) != bs || mask->size(1) != q_len || mask->size(2) != q_len || !mask->is_contiguous()))
      bad("spec_mask must be contiguous uint8 [bs, q_len, q_len]");
    if (sinks != nullptr && (sinks->device() != dev || sinks->scalar_type() != ScalarType::Float ||
                             sinks->dim() != 1 || sinks->size(0) != h_q || !sinks->is_contiguous()))
      bad("sinks must be contiguous float32 [h_q]");
    double scale = 1.0 / std::sqrt(static_cast<double>(hd));
    if (a[9] != Py_None) {
      scale = PyFloat_AsDouble(a[9]);
      if (scale == -1.0 && PyErr_Occurred()) throw PyFailure{};
    }
    const int window = small(a[11], "window"), splits = small(a[13], "num_splits");
    const int b32 = dim32(bs, "bs"), hq32 = dim32(h_q, "h_q"), hkv32 = dim32(s.h_kv, "h_kv"),
              hd32 = dim32(hd, "head_dim"), ql32 = dim32(q_len, "q_len");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out_new, lse_new, ws_new;
    if (out == nullptr) {
      out_new = make(q.sizes(), ScalarType::BFloat16, dev);
      out = &out_new;
    } else {
      need_like(*out, "out", q.sizes(), ScalarType::BFloat16, dev);
    }
    const c10::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
    if (lse == nullptr) {
      lse_new = make(rows, ScalarType::Float, dev);
      lse = &lse_new;
    } else {
      need_like(*lse, "lse", rows, ScalarType::Float, dev);
    }
    if (ws == nullptr) {
      const size_t need =
          paged_gqa_fp4_workspace_bytes(b32, hq32, hkv32, hd32, ql32, bt.size(1) * s.page, window, splits);
      if (need > 0) {
        ws_new = make({static_cast<int64_t>(need)}, ScalarType::Byte, dev);
        ws = &ws_new;
      }
    } else if (ws->device() != dev || !ws->is_contiguous()) {
      bad("workspace must be a contiguous tensor on " + dev.str());
    }
    check(paged_gqa_decode_fp4(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ptr(kb), ptr(vb),
                               dim32(s.blocks, "num_blocks"), ptr_as<const float>(ks), ptr_as<const float>(vs),
                               ptr_as<const int32_t>(&bt), dim32(bt.size(1), "max_blocks"), ptr_as<const int32_t>(&sl),
                               static_cast<float>(scale), ql32, ptr_as<const uint8_t>(mask), window,
                               ptr_as<const float>(sinks), splits, ptr(ws), ws != nullptr ? ws->nbytes() : 0,
                               out->data_ptr(), ptr_as<float>(lse), b32, hq32, hkv32, hd32, dim32(s.page, "page"),
                               stream_of(dev)),
          "paged_gqa_decode_fp4");
    written({out, lse});
    PyObject* po = wrap(out, a[14]);
    PyObject* pl = wrap(lse, a[15]);
    if (po == nullptr || pl == nullptr) {
      Py_XDECREF(po);
      Py_XDECREF(pl);
      return nullptr;
    }
    PyObject* r = PyTuple_Pack(2, po, pl);
    Py_DECREF(po);
    Py_DECREF(pl);
    return r;
  });
}

// A pair of objects, both taken over.
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// K and V caches in E4M3 with one scale each or one per row; returns whether the scales go by row.
int need_e4m3_caches(const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs, const CacheShape& s,
                     int64_t hd, const c10::Device& dev, const char* where) {
  if (kc.dim() != 4 || vc.sizes() != kc.sizes() || vc.scalar_type() != kc.scalar_type() || vc.device() != dev ||
      !vc.is_contiguous())
    bad("k_cache and v_cache must match");
  if (kv_code(kc, nullptr) != FP8MLA_KV_E4M3) throw BadStatus{FP8MLA_ERR_UNSUPPORTED_DTYPE, where};
  if (s.wide != hd) bad("head_dim mismatch");
  const bool rows = ks.numel() != 1 || vs.numel() != 1;
  need_scales("k", s, hd, FP8MLA_KV_E4M3, rows ? nullptr : &ks, rows ? &ks : nullptr, nullptr, dev);
  need_scales("v", s, hd, FP8MLA_KV_E4M3, rows ? nullptr : &vs, rows ? &vs : nullptr, nullptr, dev);
  return rows ? 1 : 0;
}
int64_t need_block_table(const Tensor& t, const char* name, int64_t n, const c10::Device& dev) {
  if (t.device() != dev || t.scalar_type() != ScalarType::Int || t.dim() != 2 || t.size(0) != n || !t.is_contiguous())
    bad(std::string(name) + " must be contiguous int32 [" + std::to_string(n) + ", max_blocks] on " + dev.str());
  return t.size(1);
}
// (a table without columns has no memory, whatever it is a view of)
const int32_t* table_ptr(const Tensor& t) { return t.numel() > 0 ? static_cast<const int32_t*>(t.data_ptr()) : nullptr; }
float softmax_scale_of(PyObject* o, int64_t hd) {
  double scale = 1.0 / std::sqrt(static_cast<double>(hd));
  if (o != Py_None) {
    scale = PyFloat_AsDouble(o);
    if (scale == -1.0 && PyErr_Occurred()) throw PyFailure{};
  }
  return static_cast<float>(scale);
}
const Tensor* need_workspace(const Tensor* ws, Tensor* made, size_t need, const c10::Device& dev) {
  if (ws == nullptr) {
    *made = make({static_cast<int64_t>(need)}, ScalarType::Byte, dev);
    return made;
  }
  if (ws->device() != dev || !ws->is_contiguous()) bad("workspace must be a contiguous tensor on " + dev.str());
  return ws;
}

// (q, k_cache, v_cache, block_table, kv_lens, k_scale, v_scale, softmax_scale, q_starts, out, lse, workspace)
// -> (out, lse)
PyObject* py_cross(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &q = given(a[0], "q"), &kc = given(a[1], "k_cache"), &vc = given(a[2], "v_cache");
    const Tensor &bt = given(a[3], "block_table"), &kl = given(a[4], "kv_lens");
    const Tensor &ks = given(a[5], "k_scale"), &vs = given(a[6], "v_scale");
    const Tensor *starts = maybe(a[8], "q_starts"), *out = maybe(a[9], "out"), *lse = maybe(a[10], "lse");
    const Tensor* ws = maybe(a[11], "workspace");
    need_no_grad({&q, &kc, &vc, &ks, &vs, out, lse});
    if (!q.is_cuda()) bad("q must be a CUDA bf16 tensor [n, h_q, head_dim]");
    const c10::Device dev = q.device();
    const int64_t n = q.dim() > 0 ? q.size(0) : 0;
    need_heads(q, "q", ScalarType::BFloat16, dev, n);
    const int64_t h_q = q.size(1), hd = q.size(2);
    const CacheShape s = cache_shape(kc, "k_cache", dev);
    const int by_row = need_e4m3_caches(kc, vc, ks, vs, s, hd, dev, "paged_cross_attention");
    need_int32(kl, "kv_lens", dev, -1);
    const int64_t bs = kl.size(0), blocks = need_block_table(bt, "block_table", bs, dev);
    if (starts != nullptr) need_int32(*starts, "q_starts", dev, bs + 1);
    if (starts == nullptr && n != bs) bad("without q_starts, q has a token for each sequence");
    const float scale = softmax_scale_of(a[7], hd);
    const int n32 = dim32(n, "n"), bs32 = dim32(bs, "bs"), hq32 = dim32(h_q, "h_q"), hkv32 = dim32(s.h_kv, "h_kv"),
              hd32 = dim32(hd, "head_dim");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out_new, lse_new, ws_new;  // nothing else will have written their rows of no sequence
    const int fill = starts != nullptr, fill_out = fill && out == nullptr, fill_lse = fill && lse == nullptr;
    if (out == nullptr) {
      out_new = make(q.sizes(), ScalarType::BFloat16, dev);
      out = &out_new;
    } else {
      need_heads_out(*out, "out", q.sizes(), ScalarType::BFloat16, dev);
    }
    const c10::IntArrayRef rows = q.sizes().slice(0, 2);
    if (lse == nullptr) {
      lse_new = make(rows, ScalarType::Float, dev);
      lse = &lse_new;
    } else {
      need_like(*lse, "lse", rows, ScalarType::Float, dev);
    }
    ws = need_workspace(ws, &ws_new, paged_cross_workspace_bytes(n32, bs32, hq32, hkv32, hd32, blocks * s.page), dev);
    check(paged_cross_attention(q.data_ptr(), stride_of(&q, 0), stride_of(&q, 1), kc.data_ptr(), vc.data_ptr(),
                                FP8MLA_KV_E4M3, dim32(s.blocks, "num_blocks"), ptr_as<const float>(&ks),
                                ptr_as<const float>(&vs), by_row, ptr_as<const int32_t>(starts),
                                table_ptr(bt), dim32(blocks, "max_blocks"), ptr_as<const int32_t>(&kl),
                                scale, ptr(ws), ws->nbytes(), out->data_ptr(), stride_of(out, 0), stride_of(out, 1),
                                ptr_as<float>(lse), fill_out, fill_lse, n32, bs32, hq32, hkv32, hd32,
                                dim32(s.page, "page"), stream_of(dev)),
          "paged_cross_attention");
    written({out, lse});
    return pair(wrap(out, a[9]), wrap(lse, a[10]));
  });
}

// (q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, block_table, seqlens, k_scale, v_scale,
//  softmax_scale, spec_mask, sinks, out, lse, workspace) -> (out, lse)
PyObject* py_shared(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 16)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &q = given(a[0], "q"), &kc = given(a[1], "k_cache"), &vc = given(a[2], "v_cache");
    const Tensor &pt = given(a[3], "prefix_table"), &pl = given(a[4], "prefix_lens"), &ps = given(a[5], "prefix_starts");
    const Tensor &bt = given(a[6], "block_table"), &sl = given(a[7], "seqlens");
    const Tensor &ks = given(a[8], "k_scale"), &vs = given(a[9], "v_scale");
    const Tensor *mask = maybe(a[11], "spec_mask"), *sinks = maybe(a[12], "sinks");
    const Tensor *out = maybe(a[13], "out"), *lse = maybe(a[14], "lse"), *ws = maybe(a[15], "workspace");
    need_no_grad({&q, &kc, &vc, &ks, &vs, sinks, out, lse});
    if (!q.is_cuda() || q.scalar_type() != ScalarType::BFloat16 || (q.dim() != 3 && q.dim() != 4) || !q.is_contiguous())
      bad("q must be a contiguous CUDA bf16 tensor [bs, q_len, h_q, hd] or [bs, h_q, hd]");
    const c10::Device dev = q.device();
    const int64_t bs = q.size(0), h_q = q.size(-2), hd = q.size(-1), q_len = q.dim() == 4 ? q.size(1) : 1;
    const CacheShape s = cache_shape(kc, "k_cache", dev);
    const int by_row = need_e4m3_caches(kc, vc, ks, vs, s, hd, dev, "paged_gqa_decode_shared");
    need_int32(pl, "prefix_lens", dev, -1);
    const int64_t n_prefixes = pl.size(0), prefix_blocks = need_block_table(pt, "prefix_table", n_prefixes, dev);
    need_int32(ps, "prefix_starts", dev, n_prefixes + 1);
    const int64_t blocks = need_block_table(bt, "block_table", bs, dev);
    need_int32(sl, "seqlens", dev, bs);
    if (mask != nullptr &&
        (mask->device() != dev || mask->scalar_type() != ScalarType::Byte || mask->dim() != 3 || mask->size(0) != bs ||
         mask->size(1) != q_len || mask->size(2) != q_len || !mask->is_contiguous()))
      bad("spec_mask must be contiguous uint8 [bs, q_len, q_len]");
    if (sinks != nullptr && (sinks->device() != dev || sinks->scalar_type() != ScalarType::Float || sinks->dim() != 1 ||
                             sinks->size(0) != h_q || !sinks->is_contiguous()))
      bad("sinks must be contiguous float32 [h_q]");
    const float scale = softmax_scale_of(a[10], hd);
    const int bs32 = dim32(bs, "bs"), ql32 = dim32(q_len, "q_len"), hq32 = dim32(h_q, "h_q"),
              hkv32 = dim32(s.h_kv, "h_kv"), hd32 = dim32(hd, "head_dim"), np32 = dim32(n_prefixes, "n_prefixes");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out_new, lse_new, ws_new;
    if (out == nullptr) {
      out_new = make(q.sizes(), ScalarType::BFloat16, dev);
      out = &out_new;
    } else {
      need_like(*out, "out", q.sizes(), ScalarType::BFloat16, dev);
    }
    const c10::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
    if (lse == nullptr) {
      lse_new = make(rows, ScalarType::Float, dev);
      lse = &lse_new;
    } else {
      need_like(*lse, "lse", rows, ScalarType::Float, dev);
    }
    ws = need_workspace(ws, &ws_new,
                        paged_gqa_shared_workspace_bytes(bs32, ql32, hq32, hkv32, hd32, np32,
                                                         np32 > 0 ? prefix_blocks * s.page : 0, blocks * s.page),
                        dev);
    check(paged_gqa_decode_shared(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), FP8MLA_KV_E4M3,
                                  dim32(s.blocks, "num_blocks"), ptr_as<const float>(&ks), ptr_as<const float>(&vs),
                                  by_row, table_ptr(pt), dim32(prefix_blocks, "prefix_blocks"),
                                  ptr_as<const int32_t>(&pl), ptr_as<const int32_t>(&ps), np32,
                                  table_ptr(bt), dim32(blocks, "max_blocks"), ptr_as<const int32_t>(&sl),
                                  scale, ql32, ptr_as<const uint8_t>(mask), ptr_as<const float>(sinks), ptr(ws),
                                  ws->nbytes(), out->data_ptr(), ptr_as<float>(lse), bs32, hq32, hkv32, hd32,
                                  dim32(s.page, "page"), stream_of(dev)),
          "paged_gqa_decode_shared");
    written({out, lse});
    return pair(wrap(out, a[13]), wrap(lse, a[14]));
  });
}

// (outs, lses, out, lse) -> (out, lse); outs and lses are lists or tuples
PyObject* py_merge(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!count(nargs, 4)) return nullptr;
  return guarded([&]() -> PyObject* {
    if ((!PyList_Check(a[0]) && !PyTuple_Check(a[0])) || (!PyList_Check(a[1]) && !PyTuple_Check(a[1])))
      bad("outs and lses must be lists or tuples of tensors");
    const Py_ssize_t parts = PySequence_Fast_GET_SIZE(a[0]);
    if (parts < 1 || parts > FP8MLA_MERGE_MAX_PARTS || PySequence_Fast_GET_SIZE(a[1]) != parts)
      bad("outs and lses must have the same 1 to " + std::to_string(FP8MLA_MERGE_MAX_PARTS) + " parts");
    const Tensor *out = maybe(a[2], "out"), *lse = maybe(a[3], "lse");
    need_no_grad({out, lse});
    const Tensor& first = given(PySequence_Fast_GET_ITEM(a[0], 0), "outs");
    if (!first.is_cuda()) bad("outs must be CUDA bf16 tensors [n, heads, dim]");
    const c10::Device dev = first.device();
    const int64_t n = first.dim() > 0 ? first.size(0) : 0;
    need_heads(first, "outs", ScalarType::BFloat16, dev, n);
    const c10::IntArrayRef rows = first.sizes().slice(0, 2);
    const void* xs[FP8MLA_MERGE_MAX_PARTS];
    const float* ls[FP8MLA_MERGE_MAX_PARTS];
    int64_t tokens[FP8MLA_MERGE_MAX_PARTS], heads[FP8MLA_MERGE_MAX_PARTS];
    for (Py_ssize_t i = 0; i < parts; ++i) {
      const Tensor& x = given(PySequence_Fast_GET_ITEM(a[0], i), "outs");
      const Tensor& l = given(PySequence_Fast_GET_ITEM(a[1], i), "lses");
      need_no_grad({&x, &l});
      need_heads(x, "outs", ScalarType::BFloat16, dev, n, first.size(2));
      if (x.sizes() != first.sizes()) bad("outs must have the same shape");
      need_like(l, "lses", rows, ScalarType::Float, dev);
      xs[i] = x.data_ptr();
      ls[i] = l.data_ptr<float>();
      tokens[i] = stride_of(&x, 0);
      heads[i] = stride_of(&x, 1);
    }
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out_new, lse_new;
    if (out == nullptr) {
      out_new = make(first.sizes(), ScalarType::BFloat16, dev);
      out = &out_new;
    } else {
      need_heads_out(*out, "out", first.sizes(), ScalarType::BFloat16, dev);
    }
    if (lse == nullptr) {
      lse_new = make(rows, ScalarType::Float, dev);
      lse = &lse_new;
    } else {
      need_like(*lse, "lse", rows, ScalarType::Float, dev);
    }
    check(attention_merge(xs, tokens, heads, ls, static_cast<int>(parts), out->data_ptr(), stride_of(out, 0),
                          stride_of(out, 1), ptr_as<float>(lse), dim32(n, "n"), dim32(first.size(1), "heads"),
                          dim32(first.size(2), "dim"), stream_of(dev)),
          "attention_merge");
    written({out, lse});
    return pair(wrap(out, a[2]), wrap(lse, a[3]));
  });
}

PyObject* py_set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_status_error);
  Py_INCREF(cls);
  g_status_error = cls;
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef g_methods[] = {
    {"rotary_apply", fast(py_rotary_apply), METH_FASTCALL, nullptr},
    {"paged_kv_append", fast(py_kv_append), METH_FASTCALL, nullptr},
    {"paged_cache_read", fast(py_cache_read), METH_FASTCALL, nullptr},
    {"paged_gqa_decode_fp4", fast(py_decode_fp4), METH_FASTCALL, nullptr},
    {"paged_cross_attention", fast(py_cross), METH_FASTCALL, nullptr},
    {"paged_gqa_decode_shared", fast(py_shared), METH_FASTCALL, nullptr},
    {"attention_merge", fast(py_merge), METH_FASTCALL, nullptr},
    {"set_error", py_set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
