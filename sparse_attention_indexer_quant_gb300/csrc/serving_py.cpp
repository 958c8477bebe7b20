// Host path of the serving operators' Python binding: checks the tensors,
// allocates outputs and workspaces on the current stream and calls the C entry
// of the same name (include/idx.h).  The operators run once per layer and step,
// and the smallest of them take a few microseconds on the GPU: marshalled
// through ctypes and Python-level checks a call cost 16 - 34 us of host time.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <math.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "idx.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_idx_error = nullptr;  // binding.IdxError
PyObject* g_oom_error = nullptr;  // torch.OutOfMemoryError

// Thrown once the Python error is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw Raised{};
}
[[noreturn]] void value_error(const std::string& msg) { raise(PyExc_ValueError, msg); }
[[noreturn]] void type_error(const std::string& msg) { raise(PyExc_TypeError, msg); }

void check(const char* fn, int status) {
  if (status == IDX_OK) return;
  PyObject* e = PyObject_CallFunction(g_idx_error, "sis", fn, status, idx_last_error_detail());
  if (e) {
    PyErr_SetObject(g_idx_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

const char* name_of(ScalarType t) {
  switch (t) {
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
    default: return at::toString(t);
  }
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}
void on_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != c10::cuda::current_device())
    value_error(std::string(name) + " must be on the current device");
}
const Tensor& need(PyObject* o, ScalarType dtype, const char* name, bool contiguous = true) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " must be " + name_of(dtype) + ", got " + name_of(t.scalar_type()));
  on_device(t, name);
  if (contiguous && !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}
template <class T = void>
T* ptr(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
// An optional tensor's pointer after the same checks; null for None.
template <class T>
T* maybe(PyObject* o, ScalarType dtype, const char* name, int64_t numel, const char* what) {
  if (o == Py_None) return nullptr;
  const Tensor& t = need(o, dtype, name);
  if (t.numel() != numel) value_error(std::string(name) + " must " + what);
  return ptr<T>(t);
}
idx_device_errors* errors_of(PyObject* o) {
  if (o == Py_None) return nullptr;
  const Tensor& t = need(o, ScalarType::Int, "errors");
  if (t.numel() < 2) value_error("errors must hold two values");
  return ptr<idx_device_errors>(t);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int32_t int32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) value_error(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
Tensor empty(at::IntArrayRef sizes, ScalarType dtype) {
  return at::detail::empty_cuda(sizes, dtype, c10::Device(c10::kCUDA, c10::cuda::current_device()),
                                std::nullopt);
}
// n values of dtype at element `at` of t's memory.
Tensor part_of(const Tensor& t, ScalarType dtype, int64_t at, int64_t n) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(),
                                                   c10::scalarTypeToTypeMeta(dtype));
  impl->set_storage_offset(at);
  impl->set_sizes_contiguous({n});
  return Tensor(std::move(impl));
}
idx_stream_t stream() {
  return reinterpret_cast<idx_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
}
PyObject* wrap_all(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}
// Runs f and turns C++ exceptions (allocation failures among them) into Python's.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_oom_error, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// A dimension of one entry has no stride to speak of: whatever torch says there
// need not be aligned.
int64_t stride_of(const Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

int dtype_of(const Tensor& q) {
  if (q.scalar_type() == ScalarType::BFloat16) return IDX_BF16;
  if (q.scalar_type() == ScalarType::Half) return IDX_FP16;
  type_error(std::string("q must be bfloat16 or float16, got ") + name_of(q.scalar_type()));
}

idx_kv_cache kv_of(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso) {
  if (!THPVariable_Check(ko) || !THPVariable_Check(vo))
    type_error("k_cache and v_cache must be torch.Tensors");
  const Tensor &k = THPVariable_Unpack(ko), &v = THPVariable_Unpack(vo);
  idx_kv_cache kv{};
  switch (k.scalar_type()) {
    case ScalarType::BFloat16: kv.dtype = IDX_BF16; break;
    case ScalarType::Half: kv.dtype = IDX_FP16; break;
    case ScalarType::Float8_e4m3fn: kv.dtype = IDX_E4M3; break;
    default: type_error("k_cache and v_cache must both be bfloat16, float16 or float8_e4m3fn");
  }
  if (v.scalar_type() != k.scalar_type())
    type_error("k_cache and v_cache must both be bfloat16, float16 or float8_e4m3fn");
  on_device(k, "k_cache");
  on_device(v, "v_cache");
  if (k.dim() != 4 || v.sizes() != k.sizes())
    value_error("k_cache and v_cache must be [num_blocks, heads, page_size, head_dim]");
  if (k.stride(3) != 1 || v.stride(3) != 1)
    value_error("k_cache and v_cache must have unit stride in the last dim");
  kv.k = ptr(k);
  kv.v = ptr(v);
  kv.num_blocks = k.size(0);
  for (int i = 1; i < 4; ++i)
    if (k.size(i) > INT32_MAX) value_error("k_cache is too large");
  kv.heads = (int32_t)k.size(1);
  kv.page_size = (int32_t)k.size(2);
  kv.head_dim = (int32_t)k.size(3);
  kv.k_block_stride = stride_of(k, 0);
  kv.k_head_stride = stride_of(k, 1);
  kv.k_token_stride = stride_of(k, 2);
  kv.v_block_stride = stride_of(v, 0);
  kv.v_head_stride = stride_of(v, 1);
  kv.v_token_stride = stride_of(v, 2);
  kv.k_scale = maybe<const float>(kso, ScalarType::Float, "k_scale", kv.heads,
                                  "have one entry per kv head");
  kv.v_scale = maybe<const float>(vso, ScalarType::Float, "v_scale", kv.heads,
                                  "have one entry per kv head");
  return kv;
}

// [rows, heads, dim] of dtype, any strides with a unit last one.
const Tensor& heads_of(PyObject* o, const char* name, int64_t rows, int64_t dim, ScalarType dtype) {
  const Tensor& t = need(o, dtype, name, false);
  if (t.dim() != 3 || t.size(0) != rows || t.size(2) != dim || t.stride(2) != 1)
    value_error(std::string(name) + " must be [" + std::to_string(rows) + ", heads, " +
                std::to_string(dim) + "] with unit stride in the last dim");
  return t;
}

// (cached_lens, new_lens, block_table, free_pages, pool_head, num_tokens,
//  num_blocks, page_size, out or None, errors or None) -> 6 tensors
PyObject* plan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10) type_error("plan_step takes 10 arguments");
    const Tensor& cached = need(a[0], ScalarType::Int, "cached_lens");
    const Tensor& fresh = need(a[1], ScalarType::Int, "new_lens");
    const Tensor& bt = need(a[2], ScalarType::Int, "block_table");
    const Tensor& free_pages = need(a[3], ScalarType::Int, "free_pages");
    const Tensor& head = need(a[4], ScalarType::Int, "pool_head");
    const int64_t B = cached.numel(), tokens = integer(a[5]);
    if (fresh.numel() != B) value_error("cached_lens and new_lens must have one entry per request");
    if (bt.dim() != 2 || bt.size(0) != B) value_error("block_table must be [B, max_blocks]");
    if (head.numel() != 1) value_error("pool_head must hold one value");
    if (tokens < 0) value_error("num_tokens must not be negative");
    if (B > INT32_MAX || bt.size(1) > INT32_MAX || free_pages.numel() > INT32_MAX)
      value_error("block_table or free_pages is too large");
    // context_lens, query_start, slot_mapping, positions, token_seq, pool_head
    const int64_t sizes[6] = {B, B + 1, tokens, tokens, tokens, 1};
    const char* names[6] = {"out.context_lens", "out.query_start", "out.slot_mapping",
                            "out.positions", "out.token_seq", "out.pool_head"};
    Tensor o[6];
    if (a[8] == Py_None) {
      // one allocation: the slots first, on its 8 bytes, then the 32-bit arrays
      const Tensor all = empty({2 * tokens + 2 * B + 2 + 2 * tokens}, ScalarType::Int);
      int64_t at = 2 * tokens;
      for (int i = 0; i < 6; ++i) {
        if (i == 2) {
          o[i] = part_of(all, ScalarType::Long, 0, tokens);
        } else {
          o[i] = part_of(all, ScalarType::Int, at, sizes[i]);
          at += sizes[i];
        }
      }
    } else {
      for (int i = 0; i < 6; ++i) {
        const ScalarType t = i == 2 ? ScalarType::Long : ScalarType::Int;
        if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 6) type_error("out must be a StepPlan");
        o[i] = need(PyTuple_GET_ITEM(a[8], i), t, names[i]);
        if (o[i].numel() != sizes[i])
          value_error(std::string(names[i]) + " must hold " + std::to_string(sizes[i]) + " values");
      }
    }
    check("idx_plan_step",
          idx_plan_step(ptr<int32_t>(cached), ptr<int32_t>(fresh), (int32_t)B, ptr<int32_t>(bt),
                        (int32_t)bt.size(1), ptr<int32_t>(free_pages), (int32_t)free_pages.numel(),
                        ptr<int32_t>(head), ptr<int32_t>(o[5]), integer(a[6]),
                        int32(a[7], "page_size"), ptr<int32_t>(o[0]), ptr<int32_t>(o[1]),
                        ptr<int64_t>(o[2]), ptr<int32_t>(o[3]), ptr<int32_t>(o[4]), tokens,
                        errors_of(a[9]), stream()));
    if (a[8] != Py_None) {
      Py_INCREF(a[8]);
      return a[8];
    }
    return wrap_all({o[0], o[1], o[2], o[3], o[4], o[5]});
  });
}

// (num_pos, rot_dim, base, scaling, factor, orig_len, beta_fast, beta_slow,
//  mscale, pos0, cos or None, sin or None) -> (cos, sin)
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) type_error("rope_table takes 12 arguments");
    const int64_t rows = integer(a[0]);
    const int32_t rot = int32(a[1], "rot_dim");
    Tensor o[2];
    for (int i = 0; i < 2; ++i) {
      if (a[10] == Py_None) {
        o[i] = empty({rows > 0 ? rows : 0, rot > 0 ? rot / 2 : 0}, ScalarType::Float);
      } else {
        o[i] = need(a[10 + i], ScalarType::Float, i ? "out[1]" : "out[0]");
        if (o[i].dim() != 2 || o[i].size(0) != rows || o[i].size(1) != rot / 2)
          value_error("out must be two tensors [num_pos, rot_dim / 2]");
      }
    }
    check("idx_rope_table",
          idx_rope_table(integer(a[9]), rows, rot, real(a[2]), int32(a[3], "scaling"), real(a[4]),
                         real(a[5]), real(a[6]), real(a[7]), real(a[8]), ptr<float>(o[0]),
                         ptr<float>(o[1]), stream()));
    return wrap_all({o[0], o[1]});
  });
}

// (q, k, v, q_weight, k_weight, eps, positions, cos, sin, rot_dim, slot_mapping,
//  k_cache, v_cache, interleaved, k_scale, v_scale, q_out or None, errors) -> q_out
PyObject* qk_norm_rope_insert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 18) type_error("qk_norm_rope_insert takes 18 arguments");
    const idx_kv_cache kv = kv_of(a[11], a[12], a[14], a[15]);
    const Tensor& q0 = tensor(a[0], "q");
    const int dtype = dtype_of(q0);
    const int64_t N = q0.dim() > 0 ? q0.size(0) : 0, dim = kv.head_dim;
    const Tensor& q = heads_of(a[0], "q", N, dim, q0.scalar_type());
    const Tensor& k = heads_of(a[1], "k", N, dim, q0.scalar_type());
    const Tensor& v = heads_of(a[2], "v", N, dim, q0.scalar_type());
    if (k.size(1) != kv.heads || v.size(1) != kv.heads)
      value_error("k and v must have the cache's " + std::to_string(kv.heads) + " heads");
    if (q.size(1) > INT32_MAX) value_error("q has too many heads");
    const Tensor& slots = need(a[10], ScalarType::Long, "slot_mapping");
    if (slots.numel() != N) value_error("slot_mapping must have one entry per token");
    const float* qw = maybe<const float>(a[3], ScalarType::Float, "q_weight", dim, "have head_dim entries");
    const float* kw = maybe<const float>(a[4], ScalarType::Float, "k_weight", dim, "have head_dim entries");
    const int32_t rot = int32(a[9], "rot_dim");
    const int32_t* pos = nullptr;
    const float *cs = nullptr, *sn = nullptr;
    int64_t num_pos = 0;
    if (rot > 0) {
      const Tensor& p = need(a[6], ScalarType::Int, "positions");
      const Tensor& c = need(a[7], ScalarType::Float, "cos");
      const Tensor& s = need(a[8], ScalarType::Float, "sin");
      if (p.numel() != N) value_error("positions must have one entry per token");
      if (c.dim() != 2 || c.sizes() != s.sizes() || c.size(1) != rot / 2)
        value_error("cos/sin must be [num_pos, rot_dim / 2]");
      pos = ptr<int32_t>(p);
      cs = ptr<float>(c);
      sn = ptr<float>(s);
      num_pos = c.size(0);
    }
    const int inter = PyObject_IsTrue(a[13]);
    if (inter < 0) throw Raised{};
    Tensor out;
    if (a[16] == Py_None) {
      out = empty(q.sizes(), q.scalar_type());
    } else {
      out = need(a[16], q.scalar_type(), "q_out");
      if (out.sizes() != q.sizes()) value_error("q_out must have q's shape");
    }
    check("idx_qk_norm_rope_insert",
          idx_qk_norm_rope_insert(ptr(q), stride_of(q, 0), stride_of(q, 1), ptr(k), stride_of(k, 0), stride_of(k, 1),
                                  ptr(v), stride_of(v, 0), stride_of(v, 1), N, (int32_t)q.size(1), dtype, qw,
                                  kw, (float)real(a[5]), pos, cs, sn, num_pos, rot, inter,
                                  ptr<int64_t>(slots), ptr(out), &kv, errors_of(a[17]), stream()));
    if (a[16] != Py_None) {
      Py_INCREF(a[16]);
      return a[16];
    }
    return THPVariable_Wrap(out);
  });
}

// (q, k_cache, v_cache, block_table, context_lens, next_n, scale or None,
//  softcap, window, topk, k_scale, v_scale, workspace, out, lse, return_lse,
//  errors) -> (out, lse or None)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 17) type_error("paged_attention takes 17 arguments");
    const idx_kv_cache kv = kv_of(a[1], a[2], a[10], a[11]);
    const Tensor& bt = need(a[3], ScalarType::Int, "block_table");
    const Tensor& lens = need(a[4], ScalarType::Int, "context_lens");
    const int64_t B = lens.numel(), dim = kv.head_dim;
    if (bt.dim() != 2 || bt.size(0) != B) value_error("block_table must be [B, max_blocks]");
    if (B > INT32_MAX || bt.size(1) > INT32_MAX) value_error("block_table is too large");
    const int32_t next_n = int32(a[5], "next_n");
    const Tensor& q0 = tensor(a[0], "q");
    const int dtype = dtype_of(q0);
    const int64_t rows = B * next_n;
    const Tensor& q = heads_of(a[0], "q", rows, dim, q0.scalar_type());
    const int64_t Hq = q.size(1);
    if (Hq > INT32_MAX) value_error("q has too many heads");
    const int32_t* topk = nullptr;
    int64_t k = 0;
    if (a[9] != Py_None) {
      const Tensor& t = need(a[9], ScalarType::Int, "topk");
      if (t.dim() != 2 || t.size(0) != rows) value_error("topk must be [B * next_n, k]");
      k = t.size(1);
      if (k == 0 || k > INT32_MAX) value_error("topk must list 1 to 2^20 positions a row");
      topk = ptr<int32_t>(t);
    }
    const int want_lse = PyObject_IsTrue(a[15]);
    if (want_lse < 0) throw Raised{};
    Tensor ws, out, lse;
    if (a[12] == Py_None) {
      const size_t need_bytes =
          idx_paged_attention_workspace_bytes((int32_t)B, next_n, (int32_t)Hq, kv.heads, kv.head_dim);
      ws = empty({(int64_t)(need_bytes > 256 ? need_bytes : 256)}, ScalarType::Byte);
    } else {
      ws = need(a[12], ScalarType::Byte, "workspace");
    }
    if (a[13] == Py_None) {
      out = empty({rows, Hq, dim}, q.scalar_type());
    } else {
      out = need(a[13], q.scalar_type(), "out");
      if (out.sizes() != q.sizes()) value_error("out must be [B * next_n, Hq, D]");
    }
    if (a[14] != Py_None) {
      lse = need(a[14], ScalarType::Float, "lse");
      if (lse.dim() != 2 || lse.size(0) != rows || lse.size(1) != Hq)
        value_error("lse must be [B * next_n, Hq]");
    } else if (want_lse) {
      lse = empty({rows, Hq}, ScalarType::Float);
    }
    const float scale = a[6] == Py_None ? (float)(1.0 / sqrt((double)dim)) : (float)real(a[6]);
    check("idx_paged_attention",
          idx_paged_attention(ptr(q), stride_of(q, 0), stride_of(q, 1), dtype, (int32_t)B, next_n,
                              (int32_t)Hq, &kv, ptr<int32_t>(bt), (int32_t)bt.size(1),
                              ptr<int32_t>(lens), topk, (int32_t)k, scale, (float)real(a[7]),
                              int32(a[8], "window"), ptr(out),
                              lse.defined() ? ptr<float>(lse) : nullptr, ptr(ws),
                              (size_t)ws.numel(), errors_of(a[16]), stream()));
    PyObject* res = PyTuple_New(2);
    PyObject* o = a[13] != Py_None ? Py_NewRef(a[13]) : THPVariable_Wrap(out);
    PyObject* l = a[14] != Py_None ? Py_NewRef(a[14])
                  : lse.defined()  ? THPVariable_Wrap(lse)
                                   : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(res, 0, o);
    PyTuple_SET_ITEM(res, 1, l);
    return res;
  });
}

// The exception types to raise: (IdxError, torch.OutOfMemoryError), once at import.
PyObject* set_errors(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 2) type_error("set_errors takes 2 arguments");
    g_idx_error = Py_NewRef(a[0]);
    g_oom_error = Py_NewRef(a[1]);
    Py_RETURN_NONE;
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {
    {"plan_step", FAST(plan_step), METH_FASTCALL, nullptr},
    {"rope_table", FAST(rope_table), METH_FASTCALL, nullptr},
    {"qk_norm_rope_insert", FAST(qk_norm_rope_insert), METH_FASTCALL, nullptr},
    {"paged_attention", FAST(paged_attention), METH_FASTCALL, nullptr},
    {"set_errors", FAST(set_errors), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&kModule); }
