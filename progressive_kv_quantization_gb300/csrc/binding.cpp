// Native side of the Python binding of the serving-step entry points: checks
// torch tensors, allocates the outputs that the caller did not pass and calls
// liblynx on the tensors' device and stream.  The same checks through Python
// attributes and ctypes took 6 of a call's 10 microseconds on a Grace core,
// several times what the small kernels run for.
//
// Every function takes its arguments by position from lynx.py, which documents
// them, with None for what was left out; a stream is the cudaStream_t as an
// integer or None for torch's current stream on the tensors' device.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/DimVector.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "lynx.h"

namespace {

PyObject* g_error = nullptr;   // lynx.LynxError

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case at::kByte: return "torch.uint8";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return "?";
  }
}

// Thrown with a Python error set; caught at each entry.
struct Raised {};

[[noreturn]] void raise(const char* fmt, const char* a = "", const char* b = "") {
  PyErr_Format(g_error, fmt, a, b);
  throw Raised{};
}

// sizes as a braced list or a vector
struct Shape {
  at::IntArrayRef sizes;
  Shape(const std::initializer_list<int64_t>& s) : sizes(s.begin(), s.size()) {}
  Shape(const at::DimVector& s) : sizes(s.data(), s.size()) {}
};

class Call {
 public:
  Call(const char* fn, PyObject* first, const char* name) : fn_(fn) {
    if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda())
      raise("%s must live on a CUDA device", name);
    device_ = THPVariable_Unpack(first).device();
    on_device_.set_device(device_);
  }

  // any tensor of the call's device
  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise("%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.device() != device_) raise("%s must live on the device of the other tensors", name);
    return t;
  }

  const at::Tensor& need(PyObject* o, at::ScalarType type, Shape shape, const char* name) {
    if (!THPVariable_Check(o)) raise("%s must be a contiguous %s tensor", name, type_name(type));
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_contiguous())
      raise("%s must be a contiguous %s tensor", name, type_name(type));
    if (!t.sizes().equals(shape.sizes)) {
      char want[128];
      int at = 0;
      for (int64_t s : shape.sizes) at += snprintf(want + at, sizeof(want) - at, at ? ", %lld" : "%lld", (long long)s);
      raise("%s must have the shape (%s)", name, want);
    }
    if (t.device() != device_) raise("%s must live on the device of the other tensors", name);
    return t;
  }

  void* at(PyObject* o, at::ScalarType type, Shape shape, const char* name) {
    return need(o, type, shape, name).data_ptr();
  }

  // an output: the caller's, checked, or a new one; a new reference
  PyObject* make(PyObject* o, at::ScalarType type, Shape shape, const char* name, void** ptr) {
    if (o != Py_None) {
      *ptr = at(o, type, shape, name);
      Py_INCREF(o);
      return o;
    }
    const at::Context& torch_state = at::globalContext();
    if (torch_state.deterministicAlgorithms() && torch_state.deterministicFillUninitializedMemory()) {
      at::Tensor filled = at::empty(shape.sizes, at::TensorOptions().dtype(type).device(device_));
      *ptr = filled.data_ptr();
      return THPVariable_Wrap(std::move(filled));
    }
    // at::empty without its dispatch, which takes longer than the rest
    c10::Allocator* const memory = c10::cuda::CUDACachingAllocator::get();
    int64_t n = 1;
    for (int64_t x : shape.sizes) n *= x;
    const size_t bytes = (size_t)n * c10::elementSize(type);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(c10::Storage::use_byte_size_t(), bytes, memory->allocate(bytes), memory, true),
        c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape.sizes);
    *ptr = t.data_ptr();
    return THPVariable_Wrap(std::move(t));
  }

  // The call's stream, torch's current one while the call lasts: what is allocated
  // here (outputs, a workspace) comes from that stream's memory and goes back to it.
  void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device_.index()).stream();
    void* const s = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Raised{};
    on_stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), device_.index()));
    return s;
  }

  template <typename F>
  void launch(F f) {
    PyThreadState* const held = PyEval_SaveThread();   // a full launch queue blocks here
    const int status = f();
    PyEval_RestoreThread(held);
    if (status != LYNX_OK) {
      PyErr_Format(g_error, "%s: %s (%s)", fn_, lynx_status_string(status), lynx_last_error());
      throw Raised{};
    }
  }

  c10::Device device() const { return device_; }

 private:
  const char* fn_;
  c10::Device device_{c10::kCPU};
  c10::cuda::OptionalCUDAGuard on_device_;   // the tensors' device is current while the call lasts
  c10::cuda::OptionalCUDAStreamGuard on_stream_;
};

// a new reference that is given up when an error is raised
struct Out {
  PyObject* o = nullptr;
  void* p = nullptr;
  ~Out() { Py_XDECREF(o); }
  PyObject* take() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};

// the caller's workspace, or one of `size()` bytes that lives as long as the call
struct Scratch {
  void* p;
  size_t bytes;
  at::Tensor own;
  template <typename F>
  Scratch(Call& c, PyObject* o, F size) {
    if (o == Py_None) {
      bytes = size();
      own = at::empty({(int64_t)(bytes < 16 ? 16 : bytes)}, at::TensorOptions().dtype(at::kByte).device(c.device()));
      p = own.data_ptr();
    } else {
      const at::Tensor& w = c.tensor(o, "workspace");
      if (!w.is_contiguous()) raise("workspace must be a contiguous tensor");
      p = w.data_ptr();
      bytes = w.nbytes();
    }
  }
};

int to_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < -2147483647 || v > 2147483647) raise("%s is out of range", name);
  return (int)v;
}

float to_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

int dim32(int64_t v, const char* name) {
  if (v > 2147483647) raise("%s is out of range", name);
  return (int)v;
}

template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {   // torch's own, such as no memory for an output
    PyErr_SetString(g_error, e.what());
    return nullptr;
  }
}

PyObject* tuple(std::initializer_list<Out*> outs) {
  PyObject* t = PyTuple_New((Py_ssize_t)outs.size());
  if (!t) throw Raised{};
  Py_ssize_t i = 0;
  for (Out* o : outs) PyTuple_SET_ITEM(t, i++, o->take());
  return t;
}

// ctx_len, new_len, page_table, free_pages, n_rows, cu_new, positions, slots, ctx_out, n_taken, stream
PyObject* assign_pages(PyObject* const* a) {
  Call c("lynx_assign_pages", a[2], "page_table");
  const at::Tensor& table = c.tensor(a[2], "page_table");
  if (table.dim() != 3) raise("page_table must be [B, Hkv, max_pages]");
  const int64_t B = table.size(0), Hkv = table.size(1), pages = table.size(2);
  const int n_rows = to_int(a[4], "n_rows");
  if (n_rows < 0) raise("n_rows must not be negative");
  void* t = c.at(a[2], at::kInt, {B, Hkv, pages}, "page_table");
  void* ctx = c.at(a[0], at::kInt, {B}, "ctx_len");
  void* fresh = c.at(a[1], at::kInt, {B}, "new_len");
  const int64_t n_free = THPVariable_Check(a[3]) ? THPVariable_Unpack(a[3]).numel() : 0;
  void* free_pages = c.at(a[3], at::kInt, {n_free}, "free_pages");
  void* stream = c.stream(a[10]);
  Out cu, pos, slots, out, taken;
  cu.o = c.make(a[5], at::kInt, {B + 1}, "cu_new", &cu.p);
  pos.o = c.make(a[6], at::kInt, {n_rows}, "positions", &pos.p);
  slots.o = c.make(a[7], at::kLong, {n_rows, Hkv}, "slots", &slots.p);
  out.o = c.make(a[8], at::kInt, {B}, "ctx_out", &out.p);
  taken.o = c.make(a[9], at::kInt, {1}, "n_taken", &taken.p);
  const int b = dim32(B, "B"), h = dim32(Hkv, "Hkv"), mp = dim32(pages, "max_pages"), nf = dim32(n_free, "free_pages");
  c.launch([&] {
    return lynx_assign_pages((int32_t*)ctx, (int32_t*)fresh, b, h, (int32_t*)t, mp, (int32_t*)free_pages, nf, n_rows,
                             (int32_t*)cu.p, (int32_t*)pos.p, (int64_t*)slots.p, (int32_t*)out.p, (int32_t*)taken.p,
                             stream);
  });
  return tuple({&cu, &pos, &slots, &out, &taken});
}

// The rows and what becomes of them, whatever the pages hold; arguments of `a`: qkv, n_q_heads, n_kv_heads, cos_sin,
// positions, slots; of `b`: q_weight, k_weight, norm_eps, interleaved, q_out, stream
template <typename F>
PyObject* append(Call& c, PyObject* const* a, PyObject* const* b, F call) {
  const at::Tensor& qkv = c.tensor(a[0], "qkv");
  const int Hq = to_int(a[1], "n_q_heads"), Hkv = to_int(a[2], "n_kv_heads");
  if (qkv.scalar_type() != at::kBFloat16 || qkv.dim() != 2 || (qkv.size(1) > 1 && qkv.stride(1) != 1))
    raise("qkv must be a bfloat16 tensor [n_rows, channels] with contiguous channels");
  const int64_t n_rows = qkv.size(0), width = ((int64_t)Hq + 2 * (int64_t)Hkv) * 128;
  if (Hq < 1 || Hkv < 1 || qkv.size(1) < width)
    raise("each row of qkv must hold (n_q_heads + 2 n_kv_heads) * 128 channels");
  const int64_t stride = n_rows > 1 ? qkv.stride(0) : width;
  int max_pos = 0, rot = 0;
  void *table = nullptr, *wq = nullptr, *wk = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor& cs = c.tensor(a[3], "cos_sin");
    if (cs.dim() != 2) raise("cos_sin must be a float32 tensor [max_pos, rot_dim]");
    max_pos = dim32(cs.size(0), "cos_sin");
    rot = dim32(cs.size(1), "cos_sin");
    table = c.at(a[3], at::kFloat, {max_pos, rot}, "cos_sin");
  }
  if (b[0] != Py_None) wq = c.at(b[0], at::kFloat, {128}, "q_weight");
  if (b[1] != Py_None) wk = c.at(b[1], at::kFloat, {128}, "k_weight");
  void* pos = c.at(a[4], at::kInt, {n_rows}, "positions");
  void* slots = c.at(a[5], at::kLong, {n_rows, Hkv}, "slots");
  const float eps = to_float(b[2]);
  const int interleaved = PyObject_IsTrue(b[3]);
  void* stream = c.stream(b[5]);
  Out q;
  q.o = c.make(b[4], at::kBFloat16, {n_rows, Hq, 128}, "q_out", &q.p);
  c.launch([&] {
    return call(qkv.data_ptr(), n_rows, stride, Hq, Hkv, 128, (float*)wq, (float*)wk, eps, (float*)table, max_pos, rot,
                interleaved, (int32_t*)pos, (int64_t*)slots, q.p, stream);
  });
  return q.take();
}

// qkv, n_q_heads, n_kv_heads, cos_sin, positions, slots, k_pages, v_pages, q_weight, k_weight, norm_eps, interleaved,
// q_out, stream
PyObject* qkv_append(PyObject* const* a) {
  Call c("lynx_qkv_append", a[0], "qkv");
  const at::Tensor& kp = c.tensor(a[6], "k_pages");
  const int64_t n_pool = kp.dim() == 3 ? kp.size(0) : 0;
  void* k = c.at(a[6], at::kBFloat16, {n_pool, 128, 256}, "k_pages");
  void* v = c.at(a[7], at::kBFloat16, {n_pool, 128, 256}, "v_pages");
  return append(c, a, a + 8, [&](auto qkv, int64_t n_rows, int64_t stride, int Hq, int Hkv, int D, auto wq, auto wk, float eps,
                                 auto table, int max_pos, int rot, int interleaved, auto pos, auto slots, auto q, auto stream) {
    return lynx_qkv_append(qkv, n_rows, stride, Hq, Hkv, D, wq, wk, eps, table, max_pos, rot, interleaved, pos, slots, q, k,
                           v, n_pool, stream);
  });
}

// The chunks' rows, tables and outputs, whatever the pages hold; arguments from `a` on: page_table, ctx_len,
// n_kv_heads, sm_scale, causal, out, lse, out is float32, workspace, stream
template <typename F>
PyObject* chunk_attn(Call& c, PyObject* rows, PyObject* bounds, PyObject* const* a, F call) {
  const at::Tensor& q = c.tensor(rows, "q");
  if (q.scalar_type() != at::kBFloat16 || q.dim() != 3 || q.size(2) != 128 || q.stride(2) != 1 ||
      (q.size(1) > 1 && q.stride(1) != 128))
    raise("q must be a bfloat16 tensor [n_rows, Hq, 128] with contiguous rows");
  const int64_t n_rows = q.size(0), stride = n_rows > 1 ? q.stride(0) : q.size(1) * 128;
  const int Hq = dim32(q.size(1), "Hq"), n_kv = to_int(a[2], "n_kv_heads");
  const at::Tensor& table = c.tensor(a[0], "page_table");
  if (table.dim() != 3 || table.size(1) != n_kv) raise("page_table must be [B, Hkv, max_pages]");
  const int B = dim32(table.size(0), "B"), pages = dim32(table.size(2), "max_pages");
  void* t = c.at(a[0], at::kInt, {B, n_kv, pages}, "page_table");
  void* cu = c.at(bounds, at::kInt, {(int64_t)B + 1}, "cu_q");
  void* ctx = c.at(a[1], at::kInt, {B}, "ctx_len");
  const float scale = a[3] == Py_None ? (float)(1.0 / std::sqrt(128.0)) : to_float(a[3]);
  const int causal = PyObject_IsTrue(a[4]);
  bool f32 = PyObject_IsTrue(a[7]) == 1;
  if (a[5] != Py_None) {
    const at::ScalarType type = c.tensor(a[5], "out").scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) raise("out must be bfloat16 or float32");
    f32 = type == at::kFloat;
  }
  void* stream = c.stream(a[9]);
  Out out, lse;
  out.o = c.make(a[5], f32 ? at::kFloat : at::kBFloat16, {n_rows, Hq, 128}, "out", &out.p);
  lse.o = c.make(a[6], at::kFloat, {n_rows, Hq}, "lse", &lse.p);
  const Scratch ws(c, a[8], [&] { return lynx_chunk_attn_workspace_size(n_rows, B, Hq, n_kv, 128); });
  c.launch([&] {
    return call(q.data_ptr(), n_rows, stride, (int32_t*)cu, B, Hq, n_kv, (int32_t*)t, pages, (int32_t*)ctx, scale, causal,
                out.p, f32 ? LYNX_OUT_F32 : LYNX_OUT_BF16, (float*)lse.p, ws.p, ws.bytes, stream);
  });
  return tuple({&out, &lse});
}

// q, cu_q, k_pages, v_pages, page_table, ctx_len, n_kv_heads, sm_scale, causal, out, lse, out is float32, workspace,
// stream
PyObject* chunk_attn_bf16(PyObject* const* a) {
  Call c("lynx_chunk_attn_bf16", a[0], "q");
  const at::Tensor& kp = c.tensor(a[2], "k_pages");
  const int64_t n_pool = kp.dim() == 3 ? kp.size(0) : 0;
  void* k = c.at(a[2], at::kBFloat16, {n_pool, 128, 256}, "k_pages");
  void* v = c.at(a[3], at::kBFloat16, {n_pool, 128, 256}, "v_pages");
  return chunk_attn(c, a[0], a[1], a + 4, [&](auto q, int64_t n_rows, int64_t stride, auto cu, int B, int Hq, int n_kv,
                                              auto... rest) {
    return lynx_chunk_attn_bf16(q, n_rows, stride, cu, B, Hq, n_kv, 128, k, v, n_pool, rest...);
  });
}

// p, q, draft, u, n_draft, tokens, n_accept, stream
PyObject* verify_drafts(PyObject* const* a) {
  Call c("lynx_verify_drafts", a[0], "p");
  const at::Tensor& p = c.tensor(a[0], "p");
  const at::ScalarType type = p.scalar_type();
  if ((type != at::kFloat && type != at::kBFloat16) || p.dim() != 3 || p.size(1) < 2 || (p.size(2) > 1 && p.stride(2) != 1))
    raise("p must be a float32 or bfloat16 tensor [B, T + 1, V] with contiguous rows");
  const int B = dim32(p.size(0), "B"), T = dim32(p.size(1), "T") - 1, V = dim32(p.size(2), "V");
  void* q_at = nullptr;
  int64_t qb = 0, qt = V;
  if (a[1] != Py_None) {
    const at::Tensor& q = c.tensor(a[1], "q");
    if (q.scalar_type() != type || q.dim() != 3 || q.size(0) != B || q.size(1) != T || q.size(2) != V ||
        (V > 1 && q.stride(2) != 1))
      raise("q must be a tensor [B, T, V] of p's type with contiguous rows");
    q_at = q.data_ptr();
    if (B > 1) qb = q.stride(0);
    if (T > 1) qt = q.stride(1);
  }
  void* draft = c.at(a[2], at::kInt, {B, T}, "draft");
  void* u = c.at(a[3], at::kFloat, {B, (int64_t)T + 1}, "u");
  void* n_draft = a[4] == Py_None ? nullptr : c.at(a[4], at::kInt, {B}, "n_draft");
  void* stream = c.stream(a[7]);
  Out tokens, n;
  tokens.o = c.make(a[5], at::kInt, {B, (int64_t)T + 1}, "tokens", &tokens.p);
  n.o = c.make(a[6], at::kInt, {B}, "n_accept", &n.p);
  c.launch([&] {
    return lynx_verify_drafts(p.data_ptr(), B > 1 ? p.stride(0) : 0, p.stride(1), q_at, qb, qt,
                              type == at::kFloat ? LYNX_OUT_F32 : LYNX_OUT_BF16, B, T, V, (int32_t*)draft,
                              (int32_t*)n_draft, (float*)u, (int32_t*)tokens.p, (int32_t*)n.p, stream);
  });
  return tuple({&tokens, &n});
}

// pools of pages in 8 bits and their scales
struct Pools8 {
  void *k, *v, *scales;
  int64_t n;
  Pools8(Call& c, PyObject* k_pages, PyObject* v_pages, PyObject* scale_bytes) {
    const at::Tensor& kp = c.tensor(k_pages, "k_pages");
    n = kp.dim() == 3 ? kp.size(0) : 0;
    k = c.at(k_pages, at::kFloat8_e4m3fn, {n, 256, 128}, "k_pages");
    v = c.at(v_pages, at::kFloat8_e4m3fn, {n, 256, 128}, "v_pages");
    scales = c.at(scale_bytes, at::kByte, {n, 2, 8}, "scales");
  }
};

// q, k_pages, v_pages, scales, page_table, ctx_len, n_kv_heads, sm_scale, causal, out, lse, workspace, stream
PyObject* decode_attn_e4m3(PyObject* const* a) {
  Call c("lynx_decode_attn_e4m3", a[0], "q");
  const at::Tensor& qt = c.tensor(a[0], "q");
  if (qt.dim() != 4) raise("q must be [B, T, Hq, 128]");
  const int64_t b = qt.size(0), t = qt.size(1), hq = qt.size(2);
  void* q = c.at(a[0], at::kBFloat16, {b, t, hq, 128}, "q");
  const int B = dim32(b, "B"), T = dim32(t, "T"), Hq = dim32(hq, "Hq"), n_kv = to_int(a[6], "n_kv_heads");
  const Pools8 pools(c, a[1], a[2], a[3]);
  const at::Tensor& tt = c.tensor(a[4], "page_table");
  if (tt.dim() != 3) raise("page_table must be [B, Hkv, max_pages]");
  const int pages = dim32(tt.size(2), "max_pages");
  void* table = c.at(a[4], at::kInt, {b, n_kv, pages}, "page_table");
  void* ctx = c.at(a[5], at::kInt, {b}, "ctx_len");
  const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt(128.0)) : to_float(a[7]);
  const int causal = PyObject_IsTrue(a[8]);
  void* stream = c.stream(a[12]);
  Out out, lse;
  out.o = c.make(a[9], at::kFloat, {b, t, hq, 128}, "out", &out.p);
  lse.o = c.make(a[10], at::kFloat, {b, t, hq}, "lse", &lse.p);
  const Scratch ws(c, a[11], [&] { return lynx_decode_attn_e4m3_workspace_size(B, T, Hq, n_kv, 128); });
  c.launch([&] {
    return lynx_decode_attn_e4m3(q, B, T, Hq, n_kv, 128, pools.k, pools.v, (uint8_t*)pools.scales, pools.n,
                                 (int32_t*)table, pages, (int32_t*)ctx, scale, causal, (float*)out.p, (float*)lse.p,
                                 ws.p, ws.bytes, stream);
  });
  return tuple({&out, &lse});
}

// qkv, n_q_heads, n_kv_heads, cos_sin, positions, slots, k_pages, v_pages, scales, q_weight, k_weight, norm_eps,
// interleaved, q_out, stream
PyObject* qkv_append_e4m3(PyObject* const* a) {
  Call c("lynx_qkv_append_e4m3", a[0], "qkv");
  const Pools8 pools(c, a[6], a[7], a[8]);
  return append(c, a, a + 9, [&](auto qkv, int64_t n_rows, int64_t stride, int Hq, int Hkv, int D, auto wq, auto wk, float eps,
                                 auto table, int max_pos, int rot, int interleaved, auto pos, auto slots, auto q, auto stream) {
    return lynx_qkv_append_e4m3(qkv, n_rows, stride, Hq, Hkv, D, wq, wk, eps, table, max_pos, rot, interleaved, pos, slots, q,
                                pools.k, pools.v, (uint8_t*)pools.scales, pools.n, stream);
  });
}

// q, cu_q, k_pages, v_pages, scales, page_table, ctx_len, n_kv_heads, sm_scale, causal, out, lse, out is float32,
// workspace, stream
PyObject* chunk_attn_e4m3(PyObject* const* a) {
  Call c("lynx_chunk_attn_e4m3", a[0], "q");
  const Pools8 pools(c, a[2], a[3], a[4]);
  return chunk_attn(c, a[0], a[1], a + 5, [&](auto q, int64_t n_rows, int64_t stride, auto cu, int B, int Hq, int n_kv,
                                              auto... rest) {
    return lynx_chunk_attn_e4m3(q, n_rows, stride, cu, B, Hq, n_kv, 128, pools.k, pools.v, (uint8_t*)pools.scales,
                                pools.n, rest...);
  });
}

// logits, tokens, n_top, logprob, entropy, top_ids, top_logprobs, stream
PyObject* token_logprobs(PyObject* const* a) {
  Call c("lynx_token_logprobs", a[0], "logits");
  const at::Tensor& x = c.tensor(a[0], "logits");
  const at::ScalarType type = x.scalar_type();
  const int64_t dims = x.dim();
  if ((type != at::kFloat && type != at::kBFloat16) || (dims != 2 && dims != 3) ||
      (x.size(dims - 1) > 1 && x.stride(dims - 1) != 1))
    raise("logits must be a float32 or bfloat16 tensor [n_rows, V] or [B, T, V] with contiguous rows");
  const int64_t B = x.size(0), T = dims == 3 ? x.size(1) : 1;
  // rows one stride apart, over both dimensions
  const int64_t stride = dims == 3 && T > 1 ? x.stride(1) : B > 1 ? x.stride(0) : x.size(dims - 1);
  if (dims == 3 && B > 1 && T > 1 && x.stride(0) != T * stride) raise("the rows of logits must lie one stride apart");
  const int V = dim32(x.size(dims - 1), "V"), n_top = to_int(a[2], "n_top");
  if (n_top < 0) raise("n_top must not be negative");
  auto shape = [&](int64_t more) {
    at::DimVector s(x.sizes().begin(), x.sizes().end() - 1);
    if (more >= 0) s.push_back(more);
    return s;
  };
  const at::DimVector rows = shape(-1), tops = shape(n_top);
  void* tokens = c.at(a[1], at::kInt, rows, "tokens");
  void* stream = c.stream(a[7]);
  Out lp, h, ids, top;
  lp.o = c.make(a[3], at::kFloat, rows, "logprob", &lp.p);
  h.o = c.make(a[4], at::kFloat, rows, "entropy", &h.p);
  ids.o = c.make(a[5], at::kInt, tops, "top_ids", &ids.p);
  top.o = c.make(a[6], at::kFloat, tops, "top_logprobs", &top.p);
  c.launch([&] {
    return lynx_token_logprobs(x.data_ptr(), stride, type == at::kFloat ? LYNX_OUT_F32 : LYNX_OUT_BF16, B * T, V,
                               (int32_t*)tokens, n_top, (float*)lp.p, (float*)h.p, (int32_t*)ids.p, (float*)top.p, stream);
  });
  return tuple({&lp, &h, &ids, &top});
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {
    {"set_error", set_error, METH_O, nullptr},
    {"assign_pages", FAST((entry<11, assign_pages>))},
    {"qkv_append", FAST((entry<14, qkv_append>))},
    {"chunk_attn_bf16", FAST((entry<14, chunk_attn_bf16>))},
    {"verify_drafts", FAST((entry<8, verify_drafts>))},
    {"decode_attn_e4m3", FAST((entry<13, decode_attn_e4m3>))},
    {"chunk_attn_e4m3", FAST((entry<15, chunk_attn_e4m3>))},
    {"qkv_append_e4m3", FAST((entry<15, qkv_append_e4m3>))},
    {"token_logprobs", FAST((entry<8, token_logprobs>))},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "lynx_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit_lynx_binding() { return PyModule_Create(&kModule); }
