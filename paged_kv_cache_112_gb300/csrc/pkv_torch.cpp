// Marshalling of torch tensors into the layer operators of the C ABI
// (include/pkv.h): the checks of dtype, shape, strides and device and the
// call itself, as a CPython extension.
//
// These operators run once or more per layer and step, some for a few
// microseconds, so what a call costs the host counts: reading a dozen tensors'
// attributes from Python and converting 30 arguments with ctypes took 15 to
// 25 us a call on the GB300's host cores, this takes 2 to 3 us, most of it the
// launch.  Nothing is computed, kept or allocated here.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "pkv.h"

namespace {

PyObject* g_error = nullptr;  // PkvError, set by the package

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

// A positional argument that must be a CUDA tensor on `device` (or None, when optional: nullptr).
const at::Tensor* tensor(PyObject* o, const char* name, int device, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != device)
    throw Refused(std::string(name) + " must be a CUDA tensor on the current device");
  return &t;
}

void need(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

const at::Tensor* dense(const at::Tensor* t, const char* name, at::ScalarType type) {
  if (t) {
    if (t->scalar_type() != type) throw Refused(std::string(name) + " must be " + c10::toString(type));
    if (!t->is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  }
  return t;
}

const at::Tensor* int32s(PyObject* o, const char* name, int device, bool optional = false) {
  return dense(tensor(o, name, device, optional), name, at::kInt);
}

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T* ptr_of(const at::Tensor* t) {
  return static_cast<T*>(ptr(t));
}

int size(const at::Tensor& t, int d) {
  const int64_t n = t.size(d);
  need(n <= 0x7fffffff, "a tensor's dimension does not fit 32 bits");
  return static_cast<int>(n);
}

pkv_dtype value_dtype(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return PKV_F16;
  if (t.scalar_type() == at::kBFloat16) return PKV_BF16;
  throw Refused("new rows, queries and 16-bit pools must be float16 or bfloat16");
}

pkv_dtype out_dtype(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? PKV_F32 : value_dtype(t); }

// Geometry of a K pool (and its V pool): 16-bit [NB, B, H, D] with dense
// blocks `stride` elements apart, or FP8 codes (uint8) with their scales
// [NB, H] and `layers` blocks of the same size between consecutive ones.
struct Pool {
  int NB, B, H, D, layers = 1;
  int64_t stride;
};

Pool pool_of(const at::Tensor& k, const at::Tensor* v, const at::Tensor* ks, const at::Tensor* vs, bool fp8) {
  need(k.dim() == 4, "pools must be [NB, block_size, H_kv, D]");
  Pool p{size(k, 0), size(k, 1), size(k, 2), size(k, 3)};
  const int64_t row = static_cast<int64_t>(p.H) * p.D, block = row * p.B;
  need(k.stride(3) == 1 && k.stride(2) == p.D && k.stride(1) == row && k.stride(0) >= block,
       "pool blocks must be dense [block_size, H_kv, D] slices");
  p.stride = k.stride(0);
  if (v) {
    need(v->sizes() == k.sizes() && v->strides() == k.strides() && v->scalar_type() == k.scalar_type(),
         "k_pool and v_pool must share shape, strides and dtype");
  }
  if (!fp8) {
    value_dtype(k);
    return p;
  }
  need(k.scalar_type() == at::kByte, "FP8 pools must be uint8 tensors of e4m3 codes");
  need(block > 0 && p.stride % block == 0 && p.stride / block <= 0x7fffffff,
       "FP8 pool blocks must be whole blocks apart");
  p.layers = static_cast<int>(p.stride / block);
  for (const at::Tensor* sc : {ks, vs})
    if (sc)
      need(sc->scalar_type() == at::kFloat && sc->dim() == 2 && sc->size(0) == p.NB && sc->size(1) == p.H &&
               sc->stride(1) == 1 && sc->stride(0) == static_cast<int64_t>(p.layers) * p.H,
           "scales must be float32 [NB, H_kv] with the pools' layer count");
  return p;
}

// A 4-bit pool of records, uint8 [NB, H, B / 16, 9 D], with dense blocks.
Pool pool4_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor* ks, const at::Tensor* vs) {
  need(k.scalar_type() == at::kByte && k.dim() == 4 && k.size(3) % 9 == 0,
       "4-bit pools must be uint8 [NB, H_kv, block_size / 16, 9 * D]");
  need(k.size(2) <= 4, "4-bit pool blocks hold 16, 32 or 64 tokens");
  Pool p{size(k, 0), size(k, 2) * 16, size(k, 1), size(k, 3) / 9};
  const int64_t tiles = k.size(2) * k.size(3), block = tiles * p.H;
  need(k.stride(3) == 1 && k.stride(2) == k.size(3) && k.stride(1) == tiles && k.stride(0) >= block,
       "4-bit pool blocks must be dense [H_kv, block_size / 16, 9 * D] slices");
  need(v.sizes() == k.sizes() && v.strides() == k.strides() && v.scalar_type() == at::kByte,
       "k_pool and v_pool must share shape, strides and dtype");
  need(block > 0 && k.stride(0) % block == 0 && k.stride(0) / block <= 0x7fffffff,
       "4-bit pool blocks must be whole blocks apart");
  p.layers = static_cast<int>(k.stride(0) / block);
  p.stride = k.stride(0);
  for (const at::Tensor* sc : {ks, vs})
    if (sc)
      need(sc->scalar_type() == at::kFloat && sc->dim() == 1 && sc->size(0) == p.H && sc->is_contiguous(),
           "scales of 4-bit pools must be float32 [H_kv]");
  return p;
}

// Row stride of [T, heads, D] rows, dense within a token; 0 where one row or none makes it meaningless.
int64_t rows(const at::Tensor* t, int64_t T, int64_t heads, int64_t D, at::ScalarType type, const char* name) {
  if (!t) return 0;
  if (t->dim() != 3 || t->size(0) != T || t->size(1) != heads || t->size(2) != D || t->scalar_type() != type)
    throw Refused(std::string(name) + " must be [T, heads, D] of the queries' dtype");
  if (T == 0) return 0;
  if (t->stride(2) != 1 || (heads > 1 && t->stride(1) != D))
    throw Refused(std::string(name) + " must have dense rows");
  if (T == 1) return 0;
  if (t->stride(0) < heads * D) throw Refused(std::string(name) + ": rows of consecutive tokens overlap");
  return t->stride(0);
}

void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* n = PyObject_GetAttrString(o, "cuda_stream");
  void* s = n ? PyLong_AsVoidPtr(n) : nullptr;
  Py_XDECREF(n);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused("stream must be a torch.cuda.Stream");
  }
  return s;
}

int integer(PyObject* o, const char* name) {
  PyObject* n = PyNumber_Index(o);
  const long long v = n ? PyLong_AsLongLong(n) : -1;
  Py_XDECREF(n);
  if (PyErr_Occurred() || v < -0x7fffffffLL || v > 0x7fffffffLL) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be an integer of 32 bits");
  }
  return static_cast<int>(v);
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be true or false");
  }
  return v == 1;
}

void done(pkv_status st, const char* what) {
  if (st == PKV_OK) return;
  std::string text = std::string(what) + ": " + pkv_status_string(st);
  if (st == PKV_ERR_CUDA) {
    const int code = pkv_last_cuda_error();
    text += std::string(" (") + pkv_cuda_error_name(code) + ", code " + std::to_string(code) + ")";
  }
  throw Refused(text);
}

// Runs `call` with every C++ exception turned into a PkvError.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F call) {
  try {
    need(got == want, "wrong number of arguments");
    call(static_cast<int>(c10::cuda::current_device()));
    Py_RETURN_NONE;
  } catch (const c10::Error& e) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// (q, k, v, k_pool, v_pool, k_scale, v_scale, slot_mapping, q_out, k_out, q_weight, k_weight, eps, cos_sin,
//  positions, interleaved, status, stream, bits)
PyObject* norm_rope_write(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 19, [&](int dev) {
    const int bits = integer(o[18], "bits");
    const bool fp8 = bits == 8;
    const at::Tensor &q = *tensor(o[0], "q", dev), &k = *tensor(o[1], "k", dev), &v = *tensor(o[2], "v", dev);
    const at::Tensor &kp = *tensor(o[3], "k_pool", dev), &vp = *tensor(o[4], "v_pool", dev);
    const at::Tensor *ks = tensor(o[5], "k_scale", dev, !fp8), *vs = tensor(o[6], "v_scale", dev, !fp8);
    const at::Tensor& slots = *int32s(o[7], "slot_mapping", dev);
    const at::Tensor& q_out = *tensor(o[8], "q_out", dev);
    const at::Tensor* k_out = tensor(o[9], "k_out", dev, true);
    const at::Tensor *qw = tensor(o[10], "q_weight", dev, true), *kw = tensor(o[11], "k_weight", dev, true);
    const at::Tensor* cs = dense(tensor(o[13], "cos_sin", dev, true), "cos_sin", at::kFloat);
    const at::Tensor* pos = int32s(o[14], "positions", dev, true);
    const at::Tensor* status = int32s(o[16], "status", dev, true);
    const Pool p = bits == 4 ? pool4_of(kp, vp, ks, vs) : pool_of(kp, &vp, ks, vs, fp8);
    const pkv_dtype dt = value_dtype(q);
    const at::ScalarType type = q.scalar_type();
    need(bits != 16 || kp.scalar_type() == type, "rows and pools must share a dtype");
    need(q.dim() == 3, "q must be [T, H_q, D]");
    const int T = size(q, 0), Hq = size(q, 1);
    const int64_t qs = rows(&q, T, Hq, p.D, type, "q"), qos = rows(&q_out, T, Hq, p.D, type, "q_out");
    const int64_t kvs = rows(&k, T, p.H, p.D, type, "k");
    need(rows(&v, T, p.H, p.D, type, "v") == kvs, "k and v must share a row stride");
    const int64_t kos = rows(k_out, T, p.H, p.D, type, "k_out");
    for (const at::Tensor* w : {qw, kw})
      if (w)
        need(w->scalar_type() == type && w->dim() == 1 && w->size(0) == p.D && w->is_contiguous(),
             "norm weights must be [D] of the rows' dtype");
    need(slots.dim() == 1 && slots.size(0) == T, "slot_mapping must be int32 [T]");
    int top = 0, rot = 0;
    if (cs) {
      need(cs->dim() == 2 && pos, "cos_sin must be float32 [max_positions, rot_dim], with int32 positions [T]");
      top = size(*cs, 0);
      rot = size(*cs, 1);
    }
    need(!pos || (pos->dim() == 1 && pos->size(0) == T), "positions must be int32 [T]");
    const float eps = number(o[12], "eps");
    const bool inter = truth(o[15], "interleaved");
    void* stream = stream_of(o[17], dev);
    if (bits == 4)
      done(pkv_norm_rope_write_fp4(ptr(&q_out), qos, ptr(k_out), kos, ptr(&q), qs, ptr(&k), ptr(&v), kvs, ptr(qw),
                                   ptr(kw), eps, ptr_of<float>(cs), ptr_of<int32_t>(pos), top, rot, inter, ptr(&kp),
                                   ptr(&vp), ptr_of<float>(ks), ptr_of<float>(vs), ptr_of<int32_t>(&slots), T, Hq, p.H,
                                   p.D, p.B, p.NB, p.layers, dt, ptr_of<int32_t>(status), stream),
           "pkv_norm_rope_write_fp4");
    else if (fp8)
      done(pkv_norm_rope_write_fp8(ptr(&q_out), qos, ptr(k_out), kos, ptr(&q), qs, ptr(&k), ptr(&v), kvs, ptr(qw),
                                   ptr(kw), eps, ptr_of<float>(cs), ptr_of<int32_t>(pos), top, rot, inter, ptr(&kp),
                                   ptr(&vp), ptr_of<float>(ks), ptr_of<float>(vs), ptr_of<int32_t>(&slots), T, Hq, p.H,
                                   p.D, p.B, p.NB, p.layers, dt, ptr_of<int32_t>(status), stream),
           "pkv_norm_rope_write_fp8");
    else
      done(pkv_norm_rope_write(ptr(&q_out), qos, ptr(k_out), kos, ptr(&q), qs, ptr(&k), ptr(&v), kvs, ptr(qw), ptr(kw),
                               eps, ptr_of<float>(cs), ptr_of<int32_t>(pos), top, rot, inter, ptr(&kp), ptr(&vp),
                               p.stride, ptr_of<int32_t>(&slots), T, Hq, p.H, p.D, p.B, p.NB, dt,
                               ptr_of<int32_t>(status), stream),
           "pkv_norm_rope_write");
  });
}

// Blocks, KV heads and head dim of a summary and its scales.
struct Summary {
  int NB, H, D;
};

Summary summary_of(const at::Tensor& s, const at::Tensor& sc) {
  need(s.dim() == 4 && s.size(2) == 2 && sc.dim() == 2 && sc.size(0) == s.size(0) && sc.size(1) == s.size(1),
       "summary must be int8 [NB, H_kv, 2, D] and summary_scale float32 [NB, H_kv]");
  return Summary{size(s, 0), size(s, 1), size(s, 3)};
}

// (summary, summary_scale, k_pool, k_scale, block_ids, status, stream, fp8)
PyObject* summarize_blocks(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 8, [&](int dev) {
    const bool fp8 = o[7] == Py_True;
    const at::Tensor& s = *dense(tensor(o[0], "summary", dev), "summary", at::kChar);
    const at::Tensor& sc = *dense(tensor(o[1], "summary_scale", dev), "summary_scale", at::kFloat);
    const at::Tensor& kp = *tensor(o[2], "k_pool", dev);
    const at::Tensor* ks = tensor(o[3], "k_scale", dev, !fp8);
    const at::Tensor& ids = *int32s(o[4], "block_ids", dev);
    const at::Tensor* status = int32s(o[5], "status", dev, true);
    const Pool p = pool_of(kp, nullptr, ks, nullptr, fp8);
    const Summary m = summary_of(s, sc);
    need(m.NB == p.NB && m.H == p.H && m.D == p.D, "summary must have the pool's blocks, KV heads and head dim");
    need(ids.dim() == 1, "block_ids must be int32 [n]");
    void* stream = stream_of(o[6], dev);
    if (fp8)
      done(pkv_summarize_blocks_fp8(ptr(&s), ptr_of<float>(&sc), ptr(&kp), ptr_of<float>(ks), ptr_of<int32_t>(&ids),
                                    size(ids, 0), p.H, p.D, p.B, p.NB, p.layers, ptr_of<int32_t>(status), stream),
           "pkv_summarize_blocks_fp8");
    else
      done(pkv_summarize_blocks(ptr(&s), ptr_of<float>(&sc), ptr(&kp), p.stride, ptr_of<int32_t>(&ids), size(ids, 0),
                                p.H, p.D, p.B, p.NB, value_dtype(kp), ptr_of<int32_t>(status), stream),
           "pkv_summarize_blocks");
  });
}

void lists(const at::Tensor& selected, const at::Tensor& counts, const at::Tensor& tables, const at::Tensor& lens,
           int64_t S, int64_t H) {
  need(selected.dim() == 3 && selected.size(0) == S && selected.size(1) == H && counts.dim() == 2 &&
           counts.size(0) == S && counts.size(1) == H && tables.dim() == 2 && tables.size(0) == S && lens.dim() == 1 &&
           lens.size(0) == S,
       "selected [S, H_kv, keep], counts [S, H_kv], block_tables [S, blocks] and context_lens [S] are needed");
}

// (selected, counts, q, summary, summary_scale, block_tables, context_lens, block_size, first_blocks, last_blocks,
//  max_context_len, status, stream)
PyObject* select_blocks(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 13, [&](int dev) {
    const at::Tensor &sel = *int32s(o[0], "selected", dev), &cnt = *int32s(o[1], "counts", dev);
    const at::Tensor& q = *tensor(o[2], "q", dev);
    const at::Tensor& s = *dense(tensor(o[3], "summary", dev), "summary", at::kChar);
    const at::Tensor& sc = *dense(tensor(o[4], "summary_scale", dev), "summary_scale", at::kFloat);
    const at::Tensor &bt = *int32s(o[5], "block_tables", dev), &cl = *int32s(o[6], "context_lens", dev);
    const at::Tensor* status = int32s(o[11], "status", dev, true);
    const Summary m = summary_of(s, sc);
    const pkv_dtype dt = value_dtype(q);
    need(q.dim() == 3 && q.size(2) == m.D && q.is_contiguous(), "q must be contiguous [S, H_q, D] with the summary's D");
    const int S = size(q, 0);
    lists(sel, cnt, bt, cl, S, m.H);
    done(pkv_select_blocks(ptr_of<int32_t>(&sel), ptr_of<int32_t>(&cnt), ptr(&q), ptr(&s), ptr_of<float>(&sc),
                           ptr_of<int32_t>(&bt), size(bt, 1), ptr_of<int32_t>(&cl), S, size(q, 1), m.H, m.D,
                           integer(o[7], "block_size"), m.NB, size(sel, 2), integer(o[8], "first_blocks"),
                           integer(o[9], "last_blocks"), integer(o[10], "max_context_len"), dt,
                           ptr_of<int32_t>(status), stream_of(o[12], dev)),
         "pkv_select_blocks");
  });
}

// (out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, selected, counts, scale, max_context_len,
//  status, stream, fp8)
PyObject* decode_sparse(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 15, [&](int dev) {
    const bool fp8 = o[14] == Py_True;
    const at::Tensor &out = *tensor(o[0], "out", dev), &q = *tensor(o[1], "q", dev);
    const at::Tensor &kp = *tensor(o[2], "k_pool", dev), &vp = *tensor(o[3], "v_pool", dev);
    const at::Tensor *ks = tensor(o[4], "k_scale", dev, !fp8), *vs = tensor(o[5], "v_scale", dev, !fp8);
    const at::Tensor &bt = *int32s(o[6], "block_tables", dev), &cl = *int32s(o[7], "context_lens", dev);
    const at::Tensor &sel = *int32s(o[8], "selected", dev), &cnt = *int32s(o[9], "counts", dev);
    const at::Tensor* status = int32s(o[12], "status", dev, true);
    const Pool p = pool_of(kp, &vp, ks, vs, fp8);
    const pkv_dtype dt = value_dtype(q), od = out_dtype(out);
    need(fp8 || kp.scalar_type() == q.scalar_type(), "q, k_pool and v_pool must share a dtype");
    need(q.dim() == 3 && q.size(2) == p.D && q.is_contiguous() && out.sizes() == q.sizes() && out.is_contiguous(),
         "q and out must be contiguous [S, H_q, D] with the pools' D");
    const int S = size(q, 0), Hq = size(q, 1);
    lists(sel, cnt, bt, cl, S, p.H);
    const float scale = number(o[10], "scale");
    const int longest = integer(o[11], "max_context_len");
    void* stream = stream_of(o[13], dev);
    if (fp8)
      done(pkv_decode_sparse_fp8(ptr(&out), ptr(&q), ptr(&kp), ptr(&vp), ptr_of<float>(ks), ptr_of<float>(vs),
                                 ptr_of<int32_t>(&bt), size(bt, 1), ptr_of<int32_t>(&cl), ptr_of<int32_t>(&sel),
                                 ptr_of<int32_t>(&cnt), size(sel, 2), S, Hq, p.H, p.D, p.B, p.NB, p.layers, scale,
                                 longest, dt, od, ptr_of<int32_t>(status), stream),
           "pkv_decode_sparse_fp8");
    else
      done(pkv_decode_sparse(ptr(&out), ptr(&q), ptr(&kp), ptr(&vp), p.stride, ptr_of<int32_t>(&bt), size(bt, 1),
                             ptr_of<int32_t>(&cl), ptr_of<int32_t>(&sel), ptr_of<int32_t>(&cnt), size(sel, 2), S, Hq,
                             p.H, p.D, p.B, p.NB, scale, longest, dt, od, ptr_of<int32_t>(status), stream),
           "pkv_decode_sparse");
  });
}

// (k_new, v_new, k_pool, v_pool, k_scale, v_scale, slot_mapping, status, stream)
PyObject* write_cache_fp4(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 9, [&](int dev) {
    const at::Tensor &k = *tensor(o[0], "k_new", dev), &v = *tensor(o[1], "v_new", dev);
    const at::Tensor &kp = *tensor(o[2], "k_pool", dev), &vp = *tensor(o[3], "v_pool", dev);
    const at::Tensor *ks = tensor(o[4], "k_scale", dev, true), *vs = tensor(o[5], "v_scale", dev, true);
    const at::Tensor& slots = *int32s(o[6], "slot_mapping", dev);
    const at::Tensor* status = int32s(o[7], "status", dev, true);
    const Pool p = pool4_of(kp, vp, ks, vs);
    const pkv_dtype dt = value_dtype(k);
    need(k.dim() == 3, "k_new must be [T, H_kv, D]");
    const int T = size(k, 0);
    const int64_t kvs = rows(&k, T, p.H, p.D, k.scalar_type(), "k_new");
    need(rows(&v, T, p.H, p.D, k.scalar_type(), "v_new") == kvs, "k_new and v_new must share a row stride");
    need(slots.dim() == 1 && slots.size(0) == T, "slot_mapping must be int32 [T]");
    done(pkv_write_cache_fp4(ptr(&k), ptr(&v), ptr(&kp), ptr(&vp), ptr_of<float>(ks), ptr_of<float>(vs),
                             ptr_of<int32_t>(&slots), T, kvs, p.H, p.D, p.B, p.NB, p.layers, dt,
                             ptr_of<int32_t>(status), stream_of(o[8], dev)),
         "pkv_write_cache_fp4");
  });
}

// (k_pool, v_pool, pairs, status, stream): whole pools, [NB, H, tiles, 9 D] or [NB, layers, H, tiles, 9 D]
PyObject* copy_blocks_fp4(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 5, [&](int dev) {
    const at::Tensor &kp = *tensor(o[0], "k_pool", dev), &vp = *tensor(o[1], "v_pool", dev);
    const at::Tensor& pairs = *int32s(o[2], "pairs", dev);
    const at::Tensor* status = int32s(o[3], "status", dev, true);
    const bool all = kp.dim() == 5;
    need(kp.scalar_type() == at::kByte && (kp.dim() == 4 || all) && kp.is_contiguous() && kp.size(-1) % 9 == 0 &&
             kp.size(-2) <= 4 && vp.is_contiguous() && vp.sizes() == kp.sizes() && vp.scalar_type() == at::kByte,
         "4-bit pools must be contiguous uint8 [NB, (layers,) H_kv, block_size / 16, 9 * D]");
    need(pairs.dim() == 2 && pairs.size(1) == 2, "pairs must be int32 [P, 2]");
    done(pkv_copy_blocks_fp4(ptr(&kp), ptr(&vp), ptr_of<int32_t>(&pairs), size(pairs, 0), all ? size(kp, 1) : 1,
                             size(kp, kp.dim() - 3), size(kp, kp.dim() - 1) / 9, size(kp, kp.dim() - 2) * 16,
                             size(kp, 0), ptr_of<int32_t>(status), stream_of(o[4], dev)),
         "pkv_copy_blocks_fp4");
  });
}

// What the decode calls over a whole or windowed history share.
struct Rows {
  int S, Hq;
  pkv_dtype dt, od;
};
Rows rows_of(const at::Tensor& out, const at::Tensor& q, const at::Tensor& bt, const at::Tensor& cl, const Pool& p) {
  need(q.dim() == 3 && q.size(2) == p.D && q.is_contiguous() && out.sizes() == q.sizes() && out.is_contiguous(),
       "q and out must be contiguous [S, H_q, D] with the pools' D");
  Rows r{size(q, 0), size(q, 1), value_dtype(q), out_dtype(out)};
  need(bt.dim() == 2 && bt.size(0) == r.S && cl.dim() == 1 && cl.size(0) == r.S,
       "block_tables [S, blocks] and context_lens [S] are needed");
  return r;
}

// (out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale, partition_size, max_context_len,
//  workspace, status, stream)
PyObject* decode_attention_fp4(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 14, [&](int dev) {
    const at::Tensor &out = *tensor(o[0], "out", dev), &q = *tensor(o[1], "q", dev);
    const at::Tensor &kp = *tensor(o[2], "k_pool", dev), &vp = *tensor(o[3], "v_pool", dev);
    const at::Tensor *ks = tensor(o[4], "k_scale", dev, true), *vs = tensor(o[5], "v_scale", dev, true);
    const at::Tensor &bt = *int32s(o[6], "block_tables", dev), &cl = *int32s(o[7], "context_lens", dev);
    const at::Tensor* ws = tensor(o[11], "workspace", dev, true);
    const at::Tensor* status = int32s(o[12], "status", dev, true);
    const Pool p = pool4_of(kp, vp, ks, vs);
    const Rows r = rows_of(out, q, bt, cl, p);
    need(!ws || ws->is_contiguous(), "workspace must be contiguous");
    done(pkv_decode_attention_fp4(ptr(&out), ptr(&q), ptr(&kp), ptr(&vp), ptr_of<float>(ks), ptr_of<float>(vs),
                                  ptr_of<int32_t>(&bt), size(bt, 1), ptr_of<int32_t>(&cl), r.S, r.Hq, p.H, p.D, p.B,
                                  p.NB, p.layers, number(o[8], "scale"), integer(o[9], "partition_size"),
                                  integer(o[10], "max_context_len"), ptr(ws), ws ? ws->nbytes() : 0, r.dt, r.od,
                                  ptr_of<int32_t>(status), stream_of(o[13], dev)),
         "pkv_decode_attention_fp4");
  });
}

// (out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale, window, sinks, max_context_len,
//  status, stream, bits)
PyObject* decode_window(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 15, [&](int dev) {
    const bool fp4 = integer(o[14], "bits") == 4;
    const at::Tensor &out = *tensor(o[0], "out", dev), &q = *tensor(o[1], "q", dev);
    const at::Tensor &kp = *tensor(o[2], "k_pool", dev), &vp = *tensor(o[3], "v_pool", dev);
    const at::Tensor *ks = tensor(o[4], "k_scale", dev, true), *vs = tensor(o[5], "v_scale", dev, true);
    const at::Tensor &bt = *int32s(o[6], "block_tables", dev), &cl = *int32s(o[7], "context_lens", dev);
    const at::Tensor* status = int32s(o[12], "status", dev, true);
    const Pool p = fp4 ? pool4_of(kp, vp, ks, vs) : pool_of(kp, &vp, nullptr, nullptr, false);
    const Rows r = rows_of(out, q, bt, cl, p);
    need(fp4 || kp.scalar_type() == q.scalar_type(), "q, k_pool and v_pool must share a dtype");
    const float scale = number(o[8], "scale");
    const int window = integer(o[9], "window"), sinks = integer(o[10], "sinks");
    const int longest = integer(o[11], "max_context_len");
    void* stream = stream_of(o[13], dev);
    if (fp4)
      done(pkv_decode_window_fp4(ptr(&out), ptr(&q), ptr(&kp), ptr(&vp), ptr_of<float>(ks), ptr_of<float>(vs),
                                 ptr_of<int32_t>(&bt), size(bt, 1), ptr_of<int32_t>(&cl), r.S, r.Hq, p.H, p.D, p.B,
                                 p.NB, p.layers, scale, window, sinks, longest, r.dt, r.od, ptr_of<int32_t>(status),
                                 stream),
           "pkv_decode_window_fp4");
    else
      done(pkv_decode_window(ptr(&out), ptr(&q), ptr(&kp), ptr(&vp), p.stride, ptr_of<int32_t>(&bt), size(bt, 1),
                             ptr_of<int32_t>(&cl), r.S, r.Hq, p.H, p.D, p.B, p.NB, scale, window, sinks, longest, r.dt,
                             r.od, ptr_of<int32_t>(status), stream),
           "pkv_decode_window");
  });
}

// (out, q, k_pool, v_pool, block_tables, context_lens, query_start, scale, window, sinks, max_context_len, status,
//  stream)
PyObject* prefill_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 13, [&](int dev) {
    const at::Tensor &out = *tensor(o[0], "out", dev), &q = *tensor(o[1], "q", dev);
    const at::Tensor &kp = *tensor(o[2], "k_pool", dev), &vp = *tensor(o[3], "v_pool", dev);
    const at::Tensor &bt = *int32s(o[4], "block_tables", dev), &cl = *int32s(o[5], "context_lens", dev);
    const at::Tensor& qs = *int32s(o[6], "query_start", dev);
    const at::Tensor* status = int32s(o[11], "status", dev, true);
    const Pool p = pool_of(kp, &vp, nullptr, nullptr, false);
    need(kp.scalar_type() == q.scalar_type(), "q, k_pool and v_pool must share a dtype");
    need(q.dim() == 3, "q must be [T, H_q, D]");
    const int T = size(q, 0), Hq = size(q, 1);
    const int64_t stride = rows(&q, T, Hq, p.D, q.scalar_type(), "q");
    need(out.sizes() == q.sizes() && out.is_contiguous(), "out must be contiguous [T, H_q, D]");
    need(bt.dim() == 2 && cl.dim() == 1 && cl.size(0) == bt.size(0) && qs.dim() == 1 && qs.size(0) == bt.size(0) + 1,
         "block_tables [S, blocks], context_lens [S] and query_start [S + 1] are needed");
    done(pkv_prefill_attention(ptr(&out), ptr(&q), stride, ptr(&kp), ptr(&vp), p.stride, ptr_of<int32_t>(&bt),
                               size(bt, 1), ptr_of<int32_t>(&cl), ptr_of<int32_t>(&qs), size(bt, 0), T, Hq, p.H, p.D,
                               p.B, p.NB, number(o[7], "scale"), integer(o[8], "window"), integer(o[9], "sinks"),
                               integer(o[10], "max_context_len"), value_dtype(q), out_dtype(out),
                               ptr_of<int32_t>(status), stream_of(o[12], dev)),
         "pkv_prefill_attention");
  });
}

PyObject* set_error_type(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"norm_rope_write", fast(norm_rope_write), METH_FASTCALL, nullptr},
    {"summarize_blocks", fast(summarize_blocks), METH_FASTCALL, nullptr},
    {"select_blocks", fast(select_blocks), METH_FASTCALL, nullptr},
    {"decode_sparse", fast(decode_sparse), METH_FASTCALL, nullptr},
    {"write_cache_fp4", fast(write_cache_fp4), METH_FASTCALL, nullptr},
    {"copy_blocks_fp4", fast(copy_blocks_fp4), METH_FASTCALL, nullptr},
    {"decode_attention_fp4", fast(decode_attention_fp4), METH_FASTCALL, nullptr},
    {"decode_window", fast(decode_window), METH_FASTCALL, nullptr},
    {"prefill_attention", fast(prefill_attention), METH_FASTCALL, nullptr},
    {"set_error_type", set_error_type, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch(void) {
  PyObject* m = PyModule_Create(&kModule);
  // The torch it was compiled against (build.py): another one's tensors may be laid out differently.
  if (m && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
