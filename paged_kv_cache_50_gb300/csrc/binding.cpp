// The argument checks of the serving-step calls, and of those over 4-bit pools, weights'
// sums, evictions and whole prompts, compiled.
//
// A step's small calls (a plan of 64 requests, the norms of 64 tokens) run for 2
// to 3 us on the GPU, and reading type, device, layout and address of a dozen
// tensors from Python costs more than that: a pa_plan_step call took 9.8 us of
// host time and takes 2.5 with these checks, 1.5 of them the launch.  Each
// function here takes one entry point's arguments as they come from
// paged_kv_cache_50_gb300/__init__.py, checks every tensor (TypeError,
// ValueError), calls the entry point and returns its status.  Nothing is computed
// or kept here.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdarg.h>

#include "pa.h"

namespace {

// A refused argument: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
  va_list v;
  va_start(v, format);
  PyErr_FormatV(type, format, v);
  va_end(v);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    default: return "torch.uint8";
  }
}

void same_device(long long dev, long long current, const char* name) {
  if (dev != current)
    refuse(PyExc_ValueError, "%s is on cuda:%lld, the current device is cuda:%lld", name, dev,
           current);
}

// The call's device: that of `t`, which must be the current one.
int call_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  const int dev = t.get_device();
  same_device(dev, c10::cuda::current_device(), name);
  return dev;
}

// Device and type of a tensor on CUDA device `dev`.
void check(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type),
           at::toString(t.scalar_type()));
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, "%s must be on cuda:%d, is on %s", name, dev,
           t.device().str().c_str());
}

void* dense(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
  check(t, name, type, dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}

// A dense tensor of the given shape.
void* shaped(PyObject* o, const char* name, at::ScalarType type, int dev,
             std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name);
  if (!t.sizes().equals(at::IntArrayRef(shape.begin(), shape.size()))) {
    std::string want, is;
    for (int64_t s : shape) want += (want.empty() ? "" : ", ") + std::to_string(s);
    for (int64_t s : t.sizes()) is += (is.empty() ? "" : ", ") + std::to_string(s);
    refuse(PyExc_ValueError, "%s must be [%s], is [%s]", name, want.c_str(), is.c_str());
  }
  return dense(t, name, type, dev);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int integer32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v != static_cast<int>(v)) refuse(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int>(v);
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}

int extent(int64_t v, const char* name) {
  if (v != static_cast<int>(v)) refuse(PyExc_ValueError, "%s is too large", name);
  return static_cast<int>(v);
}

void* pointer(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Refused();
  return p;
}

// A stream handle; None: the current stream.
void* stream_of(PyObject* o, int dev) {
  return o == Py_None ? c10::cuda::getCurrentCUDAStream(dev).stream() : pointer(o);
}

// Entry points of the loaded library.
decltype(&pa_plan_step) plan_step_fn;
decltype(&pa_qk_norm_rope_cache) norm_fn;
decltype(&pa_qk_norm_rope_cache_fp8) norm_fp8_fn;
decltype(&pa_varlen_fwd_sinks) sinks_fn;
decltype(&pa_decode_window) window_fn;
decltype(&pa_decode_window_fp8) window_fp8_fn;
decltype(&pa_reshape_and_cache_fp4) write_fp4_fn;
decltype(&pa_decode_fp4) decode_fp4_fn;
decltype(&pa_decode_scores) scores_fn;
decltype(&pa_decode_scores_fp4) scores_fp4_fn;
decltype(&pa_evict) evict_fn;
decltype(&pa_evict_fp4) evict_fp4_fn;
decltype(&pa_prompt_fwd) prompt_fn;

// The library call itself, without the interpreter's lock: a launch waits where
// the stream's queue is full, and what it waits for may need another thread of the
// interpreter.  The arguments are taken beforehand.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class... P, class... A>
PyObject* call(pa_status (*f)(P...), A... args) {
  pa_status status;
  {
    Unlocked unlocked;
    status = f(args...);
  }
  return PyLong_FromLong(status);
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) refuse(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// (device, current device, name): raises unless they agree.
PyObject* check_device(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const char* name = PyUnicode_AsUTF8(a[2]);
    if (name == nullptr) throw Refused();
    same_device(integer(a[0]), integer(a[1]), name);
    Py_RETURN_NONE;
  });
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    plan_step_fn = reinterpret_cast<decltype(plan_step_fn)>(pointer(a[0]));
    norm_fn = reinterpret_cast<decltype(norm_fn)>(pointer(a[1]));
    norm_fp8_fn = reinterpret_cast<decltype(norm_fp8_fn)>(pointer(a[2]));
    sinks_fn = reinterpret_cast<decltype(sinks_fn)>(pointer(a[3]));
    window_fn = reinterpret_cast<decltype(window_fn)>(pointer(a[4]));
    window_fp8_fn = reinterpret_cast<decltype(window_fp8_fn)>(pointer(a[5]));
    Py_RETURN_NONE;
  });
}

PyObject* bind_more(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    write_fp4_fn = reinterpret_cast<decltype(write_fp4_fn)>(pointer(a[0]));
    decode_fp4_fn = reinterpret_cast<decltype(decode_fp4_fn)>(pointer(a[1]));
    scores_fn = reinterpret_cast<decltype(scores_fn)>(pointer(a[2]));
    scores_fp4_fn = reinterpret_cast<decltype(scores_fp4_fn)>(pointer(a[3]));
    evict_fn = reinterpret_cast<decltype(evict_fn)>(pointer(a[4]));
    evict_fp4_fn = reinterpret_cast<decltype(evict_fp4_fn)>(pointer(a[5]));
    prompt_fn = reinterpret_cast<decltype(prompt_fn)>(pointer(a[6]));
    Py_RETURN_NONE;
  });
}

// (context_lens, query_lens, free_blocks, free_start | None, block_table,
//  block_size, num_blocks, max_tokens | None, query_start_loc, seq_lens, positions,
//  slot_mapping, totals, stream | None)
PyObject* plan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor& table = tensor(a[4], "block_table");
    const at::Tensor& free = tensor(a[2], "free_blocks");
    if (table.dim() != 2) refuse(PyExc_ValueError, "block_table must be [num_seqs, max_blocks]");
    if (free.dim() != 1) refuse(PyExc_ValueError, "free_blocks must be [num_free]");
    const int64_t seqs = table.size(0);
    const at::Tensor& slots = tensor(a[11], "slot_mapping");
    if (slots.dim() != 1) refuse(PyExc_ValueError, "slot_mapping must be [max_tokens]");
    const int cap = a[7] == Py_None ? extent(slots.size(0), "slot_mapping")
                                    : integer32(a[7], "max_tokens");
    const int dev = call_device(table, "block_table");
    void* ctx = shaped(a[0], "context_lens", at::kInt, dev, {seqs});
    void* qlen = shaped(a[1], "query_lens", at::kInt, dev, {seqs});
    void* start = a[3] == Py_None ? nullptr : shaped(a[3], "free_start", at::kInt, dev, {1});
    void* qsl = shaped(a[8], "query_start_loc", at::kInt, dev, {seqs + 1});
    void* seq = shaped(a[9], "seq_lens", at::kInt, dev, {seqs});
    void* pos = shaped(a[10], "positions", at::kInt, dev, {cap});
    void* slot = shaped(a[11], "slot_mapping", at::kLong, dev, {cap});
    void* totals = shaped(a[12], "totals", at::kInt, dev, {2});
    using I = int32_t*;
    return call(plan_step_fn, static_cast<I>(ctx), static_cast<I>(qlen),
                static_cast<I>(dense(free, "free_blocks", at::kInt, dev)), static_cast<I>(start),
                extent(free.size(0), "free_blocks"), extent(seqs, "block_table"),
                extent(table.size(1), "block_table"), integer32(a[5], "block_size"),
                integer32(a[6], "num_blocks"), cap,
                static_cast<I>(dense(table, "block_table", at::kInt, dev)), static_cast<I>(qsl),
                static_cast<I>(seq), static_cast<I>(pos), static_cast<int64_t*>(slot),
                static_cast<I>(totals), stream_of(a[13], dev));
  });
}

// The standard pool [num_blocks, 2, block_size, num_kv_heads, head_size].
pa_shape pool_shape(const at::Tensor& pool, int64_t seqs, int64_t heads, int64_t max_blocks) {
  if (pool.dim() != 5 || pool.size(1) != 2)
    refuse(PyExc_ValueError,
           "kv_cache must be [num_blocks, 2, block_size, num_kv_heads, head_size]");
  pa_shape s;
  s.num_seqs = extent(seqs, "seq_lens");
  s.num_q_heads = extent(heads, "q");
  s.num_kv_heads = extent(pool.size(3), "kv_cache");
  s.head_size = extent(pool.size(4), "kv_cache");
  s.block_size = extent(pool.size(2), "kv_cache");
  s.num_blocks = extent(pool.size(0), "kv_cache");
  s.max_blocks_per_seq = extent(max_blocks, "block_table");
  return s;
}

// e4m3 pools are uint8 codes or float8_e4m3fn.
void* pool_pointer(const at::Tensor& pool, bool fp8, int dev) {
  const bool codes = fp8 && pool.scalar_type() == at::kFloat8_e4m3fn;
  return dense(pool, "kv_cache", codes ? at::kFloat8_e4m3fn : fp8 ? at::kByte : at::kBFloat16, dev);
}

// A [tokens, heads, d] bf16 view with dense heads; its token stride.
void* token_rows(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t d, int dev,
                 int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, at::kBFloat16, dev);
  if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != d)
    refuse(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, (long long)tokens,
           (long long)heads, (long long)d);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
    refuse(PyExc_ValueError, "the heads of %s must be dense", name);
  *stride = tokens > 1 ? t.stride(0) : heads * d;
  return t.data_ptr();
}

// (q, key, value, kv_cache, slot_mapping, (k_scale, v_scale) | None,
//  q_weight | None, k_weight | None, eps, cos_sin | None, positions | None,
//  interleaved, q_out, stream | None)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor& pool = tensor(a[3], "kv_cache");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [num_tokens, num_q_heads, head_size]");
    const int64_t tokens = q.size(0), heads = q.size(1), d = q.size(2);
    const pa_shape s = pool_shape(pool, 0, heads, 1);
    if (d != s.head_size) refuse(PyExc_ValueError, "q head_size does not match kv_cache");
    const int dev = call_device(q, "q");
    int64_t qs, ks, vs;
    void* qp = token_rows(a[0], "q", tokens, heads, d, dev, &qs);
    void* kp = token_rows(a[1], "key", tokens, s.num_kv_heads, d, dev, &ks);
    void* vp = token_rows(a[2], "value", tokens, s.num_kv_heads, d, dev, &vs);
    void* slots = shaped(a[4], "slot_mapping", at::kLong, dev, {tokens});
    if ((a[6] == Py_None) != (a[7] == Py_None))
      refuse(PyExc_ValueError, "q_weight and k_weight must be given together");
    void *qw = nullptr, *kw = nullptr, *cs = nullptr, *pos = nullptr;
    if (a[6] != Py_None) {
      qw = shaped(a[6], "q_weight", at::kBFloat16, dev, {d});
      kw = shaped(a[7], "k_weight", at::kBFloat16, dev, {d});
    }
    int rows = 0, rot = 0;
    if (a[9] != Py_None) {
      const at::Tensor& table = tensor(a[9], "cos_sin");
      if (table.dim() != 2 || a[10] == Py_None)
        refuse(PyExc_ValueError,
               "cos_sin [max_position, rotary_dim] needs positions [num_tokens]");
      rows = extent(table.size(0), "cos_sin");
      rot = extent(table.size(1), "cos_sin");
      cs = dense(table, "cos_sin", at::kFloat, dev);
      pos = shaped(a[10], "positions", at::kInt, dev, {tokens});
    }
    const int turned = PyObject_IsTrue(a[11]);
    if (turned < 0) throw Refused();
    void* out = shaped(a[12], "q_out", at::kBFloat16, dev, {tokens, heads, d});
    const bool fp8 = a[5] != Py_None;
    void* cache = pool_pointer(pool, fp8, dev);
    const int count = extent(tokens, "q");
    const float eps = real(a[8]);
    if (fp8) {
      if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 2)
        refuse(PyExc_TypeError, "(k_scale, v_scale) expected");
      return call(norm_fp8_fn, qp, kp, vp, qs, ks, vs, qw, kw, eps, static_cast<float*>(cs), rows,
                  rot, turned, static_cast<int32_t*>(pos), cache, static_cast<int64_t*>(slots),
                  count, &s, real(PyTuple_GET_ITEM(a[5], 0)), real(PyTuple_GET_ITEM(a[5], 1)), out,
                  stream_of(a[13], dev));
    }
    return call(norm_fn, qp, kp, vp, qs, ks, vs, qw, kw, eps, static_cast<float*>(cs), rows, rot,
                turned, static_cast<int32_t*>(pos), cache, static_cast<int64_t*>(slots), count, &s,
                out, stream_of(a[13], dev));
  });
}

struct Window {
  int dev;
  int64_t rows;
  pa_shape shape;
  void *q, *pool, *table, *seq, *out, *lse;
};

// q, kv_cache, block_table, seq_lens, out, lse | None
Window window_args(PyObject* const* a, bool fp8) {
  Window w;
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor& pool = tensor(a[1], "kv_cache");
  const at::Tensor& table = tensor(a[2], "block_table");
  const at::Tensor& seq = tensor(a[3], "seq_lens");
  if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [tokens, num_q_heads, head_size]");
  if (seq.dim() != 1 || table.dim() != 2 || table.size(0) != seq.size(0))
    refuse(PyExc_ValueError,
           "seq_lens must be [num_seqs] and block_table [num_seqs, max_blocks]");
  w.rows = q.size(0);
  w.shape = pool_shape(pool, seq.size(0), q.size(1), table.size(1));
  if (q.size(2) != w.shape.head_size)
    refuse(PyExc_ValueError, "q head_size does not match kv_cache");
  w.dev = call_device(q, "q");
  w.q = dense(q, "q", at::kBFloat16, w.dev);
  w.pool = pool_pointer(pool, fp8, w.dev);
  w.table = dense(table, "block_table", at::kInt, w.dev);
  w.seq = dense(seq, "seq_lens", at::kInt, w.dev);
  w.out = shaped(a[4], "out", at::kBFloat16, w.dev, {w.rows, q.size(1), q.size(2)});
  w.lse = a[5] == Py_None ? nullptr : shaped(a[5], "lse", at::kFloat, w.dev, {w.rows, q.size(1)});
  return w;
}

// (q, kv_cache, block_table, seq_lens, out, lse | None, query_start_loc,
//  max_query_len, scale, sliding_window, num_sinks, stream | None)
PyObject* varlen_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Window w = window_args(a, false);
    void* qsl = shaped(a[6], "query_start_loc", at::kInt, w.dev,
                       {static_cast<int64_t>(w.shape.num_seqs) + 1});
    return call(sinks_fn, w.q, w.pool, static_cast<int32_t*>(w.table), static_cast<int32_t*>(qsl),
                static_cast<int32_t*>(w.seq), extent(w.rows, "q"),
                integer32(a[7], "max_query_len"), &w.shape, real(a[8]),
                integer32(a[9], "sliding_window"), integer32(a[10], "num_sinks"), w.out,
                static_cast<float*>(w.lse), stream_of(a[11], w.dev));
  });
}

// (q, kv_cache, block_table, seq_lens, out, lse | None,
//  (k_scale, v_scale) | None, scale, sliding_window, num_sinks, stream | None)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const bool fp8 = a[6] != Py_None;
    const Window w = window_args(a, fp8);
    if (w.rows != w.shape.num_seqs) refuse(PyExc_ValueError, "q must hold one row per request");
    int32_t* table = static_cast<int32_t*>(w.table);
    int32_t* seq = static_cast<int32_t*>(w.seq);
    float* lse = static_cast<float*>(w.lse);
    const float scale = real(a[7]);
    const int window = integer32(a[8], "sliding_window"), sinks = integer32(a[9], "num_sinks");
    if (fp8) {
      if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2)
        refuse(PyExc_TypeError, "(k_scale, v_scale) expected");
      return call(window_fp8_fn, w.q, w.pool, table, seq, &w.shape, scale,
                  real(PyTuple_GET_ITEM(a[6], 0)), real(PyTuple_GET_ITEM(a[6], 1)), window, sinks,
                  w.out, lse, stream_of(a[10], w.dev));
    }
    return call(window_fn, w.q, w.pool, table, seq, &w.shape, scale, window, sinks, w.out, lse,
                stream_of(a[10], w.dev));
  });
}

// The 4-bit pool [num_blocks, num_kv_heads, block_size / 16, 2, 9 * head_size].
pa_shape pool4_shape(const at::Tensor& pool, int64_t seqs, int64_t heads, int64_t max_blocks) {
  if (pool.dim() != 5 || pool.size(3) != 2 || pool.size(4) % 9 != 0)
    refuse(PyExc_ValueError,
           "kv_cache must be [num_blocks, num_kv_heads, block_size / 16, 2, 9 * head_size]");
  pa_shape s;
  s.num_seqs = extent(seqs, "seq_lens");
  s.num_kv_heads = extent(pool.size(1), "kv_cache");
  s.num_q_heads = heads < 0 ? s.num_kv_heads : extent(heads, "q");
  s.head_size = extent(pool.size(4) / 9, "kv_cache");
  s.block_size = extent(pool.size(2) * 16, "kv_cache");
  s.num_blocks = extent(pool.size(0), "kv_cache");
  s.max_blocks_per_seq = extent(max_blocks, "block_table");
  return s;
}

// (key, value, kv_cache, slot_mapping, k_scale, v_scale, stream | None)
PyObject* cache_write_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor& key = tensor(a[0], "key");
    const at::Tensor& pool = tensor(a[2], "kv_cache");
    const pa_shape s = pool4_shape(pool, 0, -1, 1);
    if (key.dim() != 3)
      refuse(PyExc_ValueError, "key must be [num_tokens, num_kv_heads, head_size]");
    const int64_t tokens = key.size(0);
    const int dev = call_device(key, "key");
    int64_t ks, vs;
    void* kp = token_rows(a[0], "key", tokens, s.num_kv_heads, s.head_size, dev, &ks);
    void* vp = token_rows(a[1], "value", tokens, s.num_kv_heads, s.head_size, dev, &vs);
    void* slots = shaped(a[3], "slot_mapping", at::kLong, dev, {tokens});
    return call(write_fp4_fn, kp, vp, ks, vs, dense(pool, "kv_cache", at::kByte, dev),
                static_cast<int64_t*>(slots), extent(tokens, "key"), &s, real(a[4]), real(a[5]),
                stream_of(a[6], dev));
  });
}

struct Decode {
  int dev;
  pa_shape shape;
  void *q, *pool, *table, *seq, *out, *lse, *workspace, *scores;
  size_t workspace_bytes;
  int score_tokens;
};

// q, kv_cache, block_table, seq_lens, out, lse | None, workspace | None, scores | None
Decode decode_args(PyObject* const* a, bool four) {
  Decode w{};
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor& pool = tensor(a[1], "kv_cache");
  const at::Tensor& table = tensor(a[2], "block_table");
  const at::Tensor& seq = tensor(a[3], "seq_lens");
  if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [num_seqs, num_q_heads, head_size]");
  if (seq.dim() != 1 || table.dim() != 2 || table.size(0) != seq.size(0))
    refuse(PyExc_ValueError,
           "seq_lens must be [num_seqs] and block_table [num_seqs, max_blocks]");
  w.shape = four ? pool4_shape(pool, seq.size(0), q.size(1), table.size(1))
                 : pool_shape(pool, seq.size(0), q.size(1), table.size(1));
  if (q.size(2) != w.shape.head_size)
    refuse(PyExc_ValueError, "q head_size does not match kv_cache");
  if (q.size(0) != seq.size(0)) refuse(PyExc_ValueError, "q must hold one row per request");
  w.dev = call_device(q, "q");
  w.q = dense(q, "q", at::kBFloat16, w.dev);
  w.pool = dense(pool, "kv_cache", four ? at::kByte : at::kBFloat16, w.dev);
  w.table = dense(table, "block_table", at::kInt, w.dev);
  w.seq = dense(seq, "seq_lens", at::kInt, w.dev);
  w.out = shaped(a[4], "out", at::kBFloat16, w.dev, {q.size(0), q.size(1), q.size(2)});
  if (a[5] != Py_None) w.lse = shaped(a[5], "lse", at::kFloat, w.dev, {q.size(0), q.size(1)});
  if (a[6] != Py_None) {
    const at::Tensor& ws = tensor(a[6], "workspace");
    w.workspace = dense(ws, "workspace", at::kByte, w.dev);
    w.workspace_bytes = static_cast<size_t>(ws.numel());
  }
  if (a[7] != Py_None) {
    const at::Tensor& sc = tensor(a[7], "scores");
    if (sc.dim() != 3 || sc.size(0) != seq.size(0) || sc.size(1) != w.shape.num_kv_heads)
      refuse(PyExc_ValueError, "scores must be [num_seqs, num_kv_heads, score_tokens]");
    w.scores = dense(sc, "scores", at::kFloat, w.dev);
    w.score_tokens = extent(sc.size(2), "scores");
  }
  return w;
}

// (q, kv_cache, block_table, seq_lens, out, lse | None, workspace | None,
//  scores | None, (k_scale, v_scale) | None, scale, max_seq_len, stream | None)
PyObject* decode_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const bool four = a[8] != Py_None;
    const Decode w = decode_args(a, four);
    int32_t* table = static_cast<int32_t*>(w.table);
    int32_t* seq = static_cast<int32_t*>(w.seq);
    float *lse = static_cast<float*>(w.lse), *scores = static_cast<float*>(w.scores);
    const float scale = real(a[9]);
    const int longest = integer32(a[10], "max_seq_len");
    void* stream = stream_of(a[11], w.dev);
    if (!four)
      return call(scores_fn, w.q, w.pool, table, seq, &w.shape, scale, longest, w.workspace,
                  w.workspace_bytes, scores, w.score_tokens, w.out, lse, stream);
    if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 2)
      refuse(PyExc_TypeError, "(k_scale, v_scale) expected");
    const float ks = real(PyTuple_GET_ITEM(a[8], 0)), vs = real(PyTuple_GET_ITEM(a[8], 1));
    if (a[7] == Py_None)
      return call(decode_fp4_fn, w.q, w.pool, table, seq, &w.shape, scale, ks, vs, longest,
                  w.workspace, w.workspace_bytes, w.out, lse, stream);
    return call(scores_fp4_fn, w.q, w.pool, table, seq, &w.shape, scale, ks, vs, longest,
                w.workspace, w.workspace_bytes, scores, w.score_tokens, w.out, lse, stream);
  });
}

// (kv_cache, 4-bit, block_table, seq_lens, scores, budget, num_recent, num_first,
//  new_lens, new_scores, kept, free_blocks | None, free_start | None,
//  new_free_start | None, stream | None)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const int four = PyObject_IsTrue(a[1]);
    if (four < 0) throw Refused();
    const at::Tensor& pool = tensor(a[0], "kv_cache");
    const at::Tensor& table = tensor(a[2], "block_table");
    const at::Tensor& seq = tensor(a[3], "seq_lens");
    const at::Tensor& sc = tensor(a[4], "scores");
    if (seq.dim() != 1 || table.dim() != 2 || table.size(0) != seq.size(0))
      refuse(PyExc_ValueError,
             "seq_lens must be [num_seqs] and block_table [num_seqs, max_blocks]");
    const int64_t seqs = seq.size(0);
    if (!four && (pool.dim() != 5 || pool.size(1) != 2))
      refuse(PyExc_ValueError,
             "kv_cache must be [num_blocks, 2, block_size, num_kv_heads, head_size]");
    const pa_shape s = four ? pool4_shape(pool, seqs, -1, table.size(1))
                            : pool_shape(pool, seqs, pool.size(3), table.size(1));
    if (sc.dim() != 3 || sc.size(0) != seqs || sc.size(1) != s.num_kv_heads)
      refuse(PyExc_ValueError, "scores must be [num_seqs, num_kv_heads, score_tokens]");
    const int dev = call_device(pool, "kv_cache");
    const bool bf16 = !four && pool.scalar_type() == at::kBFloat16;
    void* cache = four   ? dense(pool, "kv_cache", at::kByte, dev)
                  : bf16 ? dense(pool, "kv_cache", at::kBFloat16, dev)
                         : pool_pointer(pool, true, dev);
    using I = int32_t*;
    I tp = static_cast<I>(dense(table, "block_table", at::kInt, dev));
    I lp = static_cast<I>(dense(seq, "seq_lens", at::kInt, dev));
    float* sp = static_cast<float*>(dense(sc, "scores", at::kFloat, dev));
    const int cap = extent(sc.size(2), "scores"), budget = integer32(a[5], "budget");
    const int recent = integer32(a[6], "num_recent"), first = integer32(a[7], "num_first");
    I nl = static_cast<I>(shaped(a[8], "new_lens", at::kInt, dev, {seqs}));
    float* ns = static_cast<float*>(
        shaped(a[9], "new_scores", at::kFloat, dev, {seqs, s.num_kv_heads, sc.size(2)}));
    I kept = static_cast<I>(shaped(a[10], "kept", at::kInt, dev, {seqs, s.num_kv_heads, budget}));
    I fb = nullptr, fs = nullptr, nf = nullptr;
    int count = 0;
    if (a[11] != Py_None) {
      const at::Tensor& f = tensor(a[11], "free_blocks");
      if (f.dim() != 1) refuse(PyExc_ValueError, "free_blocks must be [num_free]");
      if (a[12] == Py_None || a[13] == Py_None)
        refuse(PyExc_ValueError, "free_blocks needs free_start");
      fb = static_cast<I>(dense(f, "free_blocks", at::kInt, dev));
      count = extent(f.size(0), "free_blocks");
      fs = static_cast<I>(shaped(a[12], "free_start", at::kInt, dev, {1}));
      nf = static_cast<I>(shaped(a[13], "new_free_start", at::kInt, dev, {1}));
    } else if (a[12] != Py_None || a[13] != Py_None) {
      refuse(PyExc_ValueError, "free_start needs free_blocks");
    }
    void* stream = stream_of(a[14], dev);
    if (four)
      return call(evict_fp4_fn, cache, &s, tp, lp, sp, cap, budget, recent, first, nl, ns, kept, fb,
                  count, fs, nf, stream);
    return call(evict_fn, cache, &s, bf16 ? 2 : 1, tp, lp, sp, cap, budget, recent, first, nl, ns,
                kept, fb, count, fs, nf, stream);
  });
}

// (q, key, value, query_start_loc, max_query_len, scale, out, lse | None, stream | None)
PyObject* prompt_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor& key = tensor(a[1], "key");
    const at::Tensor& qsl = tensor(a[3], "query_start_loc");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [total_q, num_q_heads, head_size]");
    if (key.dim() != 3)
      refuse(PyExc_ValueError, "key must be [total_q, num_kv_heads, head_size]");
    if (qsl.dim() != 1 || qsl.size(0) < 1)
      refuse(PyExc_ValueError, "query_start_loc must be [num_seqs + 1]");
    const int64_t tokens = q.size(0), heads = q.size(1), kv = key.size(1), d = q.size(2);
    const int dev = call_device(q, "q");
    int64_t qs, ks, vs;
    void* qp = token_rows(a[0], "q", tokens, heads, d, dev, &qs);
    void* kp = token_rows(a[1], "key", tokens, kv, d, dev, &ks);
    void* vp = token_rows(a[2], "value", tokens, kv, d, dev, &vs);
    void* sp = dense(qsl, "query_start_loc", at::kInt, dev);
    void* out = shaped(a[6], "out", at::kBFloat16, dev, {tokens, heads, d});
    void* lse = a[7] == Py_None ? nullptr : shaped(a[7], "lse", at::kFloat, dev, {tokens, heads});
    return call(prompt_fn, qp, kp, vp, qs, ks, vs, static_cast<int32_t*>(sp),
                extent(qsl.size(0) - 1, "query_start_loc"), extent(tokens, "q"),
                integer32(a[4], "max_query_len"), extent(heads, "q"), extent(kv, "key"),
                extent(d, "q"), real(a[5]), out, static_cast<float*>(lse), stream_of(a[8], dev));
  });
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"check_device", fast(check_device), METH_FASTCALL, "Refuses a device that is not current."},
    {"bind", fast(bind), METH_FASTCALL, "Takes the library's entry points (addresses)."},
    {"bind_more", fast(bind_more), METH_FASTCALL, "Takes more of them."},
    {"cache_write_fp4", fast(cache_write_fp4), METH_FASTCALL, "pa_reshape_and_cache_fp4"},
    {"decode_scores", fast(decode_scores), METH_FASTCALL,
     "pa_decode_scores, with scales pa_decode_fp4 or pa_decode_scores_fp4"},
    {"evict", fast(evict), METH_FASTCALL, "pa_evict, pa_evict_fp4"},
    {"prompt_fwd", fast(prompt_fwd), METH_FASTCALL, "pa_prompt_fwd"},
    {"plan_step", fast(plan_step), METH_FASTCALL, "pa_plan_step"},
    {"norm_rope", fast(norm_rope), METH_FASTCALL, "pa_qk_norm_rope_cache, with scales _fp8"},
    {"varlen_sinks", fast(varlen_sinks), METH_FASTCALL, "pa_varlen_fwd_sinks"},
    {"decode_window", fast(decode_window), METH_FASTCALL, "pa_decode_window, with scales _fp8"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__binding() { return PyModule_Create(&module); }
