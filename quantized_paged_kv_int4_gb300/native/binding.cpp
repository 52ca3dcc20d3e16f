// Argument marshalling of the serving-step calls (kvq_plan_step, kvq_rope, kvq_write_kv, kvq_decode_kv): torch tensors are
// checked and their pointers, strides and the current stream handed to the C ABI. These calls are small and frequent --
// a step of 32 tokens runs a few microseconds on the GPU -- and a dozen tensors checked in Python cost 6 to 10 us a
// call; here they cost about one. kvq.py holds the public functions; every check and every error is raised here.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "../../include/kvq.h"

namespace {

struct PyError {};  // a Python exception is set

[[noreturn]] void fail(PyObject *type, const char *format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw PyError{};
}

PyObject *g_error = nullptr;  // KvqError(status, where)

void check(kvq_status status, const char *where) {
  if (status == KVQ_OK) return;
  PyObject *e = g_error ? PyObject_CallFunction(g_error, "is", static_cast<int>(status), where) : nullptr;
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, where);
  }
  throw PyError{};
}

const at::Tensor &cuda_tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}

void same_device(const at::Tensor &t, const char *name, int dev) {
  if (t.get_device() != dev) fail(PyExc_ValueError, "%s is on cuda:%d, the call on cuda:%d", name, static_cast<int>(t.get_device()), dev);
}

// A contiguous tensor of a type on the call's device.
const at::Tensor &on(PyObject *o, const char *name, at::ScalarType type, int dev) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  same_device(t, name, dev);
  return t;
}
void *sized(PyObject *o, const char *name, at::ScalarType type, int dev, int64_t size) {
  const at::Tensor &t = on(o, name, type, dev);
  if (t.numel() != size)
    fail(PyExc_ValueError, "%s must have %lld entries, got %lld", name, static_cast<long long>(size), static_cast<long long>(t.numel()));
  return t.data_ptr();
}
void *sized_or_null(PyObject *o, const char *name, at::ScalarType type, int dev, int64_t size) {
  return o == Py_None ? nullptr : sized(o, name, type, dev, size);
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}
int32_t integer32(PyObject *o, const char *name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(v);
}
int32_t count32(int64_t v, const char *name) {
  if (v > INT32_MAX) fail(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(v);
}
float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return static_cast<float>(v);
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError{};
  return v != 0;
}

int64_t attribute(PyObject *o, const char *name) {
  PyObject *v = PyObject_GetAttrString(o, name);
  if (v == nullptr) throw PyError{};
  const long long r = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (r == -1 && PyErr_Occurred()) throw PyError{};
  return r;
}

// The call's stream and, while it lives, its device and (when given) its stream as the current ones: memory for outputs
// and workspaces has to come from the stream that uses it, as another's may still be in use there.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard on_stream;
  kvq_stream_t stream;
  Place(PyObject *o, int dev) {
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    } else {
      const int64_t at = attribute(o, "device_index");
      if (at != dev) fail(PyExc_ValueError, "the stream is on cuda:%d, the call on cuda:%d", static_cast<int>(at), dev);
      const c10::cuda::CUDAStream s = c10::cuda::CUDAStream::unpack3(attribute(o, "stream_id"), static_cast<c10::DeviceIndex>(at),
                                                                     c10::DeviceType::CUDA);
      on_stream.reset_stream(s);
      stream = s.stream();
    }
  }
};

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// An output: the caller's object, or a new tensor of the given shape. Gives a new reference in *made.
struct Made {
  PyObject *o = nullptr;
  ~Made() { Py_XDECREF(o); }
  PyObject *take(PyObject *given) {
    Py_INCREF(given);
    return o = given;
  }
  PyObject *make(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
    o = THPVariable_Wrap(empty(sizes, type, like));
    if (o == nullptr) throw PyError{};
    return o;
  }
  PyObject *release() {
    PyObject *r = o;
    o = nullptr;
    return r;
  }
};

kvq_dtype row_code(at::ScalarType t) {
  return t == at::kBFloat16 ? KVQ_BF16 : t == at::kHalf ? KVQ_F16 : KVQ_F32;
}

// [T, heads, D] rows with a contiguous last dim.
struct Rows {
  void *p = nullptr;
  int64_t st = 0, sh = 0, heads = 0;
};
Rows rows_of(PyObject *o, const char *name, at::ScalarType type, int dev, int64_t T, int64_t D) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  if (t.dim() != 3 || t.size(0) != T || t.size(2) != D)
    fail(PyExc_ValueError, "%s must be [%lld, heads, %lld]", name, static_cast<long long>(T), static_cast<long long>(D));
  if (t.stride(2) != 1 && D > 1) fail(PyExc_ValueError, "%s must have a contiguous last dim", name);
  same_device(t, name, dev);
  return {t.data_ptr(), t.stride(0), t.stride(1), t.size(1)};
}

kvq_rotary rotary_of(PyObject *positions, PyObject *freqs, PyObject *interleaved, PyObject *factor, int64_t T, int64_t D, int dev) {
  kvq_rotary r;
  r.positions = static_cast<const int32_t *>(sized(positions, "positions", at::kInt, dev, T));
  const at::Tensor &f = on(freqs, "freqs", at::kLong, dev);
  if (f.dim() != 1 || f.numel() < 1 || f.numel() > D / 2)
    fail(PyExc_ValueError, "freqs must be [rotary_dim / 2] with rotary_dim <= D = %lld", static_cast<long long>(D));
  r.freqs = static_cast<const uint64_t *>(f.data_ptr());
  r.rotary_dim = static_cast<int32_t>(2 * f.numel());
  r.interleaved = truth(interleaved);
  r.attn_factor = real(factor);
  return r;
}

// The paged cache of two [num_blocks, block_size, Hk, D] views; type: of the rows beside it; heads: Hk, or -1 for any.
kvq_paged_kv paged_of(PyObject *ko, PyObject *vo, PyObject *ks, PyObject *vs, at::ScalarType type, int dev, int64_t heads, int64_t D) {
  const at::Tensor &k = cuda_tensor(ko, "k_cache"), &v = cuda_tensor(vo, "v_cache");
  const at::ScalarType c = k.scalar_type();
  if ((c != at::kBFloat16 && c != at::kHalf && c != at::kFloat8_e4m3fn) || v.scalar_type() != c)
    fail(PyExc_TypeError, "k_cache / v_cache must both be bfloat16, float16 or float8_e4m3fn");
  if (k.dim() != 4 || v.sizes() != k.sizes()) fail(PyExc_ValueError, "k_cache / v_cache must both be [num_blocks, block_size, Hk, D]");
  if (k.stride(3) != 1 || v.stride(3) != 1) fail(PyExc_ValueError, "k_cache / v_cache must have a contiguous last dim");
  if (k.size(3) != D || (heads >= 0 && k.size(2) != heads))
    fail(PyExc_ValueError, "the cache's heads are [%lld, %lld], which the rows are not", static_cast<long long>(k.size(2)),
         static_cast<long long>(k.size(3)));
  if (c != at::kFloat8_e4m3fn && (c != type || ks != Py_None || vs != Py_None))
    fail(PyExc_TypeError, "a 16-bit cache has the type of the rows (%s) and no scales", c10::toString(type));
  same_device(k, "k_cache", dev);
  same_device(v, "v_cache", dev);
  kvq_paged_kv r;
  r.k = k.data_ptr();
  r.v = v.data_ptr();
  r.k_stride_block = k.stride(0);
  r.k_stride_token = k.stride(1);
  r.k_stride_head = k.stride(2);
  r.v_stride_block = v.stride(0);
  r.v_stride_token = v.stride(1);
  r.v_stride_head = v.stride(2);
  r.k_scale = static_cast<const float *>(sized_or_null(ks, "k_scale", at::kFloat, dev, k.size(2)));
  r.v_scale = static_cast<const float *>(sized_or_null(vs, "v_scale", at::kFloat, dev, k.size(2)));
  r.dtype = c == at::kFloat8_e4m3fn ? KVQ_E4M3 : row_code(c);
  r.block_size = count32(k.size(1), "block_size");
  r.num_blocks = k.size(0);
  return r;
}

// context, query, table, free, cursor, block_size, num_blocks, rows, batch, cursor_out, seq_lens, starts, positions,
// slots, T, stream
PyObject *plan_step(PyObject *const *a) {
  const at::Tensor &context = cuda_tensor(a[0], "context_lens");
  const int dev = context.get_device();
  on(a[0], "context_lens", at::kInt, dev);
  const int64_t B = context.numel();
  const at::Tensor &table = on(a[2], "block_table", at::kInt, dev);
  if (table.dim() != 2) fail(PyExc_ValueError, "block_table must be [rows, max_blocks]");
  const int64_t width = table.size(1);
  if ((a[3] == Py_None) != (a[4] == Py_None)) fail(PyExc_ValueError, "free_blocks and cursor go together");
  const void *free_blocks = nullptr;
  int64_t num_free = 0;
  if (a[3] != Py_None) {
    const at::Tensor &f = on(a[3], "free_blocks", at::kInt, dev);
    free_blocks = f.data_ptr();
    num_free = f.numel();
  }
  int64_t T;
  if (a[14] != Py_None) {
    T = integer(a[14]);
    if (T < 0) fail(PyExc_ValueError, "T must not be negative");
  } else {
    PyObject *given = a[12] != Py_None ? a[12] : a[13];
    if (given == Py_None) fail(PyExc_ValueError, "T, the rows of positions and slot_mapping, is needed");
    T = cuda_tensor(given, "positions / slot_mapping").numel();
  }
  Made out[4];
  const Place place(a[15], dev);
  const int64_t sizes[4] = {B, B + 1, T, T};
  const char *names[4] = {"seq_lens", "query_start_loc", "positions", "slot_mapping"};
  void *p[4];
  for (int i = 0; i < 4; ++i) {
    const at::ScalarType type = i == 3 ? at::kLong : at::kInt;
    PyObject *o = a[10 + i] != Py_None ? out[i].take(a[10 + i]) : out[i].make({sizes[i]}, type, context);
    p[i] = sized(o, names[i], type, dev, sizes[i]);
  }
  void *batch = nullptr;
  if (a[8] != Py_None) {
    const at::Tensor &b = on(a[8], "batch_table", at::kInt, dev);
    if (b.dim() != 2 || b.size(0) != B || b.size(1) != width)
      fail(PyExc_ValueError, "batch_table must be [B, max_blocks] = (%lld, %lld)", static_cast<long long>(B), static_cast<long long>(width));
    batch = b.data_ptr();
  }
  const void *query = sized_or_null(a[1], "query_lens", at::kInt, dev, B), *rows = sized_or_null(a[7], "rows", at::kInt, dev, B);
  const void *cursor = sized_or_null(a[4], "cursor", at::kLong, dev, 1);
  void *cursor_out = a[9] == Py_None ? const_cast<void *>(cursor) : sized(a[9], "cursor_out", at::kLong, dev, 1);
  check(kvq_plan_step(static_cast<const int32_t *>(context.data_ptr()), static_cast<const int32_t *>(query),
                      static_cast<const int32_t *>(rows), static_cast<int32_t *>(table.data_ptr()), count32(width, "max_blocks"),
                      table.size(0), static_cast<const int32_t *>(free_blocks), num_free, static_cast<const int64_t *>(cursor),
                      static_cast<int64_t *>(cursor_out), static_cast<int32_t *>(p[0]), static_cast<int32_t *>(p[1]),
                      static_cast<int32_t *>(p[2]), static_cast<int64_t *>(p[3]), static_cast<int32_t *>(batch), count32(B, "B"),
                      count32(T, "T"), integer32(a[5], "block_size"), integer(a[6]), place.stream),
        "kvq_plan_step");
  PyObject *r = PyTuple_New(4);
  if (r == nullptr) throw PyError{};
  for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(r, i, out[i].release());
  return r;
}

// A rotated row set and its output (a new one for None).
struct Rotated {
  Rows in, out;
  Made made;
  void set(PyObject *o, PyObject *given, const char *name, const char *out_name, at::ScalarType type, int dev, int64_t T, int64_t D) {
    in = rows_of(o, name, type, dev, T, D);
    PyObject *to = given != Py_None ? made.take(given) : made.make({T, in.heads, D}, type, THPVariable_Unpack(o));
    out = rows_of(to, out_name, type, dev, T, D);
    if (out.heads != in.heads) fail(PyExc_ValueError, "%s must have %s's shape", out_name, name);
  }
  PyObject *result() {
    if (made.o != nullptr) return made.release();
    Py_RETURN_NONE;
  }
};

// q, k, positions, freqs, interleaved, attn_factor, q_out, k_out, stream
PyObject *rope(PyObject *const *a) {
  PyObject *ref = a[0] != Py_None ? a[0] : a[1];
  const at::Tensor &x = cuda_tensor(ref, a[0] != Py_None ? "q" : "k");
  const int dev = x.get_device();
  const at::ScalarType type = x.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat)
    fail(PyExc_TypeError, "q / k must be bfloat16, float16 or float32, got %s", c10::toString(type));
  if (x.dim() != 3) fail(PyExc_ValueError, "q / k must be [T, heads, D]");
  const int64_t T = x.size(0), D = x.size(2);
  if ((a[0] == Py_None && a[6] != Py_None) || (a[1] == Py_None && a[7] != Py_None)) fail(PyExc_ValueError, "an output without its input");
  const Place place(a[8], dev);
  Rotated q, k;
  if (a[0] != Py_None) q.set(a[0], a[6], "q", "q_out", type, dev, T, D);
  if (a[1] != Py_None) k.set(a[1], a[7], "k", "k_out", type, dev, T, D);
  const kvq_rotary r = rotary_of(a[2], a[3], a[4], a[5], T, D, dev);
  check(kvq_rope(q.in.p, q.in.st, q.in.sh, q.out.p, q.out.st, q.out.sh, count32(q.in.heads, "heads"), k.in.p, k.in.st, k.in.sh,
                 k.out.p, k.out.st, k.out.sh, count32(k.in.heads, "heads"), &r, row_code(type), count32(T, "T"), count32(D, "D"),
                 place.stream),
        "kvq_rope");
  PyObject *qo = q.result(), *ko = k.result();
  PyObject *t = PyTuple_Pack(2, qo, ko);
  Py_DECREF(qo);
  Py_DECREF(ko);
  if (t == nullptr) throw PyError{};
  return t;
}

// key, value, k_cache, v_cache, slot_mapping, k_scale, v_scale, q, positions, freqs, interleaved, attn_factor, q_out, stream
PyObject *write_kv(PyObject *const *a) {
  const at::Tensor &key = cuda_tensor(a[0], "key");
  const int dev = key.get_device();
  const at::ScalarType type = key.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf) fail(PyExc_TypeError, "key must be a CUDA bfloat16 or float16 tensor");
  if (key.dim() != 3) fail(PyExc_ValueError, "key must be [T, Hk, D]");
  const int64_t T = key.size(0), D = key.size(2);
  const Rows k = rows_of(a[0], "key", type, dev, T, D), v = rows_of(a[1], "value", type, dev, T, D);
  if (v.heads != k.heads) fail(PyExc_ValueError, "value must have key's shape");
  const kvq_paged_kv cache = paged_of(a[2], a[3], a[5], a[6], type, dev, k.heads, D);
  const void *slots = sized(a[4], "slot_mapping", at::kLong, dev, T);
  if ((a[8] == Py_None) != (a[9] == Py_None)) fail(PyExc_ValueError, "positions and freqs go together");
  kvq_rotary r;
  const bool rot = a[8] != Py_None;
  const Place place(a[13], dev);
  if (rot) r = rotary_of(a[8], a[9], a[10], a[11], T, D, dev);
  Rotated q;
  if (a[7] != Py_None) {
    if (!rot) fail(PyExc_ValueError, "q is only rotated: positions and freqs are needed");
    q.set(a[7], a[12], "q", "q_out", type, dev, T, D);
  } else if (a[12] != Py_None) {
    fail(PyExc_ValueError, "q_out without q");
  }
  check(kvq_write_kv(k.p, k.st, k.sh, v.p, v.st, v.sh, &cache, static_cast<const int64_t *>(slots), q.in.p, q.in.st, q.in.sh, q.out.p,
                     q.out.st, q.out.sh, count32(q.in.heads, "heads"), rot ? &r : nullptr, row_code(type), count32(T, "T"),
                     count32(k.heads, "heads"), count32(D, "D"), place.stream),
        "kvq_write_kv");
  return q.result();
}

// q, k_cache, v_cache, block_table, seq_lens, softmax_scale, k_scale, v_scale, out, workspace, num_splits, out_dtype, stream,
// sliding_window, softcap, sinks, alibi_slopes, lse_out
PyObject *decode_kv(PyObject *const *a) {
  const at::Tensor &q = cuda_tensor(a[0], "q");
  const int dev = q.get_device();
  const at::ScalarType type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf) fail(PyExc_TypeError, "q must be a CUDA bfloat16 or float16 tensor");
  on(a[0], "q", type, dev);
  if (q.dim() != 3) fail(PyExc_ValueError, "q must be [B, Hq, D]");
  const int32_t B = count32(q.size(0), "B"), Hq = count32(q.size(1), "Hq"), D = count32(q.size(2), "D");
  const kvq_paged_kv cache = paged_of(a[1], a[2], a[6], a[7], type, dev, -1, D);
  const int32_t Hk = count32(THPVariable_Unpack(a[1]).size(2), "Hk");
  const at::Tensor &table = on(a[3], "block_table", at::kInt, dev);
  if (table.dim() != 2 || table.size(0) != B) fail(PyExc_ValueError, "block_table must be [B, max_blocks] with B = %d", B);
  const void *lens = sized(a[4], "seq_lens", at::kInt, dev, B);
  Made out, ws;
  const Place place(a[12], dev);
  PyObject *o = a[8];
  if (o != Py_None) {
    out.take(o);
  } else {
    at::ScalarType t = type;
    if (a[11] != Py_None) {
      if (!THPDtype_Check(a[11])) fail(PyExc_TypeError, "out_dtype must be a torch dtype");
      t = reinterpret_cast<THPDtype *>(a[11])->scalar_type;
    }
    o = out.make({B, Hq, D}, t, q);
  }
  const at::Tensor &to = cuda_tensor(o, "out");
  const at::ScalarType ot = to.scalar_type();
  if (ot != at::kBFloat16 && ot != at::kHalf && ot != at::kFloat)
    fail(PyExc_TypeError, "out must be bfloat16, float16 or float32, got %s", c10::toString(ot));
  on(o, "out", ot, dev);
  if (to.sizes() != q.sizes()) fail(PyExc_ValueError, "out must have q's shape");
  const int32_t splits = integer32(a[10], "num_splits");
  kvq_score_mods mods = {};
  mods.sliding_window = integer32(a[13], "sliding_window");
  mods.softcap = real(a[14]);
  mods.sinks = static_cast<const float *>(sized_or_null(a[15], "sinks", at::kFloat, dev, Hq));
  mods.alibi_slopes = static_cast<const float *>(sized_or_null(a[16], "alibi_slopes", at::kFloat, dev, Hq));
  if (a[17] != Py_None) {
    const at::Tensor &l = on(a[17], "lse_out", at::kFloat, dev);
    if (l.dim() != 2 || l.size(0) != B || l.size(1) != Hq) fail(PyExc_ValueError, "lse_out must be [%d, %d]", B, Hq);
    mods.lse_out = static_cast<float *>(l.data_ptr());
  }
  PyObject *w = a[9];
  if (w == Py_None) {
    const int64_t need = static_cast<int64_t>(kvq_decode_kv_workspace_bytes(B, Hq, Hk, D, splits));
    w = ws.make({need > 16 ? need : 16}, at::kByte, q);
  }
  const at::Tensor &work = on(w, "workspace", at::kByte, dev);
  check(kvq_decode_kv(q.data_ptr(), row_code(type), &cache, static_cast<const int32_t *>(table.data_ptr()),
                      count32(table.size(1), "max_blocks"), static_cast<const int32_t *>(lens), real(a[5]), splits, work.data_ptr(),
                      static_cast<size_t>(work.numel()), to.data_ptr(), row_code(ot), B, Hq, Hk, D, &mods, place.stream),
        "kvq_decode_kv");
  return out.release();
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", N, static_cast<int>(n));
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyError &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject *set_error(PyObject *, PyObject *cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"plan_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<plan_step, 16>)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<rope, 9>)), METH_FASTCALL, nullptr},
    {"write_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<write_kv, 14>)), METH_FASTCALL, nullptr},
    {"decode_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<decode_kv, 18>)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvq_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kvq_native(void) { return PyModule_Create(&module); }
