// binding.cpp -- the serving calls for Python: torch tensors to the argument
// structs of splash.h.
//
// The rest of the library is called through ctypes.  A serving step's kernels
// take 2 to 5 us each, and reading some forty tensor attributes from Python
// took 8 to 10 us a call; here it takes half a microsecond.  Host time of a
// call: append 10.7 -> 3.0 .. 3.6 us, a short rope 13.2 -> 5.2 .. 6.0, a short
// decode 13.8 -> 5.4 .. 6.4, most of it the launch and the outputs' allocation.
//
// Shapes and types are checked before the device, so that the refusals can be
// tested without one.  Nothing here computes.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "splash.h"

namespace {

PyObject *g_error = nullptr;  // SplashError(status, what)

// Thrown for a Python error that is already set.
struct PythonError {};

[[noreturn]] void value_error(const std::string &what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw PythonError();
}

std::string text(at::IntArrayRef shape) {
  std::string s = "[";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "]";
}

const at::Tensor &tensor(PyObject *x, const char *name) {
  if (!THPVariable_Check(x)) value_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(x);
}

int64_t integer(PyObject *x) {
  const long long v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

int32_t integer32(PyObject *x, const char *name) {
  const int64_t v = integer(x);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
  return (int32_t)v;
}

int32_t truth(PyObject *x) {
  const int v = PyObject_IsTrue(x);
  if (v < 0) throw PythonError();
  return v;
}

float number(PyObject *x) {
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return (float)v;
}

// The tensors of a call; all must be on the current device.
struct Call {
  const at::Tensor *on[16];
  int n = 0;

  const at::Tensor &take(const at::Tensor &t) {
    on[n++] = &t;
    return t;
  }

  void check_device() const {
    int current = -1;
    for (int i = 0; i < n; ++i) {
      if (on[i]->is_cuda() && current < 0) current = c10::cuda::current_device();
      if (!on[i]->is_cuda() || on[i]->get_device() != current)
        value_error("the tensors must be on the current CUDA device (got " + on[i]->device().str() + ")");
    }
  }

  // bf16 [B, H, L, d], contiguous in d
  splash_view view(const at::Tensor &t, const char *name, at::IntArrayRef shape) {
    if (t.scalar_type() != at::kBFloat16 || t.sizes() != shape || t.strides()[3] != 1)
      value_error(std::string(name) + " must be a bf16 tensor of shape " + text(shape) + ", contiguous in its last dimension (got " +
                  text(t.sizes()) + ")");
    const auto s = take(t).strides();
    return {t.data_ptr(), s[0], s[1], s[2]};
  }

  // int32 [axes, B, L]
  const int32_t *axis_index(PyObject *x, const char *name, int64_t B, int64_t L, int64_t *axes, int64_t *stride_a, int64_t *stride_b) {
    const at::Tensor &t = tensor(x, name);
    if (t.scalar_type() != at::kInt || t.dim() != 3 || t.size(0) < 1 || t.size(1) != B || t.size(2) != L || (L > 1 && t.stride(2) != 1))
      value_error(std::string(name) + " must be an int32 tensor [axes, " + std::to_string(B) + ", " + std::to_string(L) +
                  "], contiguous in its last dimension (got " + text(t.sizes()) + ")");
    *axes = t.size(0);
    *stride_a = t.stride(0);
    *stride_b = t.stride(1);
    return static_cast<const int32_t *>(take(t).data_ptr());
  }

  // A contiguous int32 tensor of a shape.
  int32_t *ints(const at::Tensor &t, const char *name, at::IntArrayRef shape) {
    if (t.scalar_type() != at::kInt || t.sizes() != shape || !t.is_contiguous())
      value_error(std::string(name) + " must be a contiguous int32 tensor of shape " + text(shape) + " (got " + text(t.sizes()) + ")");
    return static_cast<int32_t *>(take(t).data_ptr());
  }

  // int32 [B, L] or [L]
  const int32_t *index(PyObject *x, const char *name, int64_t B, int64_t L, int64_t *stride) {
    const at::Tensor &t = tensor(x, name);
    const bool two = t.dim() == 2 && t.size(0) == B && t.size(1) == L, one = t.dim() == 1 && t.size(0) == L;
    if (t.scalar_type() != at::kInt || !(two || one) || (L > 1 && t.strides().back() != 1))
      value_error(std::string(name) + " must be an int32 tensor of shape " + text({B, L}) + " or " + text({L}) +
                  ", contiguous in its last dimension (got " + text(t.sizes()) + ")");
    *stride = two ? t.stride(0) : 0;
    return static_cast<const int32_t *>(take(t).data_ptr());
  }

  const float *table(PyObject *x, int64_t *rows, int32_t *rot) {
    const at::Tensor &t = tensor(x, "table");
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous() || t.size(1) > INT32_MAX)
      value_error("table must be a contiguous fp32 tensor [positions, rot_dim]");
    *rows = t.size(0);
    *rot = (int32_t)t.size(1);
    return static_cast<const float *>(take(t).data_ptr());
  }

  const float *scale(PyObject *x, const char *name, int64_t heads) {
    if (x != Py_None) {
      const at::Tensor &t = tensor(x, name);
      if (t.scalar_type() == at::kFloat && t.dim() == 1 && t.size(0) == heads && t.is_contiguous())
        return static_cast<const float *>(take(t).data_ptr());
    }
    value_error(std::string(name) + " must be a contiguous fp32 tensor of shape " + text({heads}) + " for an e4m3 cache");
  }

  // The caches of an argument struct; returns whether they are e4m3.
  template <class Args>
  bool cache_pair(Args &a, PyObject *kx, PyObject *vx) {
    const at::Tensor &k = tensor(kx, "k_cache"), &v = tensor(vx, "v_cache");
    const auto type = k.scalar_type();
    const bool e4m3 = type == at::kFloat8_e4m3fn;
    if ((!e4m3 && type != at::kBFloat16) || v.scalar_type() != type || k.dim() != 4 || v.dim() != 4 ||
        k.sizes().slice(0, 3) != v.sizes().slice(0, 3) || k.strides()[3] != 1 || v.strides()[3] != 1)
      value_error("k_cache and v_cache must be bf16 or float8_e4m3fn tensors [pages, Hkv, page_size, d], contiguous in the "
                  "last dimension and alike in the others");
    const auto shape = k.sizes();
    if (shape[1] > INT32_MAX || shape[2] > INT32_MAX || shape[3] > INT32_MAX || v.size(3) > INT32_MAX)
      value_error("k_cache and v_cache are too large");
    a.k_cache = {take(k).data_ptr(), k.stride(0), k.stride(1), k.stride(2)};
    a.v_cache = {take(v).data_ptr(), v.stride(0), v.stride(1), v.stride(2)};
    a.num_pages = shape[0];
    a.Hkv = (int32_t)shape[1];
    a.page_size = (int32_t)shape[2];
    a.dqk = (int32_t)shape[3];
    a.dv = (int32_t)v.size(3);
    a.cache_type = e4m3 ? SPLASH_CACHE_E4M3 : SPLASH_CACHE_BF16;
    return e4m3;
  }

  // The same with their scales.
  template <class Args>
  void caches(Args &a, PyObject *kx, PyObject *vx, PyObject *ks, PyObject *vs) {
    if (cache_pair(a, kx, vx)) {
      a.k_scale = scale(ks, "k_scale", a.Hkv);
      a.v_scale = scale(vs, "v_scale", a.Hkv);
    } else if (ks != Py_None || vs != Py_None) {
      value_error("k_scale and v_scale belong to an e4m3 cache");
    }
  }

  template <class Args>
  int64_t block_table(Args &a, PyObject *x) {
    const at::Tensor &t = tensor(x, "block_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1) || t.size(0) > INT32_MAX ||
        t.size(1) > INT32_MAX)
      value_error("block_table must be an int32 tensor [sequences, pages], contiguous in its last dimension");
    a.block_table = static_cast<const int32_t *>(take(t).data_ptr());
    a.block_table_stride = t.stride(0);
    a.max_pages = (int32_t)t.size(1);
    return t.size(0);
  }
};

int32_t size32(int64_t v, const char *name) {
  if (v > INT32_MAX) value_error(std::string(name) + " is too large");
  return (int32_t)v;
}

// The axis of each rotated pair, as bytes; the library checks their values.
const uint8_t *axis_map(PyObject *x, int64_t rot) {
  char *p = nullptr;
  Py_ssize_t n = 0;
  if (!PyBytes_Check(x) || PyBytes_AsStringAndSize(x, &p, &n) != 0 || n != rot / 2) {
    PyErr_Clear();
    value_error("axes must be bytes, an axis for each of the table's " + std::to_string(rot / 2) + " pairs (rope_axis_map)");
  }
  return reinterpret_cast<const uint8_t *>(p);
}

// A new tensor of the call, or the given one.
struct Output {
  PyObject *object;  // given, or nullptr
  at::Tensor made;

  PyObject *python() {
    if (object != nullptr) return Py_NewRef(object);
    return THPVariable_Wrap(std::move(made));
  }
};

// The stream of a call: torch's current one, or a given handle.
struct Stream {
  c10::cuda::CUDAStream current, used;

  // after check_device
  explicit Stream(PyObject *x)
      : current(c10::cuda::getCurrentCUDAStream()),
        used(x == Py_None ? current
                          : c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>((uintptr_t)integer(x)),
                                                             current.device_index())) {}

  // A new tensor of the call, from the memory of its stream, so that nothing
  // another stream still uses is overwritten; kept until the current stream's
  // later work is done with it.
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) const {
    const auto options = like.options().dtype(type);
    if (used == current) return at::empty(shape, options, at::MemoryFormat::Contiguous);
    const c10::cuda::CUDAStreamGuard guard(used);
    at::Tensor t = at::empty(shape, options, at::MemoryFormat::Contiguous);
    t.record_stream(current.unwrap());
    return t;
  }
};

template <class Args>
void run(splash_status (*f)(const Args *, void *), const Args &a, const Stream &stream, const char *what) {
  splash_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f(&a, stream.used.stream());
  Py_END_ALLOW_THREADS;
  if (st == SPLASH_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, what);
  if (e != nullptr) {
    PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw PythonError();
}

PyObject *pair(Output &a, Output &b) {
  PyObject *x = a.python(), *y = b.python();
  PyObject *t = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
    throw PythonError();
  }
}

// rope(q, k, positions, table, rot_offset, interleaved, inverse, q_out, k_out, stream), with `axes` after the table
// for several of them
template <bool AXES>
PyObject *rope(PyObject *const *x, Py_ssize_t n) {
  count(n, AXES ? 11 : 10);
  PyObject *const *y = AXES ? x + 1 : x;  // the arguments behind the table
  Call c;
  splash_rope_axes_args all = {};
  all.struct_bytes = sizeof all;
  splash_rope_args &a = all.rope;
  a.struct_bytes = sizeof a;
  const at::Tensor &q = tensor(x[0], "q");
  if (q.dim() != 4) value_error("q must be 4-D");
  const auto shape = q.sizes();
  a.q = c.view(q, "q", shape);
  a.B = size32(shape[0], "B");
  a.Hq = size32(shape[1], "Hq");
  a.L = shape[2];
  a.d = size32(shape[3], "d");
  const bool has_k = x[1] != Py_None;
  const at::Tensor *k = nullptr;
  if (has_k) {
    k = &tensor(x[1], "k");
    if (k->dim() != 4) value_error("k must be 4-D");
    a.Hkv = size32(k->size(1), "Hkv");
    a.k = c.view(*k, "k", {shape[0], k->size(1), shape[2], shape[3]});
  } else if (y[8] != Py_None) {
    value_error("k_out without k");
  }
  int64_t axes = 0;
  a.positions = AXES ? c.axis_index(x[2], "positions", shape[0], shape[2], &axes, &all.positions_stride_a, &a.positions_stride_b)
                     : c.index(x[2], "positions", shape[0], shape[2], &a.positions_stride_b);
  a.table = c.table(x[3], &a.table_rows, &a.rot_dim);
  if (AXES) {
    all.axes = axis_map(x[4], a.rot_dim);
    all.num_axes = size32(axes, "positions");
  }
  a.rot_offset = integer32(y[4], "rot_offset");
  a.interleaved = truth(y[5]);
  a.inverse = truth(y[6]);
  Output qo{y[7] != Py_None ? y[7] : nullptr, {}}, ko{y[8] != Py_None || !has_k ? y[8] : nullptr, {}};
  if (qo.object != nullptr) a.q_out = c.view(tensor(y[7], "q_out"), "q_out", shape);
  if (has_k && ko.object != nullptr) a.k_out = c.view(tensor(y[8], "k_out"), "k_out", k->sizes());
  c.check_device();
  const Stream stream(y[9]);
  const int64_t row = shape[3], head = shape[2] * row;
  if (qo.object == nullptr) {
    qo.made = stream.make(shape, at::kBFloat16, q);
    a.q_out = {qo.made.data_ptr(), shape[1] * head, head, row};
  }
  if (ko.object == nullptr) {
    ko.made = stream.make(k->sizes(), at::kBFloat16, q);
    a.k_out = {ko.made.data_ptr(), k->size(1) * head, head, row};
  }
  if (AXES)
    run(splash_rope_axes, all, stream, "splash_rope_axes");
  else
    run(splash_rope, a, stream, "splash_rope");
  return pair(qo, ko);
}

// paged_append(k, v, k_cache, v_cache, block_table, positions, q, table, rot_offset, interleaved, seq_ids,
//              k_scale, v_scale, q_out, k_out, stream), with `rot_positions, axes` at the end for several axes
template <bool AXES>
PyObject *paged_append(PyObject *const *x, Py_ssize_t n) {
  count(n, AXES ? 18 : 16);
  Call c;
  splash_paged_append_axes_args all = {};
  all.struct_bytes = sizeof all;
  splash_paged_append_args &a = all.append;
  a.struct_bytes = sizeof a;
  c.caches(a, x[2], x[3], x[11], x[12]);
  const at::Tensor &k = tensor(x[0], "k"), &v = tensor(x[1], "v");
  if (k.dim() != 4 || v.dim() != 4) value_error("k and v must be 4-D");
  const int64_t B = k.size(0), L = k.size(2);
  a.B = size32(B, "B");
  a.L = L;
  a.k = c.view(k, "k", {B, a.Hkv, L, a.dqk});
  a.v = c.view(v, "v", {B, a.Hkv, L, a.dv});
  a.num_seqs = (int32_t)c.block_table(a, x[4]);
  a.positions = c.index(x[5], "positions", B, L, &a.positions_stride_b);
  if (x[10] != Py_None) a.seq_ids = c.index(x[10], "seq_ids", B, L, &a.seq_ids_stride_b);
  if (AXES || x[7] != Py_None) a.table = c.table(x[7], &a.table_rows, &a.rot_dim);
  if (AXES) {
    int64_t axes = 0;
    all.rot_positions = c.axis_index(x[16], "rot_positions", B, L, &axes, &all.rot_positions_stride_a, &all.rot_positions_stride_b);
    all.axes = axis_map(x[17], a.rot_dim);
    all.num_axes = size32(axes, "rot_positions");
  }
  a.rot_offset = integer32(x[8], "rot_offset");
  a.interleaved = truth(x[9]);
  const bool has_q = x[6] != Py_None;
  const at::Tensor *q = nullptr;
  Output qo{x[13] != Py_None || !has_q ? x[13] : nullptr, {}}, ko{x[14], {}};
  if (has_q) {
    q = &tensor(x[6], "q");
    if (q->dim() != 4) value_error("q must be 4-D");
    a.Hq = size32(q->size(1), "Hq");
    a.q = c.view(*q, "q", {B, q->size(1), L, a.dqk});
    if (qo.object != nullptr) a.q_out = c.view(tensor(x[13], "q_out"), "q_out", q->sizes());
  } else if (x[13] != Py_None) {
    value_error("q_out without q");
  }
  if (x[14] != Py_None) a.k_out = c.view(tensor(x[14], "k_out"), "k_out", k.sizes());
  c.check_device();
  const Stream stream(x[15]);
  if (qo.object == nullptr) {
    qo.made = stream.make(q->sizes(), at::kBFloat16, k);
    a.q_out = {qo.made.data_ptr(), q->size(1) * L * a.dqk, L * a.dqk, a.dqk};
  }
  if (AXES)
    run(splash_paged_append_axes, all, stream, "splash_paged_append_axes");
  else
    run(splash_paged_append, a, stream, "splash_paged_append");
  return pair(qo, ko);
}

// paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, softcap, window_left, k_scale, v_scale,
//              out, lse, workspace, stream), with `parents` at the end for a tree
template <bool TREE>
PyObject *paged_decode(PyObject *const *x, Py_ssize_t n) {
  count(n, TREE ? 15 : 14);
  Call c;
  splash_paged_tree_decode_args all = {};
  all.struct_bytes = sizeof all;
  splash_paged_decode_args &a = all.decode;
  a.struct_bytes = sizeof a;
  c.caches(a, x[1], x[2], x[8], x[9]);
  const at::Tensor &q = tensor(x[0], "q");
  if (q.dim() != 4) value_error("q must be 4-D");
  const int64_t B = q.size(0), Hq = q.size(1), Lq = q.size(2);
  a.B = size32(B, "B");
  a.Hq = size32(Hq, "Hq");
  a.Lq = size32(Lq, "Lq");
  a.q = c.view(q, "q", {B, Hq, Lq, a.dqk});
  if (c.block_table(a, x[3]) != B) value_error("block_table must have a row for each of the " + std::to_string(B) + " sequences");
  const at::Tensor &lens = tensor(x[4], "seq_lens");
  if (lens.scalar_type() != at::kInt || lens.dim() != 1 || lens.size(0) != B || !lens.is_contiguous())
    value_error("seq_lens must be a contiguous int32 tensor of shape " + text({B}));
  a.seq_lens = static_cast<const int32_t *>(c.take(lens).data_ptr());
  if (TREE) all.parents = c.index(x[14], "parents", B, Lq, &all.parents_stride_b);
  a.scale = number(x[5]);
  a.softcap = number(x[6]);
  a.window_left = integer(x[7]);
  Output out{x[10] != Py_None ? x[10] : nullptr, {}}, lse{x[11] != Py_None ? x[11] : nullptr, {}};
  const int64_t oshape[4] = {B, Hq, Lq, a.dv};
  const at::IntArrayRef full(oshape, 4), rows(oshape, 3);
  if (out.object != nullptr) {
    const at::Tensor &t = tensor(x[10], "out");
    if (t.scalar_type() != at::kBFloat16 || t.sizes() != full || !t.is_contiguous())
      value_error("out must be a contiguous bf16 tensor of shape " + text(full));
    a.out = c.take(t).data_ptr();
  }
  if (lse.object != nullptr) {
    const at::Tensor &t = tensor(x[11], "lse");
    if (t.scalar_type() != at::kFloat || t.sizes() != rows || !t.is_contiguous())
      value_error("lse must be a contiguous fp32 tensor of shape " + text(rows));
    a.lse = static_cast<float *>(c.take(t).data_ptr());
  }
  if (x[12] != Py_None) {
    const at::Tensor &t = tensor(x[12], "workspace");
    if (!t.is_contiguous()) value_error("workspace must be contiguous");
    a.workspace = c.take(t).data_ptr();
    a.workspace_bytes = t.nbytes();
  }
  c.check_device();
  const Stream stream(x[13]);
  at::Tensor workspace;
  if (x[12] == Py_None) {
    size_t bytes = 0;  // (an error here is the call's own: it is reported there)
    const auto size = TREE ? splash_paged_tree_decode_workspace_size : splash_paged_decode_workspace_size;
    size(a.B, a.Hq, a.Hkv, a.Lq, a.dqk, a.dv, a.max_pages, a.page_size, a.cache_type, a.window_left, &bytes);
    if (bytes > 0) {
      workspace = stream.make({(int64_t)bytes}, at::kByte, q);
      a.workspace = workspace.data_ptr();
      a.workspace_bytes = bytes;
    }
  }
  if (out.object == nullptr) {
    out.made = stream.make(full, at::kBFloat16, q);
    a.out = out.made.data_ptr();
  }
  if (lse.object == nullptr) {
    lse.made = stream.make(rows, at::kFloat, q);
    a.lse = static_cast<float *>(lse.made.data_ptr());
  }
  if (TREE)
    run(splash_paged_tree_decode, all, stream, "splash_paged_tree_decode");
  else
    run(splash_paged_decode, a, stream, "splash_paged_decode");
  return pair(out, lse);
}

// paged_compact(k_cache, v_cache, block_table, src, start, stream)
PyObject *paged_compact(PyObject *const *x, Py_ssize_t n) {
  count(n, 6);
  Call c;
  splash_paged_compact_args a = {};
  a.struct_bytes = sizeof a;
  c.cache_pair(a, x[0], x[1]);
  const int64_t B = c.block_table(a, x[2]);
  a.B = size32(B, "B");
  const at::Tensor &src = tensor(x[3], "src");
  if (src.scalar_type() != at::kInt || src.dim() != 2 || src.size(0) != B || (src.size(1) > 1 && src.stride(1) != 1))
    value_error("src must be an int32 tensor [" + std::to_string(B) + ", moves], contiguous in its last dimension (got " +
                text(src.sizes()) + ")");
  a.src = static_cast<const int32_t *>(c.take(src).data_ptr());
  a.src_stride = src.stride(0);
  a.moves = src.size(1);
  a.start = c.ints(tensor(x[4], "start"), "start", {B});
  c.check_device();
  const Stream stream(x[5]);
  run(splash_paged_compact, a, stream, "splash_paged_compact");
  Py_RETURN_NONE;
}

// paged_copy(k_cache, v_cache, copies, stream)
PyObject *paged_copy(PyObject *const *x, Py_ssize_t n) {
  count(n, 4);
  Call c;
  splash_paged_copy_args a = {};
  a.struct_bytes = sizeof a;
  c.cache_pair(a, x[0], x[1]);
  const at::Tensor &copies = tensor(x[2], "copies");
  const int64_t rows = copies.dim() == 2 ? copies.size(0) : 0;
  a.copies = c.ints(copies, "copies", {rows, 3});
  a.count = size32(rows, "copies");
  c.check_device();
  const Stream stream(x[3]);
  run(splash_paged_copy, a, stream, "splash_paged_copy");
  Py_RETURN_NONE;
}

// paged_remap(block_table, parents, keep, room, refs, page_size, new_table, refs_out, copies, short, workspace, stream)
PyObject *paged_remap(PyObject *const *x, Py_ssize_t n) {
  count(n, 12);
  Call c;
  splash_paged_remap_args a = {};
  a.struct_bytes = sizeof a;
  a.num_rows = (int32_t)c.block_table(a, x[0]);
  const at::Tensor &parents = tensor(x[1], "parents"), &refs = tensor(x[4], "refs");
  if (parents.dim() != 1) value_error("parents must be 1-D");
  if (refs.dim() != 1) value_error("refs must be 1-D");
  const int64_t rows = parents.size(0), pages = refs.size(0);
  a.new_rows = size32(rows, "parents");
  a.num_pages = pages;
  a.parents = c.ints(parents, "parents", {rows});
  a.keep = c.ints(tensor(x[2], "keep"), "keep", {rows});
  a.room = c.ints(tensor(x[3], "room"), "room", {rows});
  a.refs = c.ints(refs, "refs", {pages});
  a.page_size = integer32(x[5], "page_size");
  Output made[4];
  const int64_t shapes[4][2] = {{rows, a.max_pages}, {pages, 0}, {rows, 3}, {1, 0}};
  const char *const names[4] = {"new_table", "refs_out", "copies", "short"};
  int32_t **const ptrs[4] = {&a.new_table, &a.refs_out, &a.copies, &a.short_pages};
  for (int i = 0; i < 4; ++i) {
    made[i].object = x[6 + i] != Py_None ? x[6 + i] : nullptr;
    if (made[i].object != nullptr) *ptrs[i] = c.ints(tensor(x[6 + i], names[i]), names[i], at::IntArrayRef(shapes[i], i % 2 ? 1 : 2));
  }
  if (x[10] != Py_None) {
    const at::Tensor &t = tensor(x[10], "workspace");
    if (!t.is_contiguous()) value_error("workspace must be contiguous");
    a.workspace = c.take(t).data_ptr();
    a.workspace_bytes = t.nbytes();
  }
  c.check_device();
  a.new_table_stride = a.max_pages;
  const Stream stream(x[11]);
  at::Tensor workspace;
  if (x[10] == Py_None) {
    size_t bytes = 0;  // (an error here is the call's own: it is reported there)
    splash_paged_remap_workspace_size(a.num_pages, a.new_rows, &bytes);
    workspace = stream.make({(int64_t)bytes}, at::kByte, refs);
    a.workspace = workspace.data_ptr();
    a.workspace_bytes = bytes;
  }
  for (int i = 0; i < 4; ++i) {
    if (made[i].object != nullptr) continue;
    made[i].made = stream.make(at::IntArrayRef(shapes[i], i % 2 ? 1 : 2), at::kInt, refs);
    *ptrs[i] = static_cast<int32_t *>(made[i].made.data_ptr());
  }
  run(splash_paged_remap, a, stream, "splash_paged_remap");
  PyObject *t = PyTuple_New(4);
  for (int i = 0; t != nullptr && i < 4; ++i) {
    PyObject *o = made[i].python();
    if (o == nullptr) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i, o);
  }
  return t;
}

// No C++ exception reaches Python's frames: torch's become its Python errors.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *x, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(x, n);
  } catch (const PythonError &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *type) {
  PyObject *old = g_error;
  g_error = Py_NewRef(type);
  Py_XDECREF(old);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<F>));
}

PyMethodDef methods[] = {{"rope", entry<rope<false>>(), METH_FASTCALL, nullptr},
                         {"rope_axes", entry<rope<true>>(), METH_FASTCALL, nullptr},
                         {"paged_append", entry<paged_append<false>>(), METH_FASTCALL, nullptr},
                         {"paged_append_axes", entry<paged_append<true>>(), METH_FASTCALL, nullptr},
                         {"paged_decode", entry<paged_decode<false>>(), METH_FASTCALL, nullptr},
                         {"paged_tree_decode", entry<paged_decode<true>>(), METH_FASTCALL, nullptr},
                         {"paged_compact", entry<paged_compact>(), METH_FASTCALL, nullptr},
                         {"paged_copy", entry<paged_copy>(), METH_FASTCALL, nullptr},
                         {"paged_remap", entry<paged_remap>(), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding() { return PyModule_Create(&module); }
