// Argument checks and marshalling of the paged serving operators, compiled: a
// decode step makes a few of these calls a layer, each on a kernel of a few
// microseconds, and the same checks written in Python cost 6 to 10 us a call
// (measured on Grace's Arm cores), more than the kernels of a small
// batch. Nothing is computed here. Each function takes its tensors by
// position, raises TypeError or ValueError, and returns the status of the C
// entry.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gqa.h"

namespace {

constexpr int64_t DIM = GQA_HEAD_DIM;

// Thrown once a Python exception is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const char* name, const char* what) {
  PyErr_Format(kind, "%s %s", name, what);
  throw Refused();
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "must be torch.bfloat16";
    case at::kInt: return "must be torch.int32";
    case at::kFloat: return "must be torch.float32";
    case at::kFloat8_e4m3fn: return "must be torch.float8_e4m3fn";
    default: return "must be torch.uint8";
  }
}

const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type) refuse(PyExc_TypeError, name, type_name(type));
  if (t.layout() != at::kStrided) refuse(PyExc_ValueError, name, "must be a dense tensor");
  return t;
}

// The device of a call: that of its first tensor; every other is on it too.
struct Device {
  c10::Device d;
  void same(const at::Tensor& t, const char* name) const {
    if (t.device() != d) refuse(PyExc_ValueError, name, "must be on the device of the other tensors");
  }
  void cuda(const char* name) const {
    if (!d.is_cuda()) refuse(PyExc_ValueError, name, "must be a CUDA tensor");
  }
};

// Packed rows [n, heads, 128] whose heads follow each other.
struct Rows {
  gqa_bf16* p;
  int64_t n, heads, stride;
};
Rows rows(const at::Tensor& t, const char* name, int64_t n = -1, int64_t heads = -1) {
  if (t.dim() != 3 || t.size(2) != DIM || (n >= 0 && t.size(0) != n) || (heads >= 0 && t.size(1) != heads)) {
    if (n < 0)
      PyErr_Format(PyExc_ValueError, "%s must be [tokens, heads, 128]", name);
    else if (heads < 0)
      PyErr_Format(PyExc_ValueError, "%s must be [%lld, heads, 128]", name, (long long)n);
    else
      PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, 128]", name, (long long)n, (long long)heads);
    throw Refused();
  }
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) refuse(PyExc_ValueError, name, "has too many rows");
  if (t.stride(2) != 1 || (t.stride(1) != DIM && t.size(1) > 1))
    refuse(PyExc_ValueError, name, "must have a head's 128 elements, and a token's heads, one after the other");
  // the stride of an axis of one element says nothing
  return {static_cast<gqa_bf16*>(t.data_ptr()), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1) * DIM};
}

gqa_bf16* output(PyObject* o, const char* name, int64_t n, int64_t heads, const Device& d) {
  const at::Tensor& t = tensor(o, name, at::kBFloat16);
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != DIM || !t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous [%lld, %lld, 128] tensor", name, (long long)n,
                 (long long)heads);
    throw Refused();
  }
  d.same(t, name);
  return static_cast<gqa_bf16*>(t.data_ptr());
}

// Contiguous int32 [n] (n < 0: any length); the length goes to *len.
const int32_t* ints(PyObject* o, const char* name, int64_t n, const Device& d, int64_t* len = nullptr) {
  const at::Tensor& t = tensor(o, name, at::kInt);
  if (t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous()) {
    if (n < 0)
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous one-dimensional tensor", name);
    else
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous [%lld] tensor", name, (long long)n);
    throw Refused();
  }
  if (t.size(0) > INT32_MAX) refuse(PyExc_ValueError, name, "is too long");
  d.same(t, name);
  if (len) *len = t.size(0);
  return static_cast<const int32_t*>(t.data_ptr());
}

// The pages of k or of v by their common shape and strides, the table.
struct Pages {
  const at::Tensor &k, &v, &table;
  int64_t stride(int axis) const { return k.size(axis) > 1 ? k.stride(axis) : DIM; }
  template <class C>
  void put(C& g, int64_t B) const {
    g.page_stride = stride(0);
    g.row_stride = stride(1);
    g.head_stride = stride(2);
    g.block_table = static_cast<const int32_t*>(table.data_ptr());
    g.num_pages = static_cast<int>(k.size(0));
    g.page_size = static_cast<int>(k.size(1));
    g.n_kv_heads = static_cast<int>(k.size(2));
    g.columns = static_cast<int>(table.size(1));
    g.table_stride = B > 1 ? static_cast<int>(table.stride(0)) : g.columns;
  }
};
struct PageNames {
  const char *k, *v, *table;
};
Pages page_tensors(PyObject* k_, PyObject* v_, PyObject* table_, int64_t B, const Device& d, at::ScalarType type,
                   const PageNames& names) {
  const at::Tensor& k = tensor(k_, names.k, type);
  const at::Tensor& v = tensor(v_, names.v, type);
  const at::Tensor& t = tensor(table_, names.table, at::kInt);
  if (k.dim() != 4 || k.size(3) != DIM) refuse(PyExc_ValueError, names.k, "must be [pages, page_size, n_kv, 128]");
  if (v.sizes() != k.sizes() || v.strides() != k.strides()) {
    PyErr_Format(PyExc_ValueError, "%s must have the shape and the strides of %s", names.v, names.k);
    throw Refused();
  }
  if (k.stride(3) != 1) refuse(PyExc_ValueError, names.k, "must have a head's 128 elements one after the other");
  if (t.dim() != 2 || t.size(0) != B || (t.size(1) > 1 && t.stride(1) != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, columns] with adjacent columns", names.table, (long long)B);
    throw Refused();
  }
  for (int i = 0; i < 3; ++i)
    if (k.size(i) > INT32_MAX) refuse(PyExc_ValueError, names.k, "is too large");
  if (t.size(1) > INT32_MAX || t.stride(0) > INT32_MAX) refuse(PyExc_ValueError, names.table, "is too wide");
  d.same(k, names.k);
  d.same(v, names.v);
  d.same(t, names.table);
  return {k, v, t};
}

gqa_pages pages(PyObject* k, PyObject* v, PyObject* table, int64_t B, const Device& d,
                const PageNames& names = {"k_pages", "v_pages", "block_table"}) {
  const Pages p = page_tensors(k, v, table, B, d, at::kBFloat16, names);
  gqa_pages g;
  g.k = static_cast<gqa_bf16*>(p.k.data_ptr());
  g.v = static_cast<gqa_bf16*>(p.v.data_ptr());
  p.put(g, B);
  return g;
}

gqa_fp8_pages fp8_pages(PyObject* k, PyObject* v, PyObject* ks_, PyObject* vs_, PyObject* table, int64_t B,
                        const Device& d) {
  const Pages p = page_tensors(k, v, table, B, d, at::kFloat8_e4m3fn, {"k_pages", "v_pages", "block_table"});
  const at::Tensor& ks = tensor(ks_, "k_scales", at::kByte);
  const at::Tensor& vs = tensor(vs_, "v_scales", at::kByte);
  if (ks.dim() != 3 || ks.size(0) != p.k.size(0) || ks.size(1) != p.k.size(1) || ks.size(2) != p.k.size(2))
    refuse(PyExc_ValueError, "k_scales", "must be [pages, page_size, n_kv] like k_pages");
  if (vs.sizes() != ks.sizes() || vs.strides() != ks.strides())
    refuse(PyExc_ValueError, "v_scales", "must have the shape and the strides of k_scales");
  d.same(ks, "k_scales");
  d.same(vs, "v_scales");
  gqa_fp8_pages g;
  g.k = static_cast<uint8_t*>(p.k.data_ptr());
  g.v = static_cast<uint8_t*>(p.v.data_ptr());
  g.k_scale = static_cast<uint8_t*>(ks.data_ptr());
  g.v_scale = static_cast<uint8_t*>(vs.data_ptr());
  int64_t* strides[3] = {&g.scale_page_stride, &g.scale_row_stride, &g.scale_head_stride};
  for (int i = 0; i < 3; ++i) *strides[i] = ks.size(i) > 1 ? ks.stride(i) : 1;
  p.put(g, B);
  return g;
}

struct Workspace {
  void* p;
  size_t bytes;
};
Workspace workspace(PyObject* o, const Device& d) {
  const at::Tensor& t = tensor(o, "workspace", at::kByte);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace", "must be contiguous");
  d.same(t, "workspace");
  return {t.data_ptr(), static_cast<size_t>(t.numel())};
}

// A stream handle, or None: torch's current stream on the device.
void* stream(PyObject* o, const Device& d) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(d.d.index()).stream();
  void* s = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw Refused();
  return s;
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(x);
}

template <int N, int (*Call)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(Call(a));
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

int number_of(PyObject* o, const char* name) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refused();
  if (x < INT32_MIN || x > INT32_MAX) refuse(PyExc_ValueError, name, "is out of range");
  return static_cast<int>(x);
}

// The tokens of an append: q, k, v, start_pos, rope, cu_tokens, q_out.
struct Tokens {
  Device d;
  Rows q, k, v;
  int64_t B;
  const int32_t *start, *cu;
  const float* rope;
  int rope_rows;
};
Tokens tokens(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* start_, PyObject* rope_, PyObject* cu_, int rotary_dim) {
  const at::Tensor& kt = tensor(k_, "k", at::kBFloat16);
  const Device d{kt.device()};
  const Rows k = rows(kt, "k");
  const at::Tensor& vt = tensor(v_, "v", at::kBFloat16);
  d.same(vt, "v");
  const Rows v = rows(vt, "v", k.n, k.heads);
  int64_t B = 0;
  const int32_t* start = ints(start_, "start_pos", -1, d, &B);
  const int32_t* cu = cu_ == Py_None ? nullptr : ints(cu_, "cu_tokens", B + 1, d);
  if (!cu && B != k.n) refuse(PyExc_ValueError, "start_pos", "must have one value per token without cu_tokens");
  const at::Tensor& rope = tensor(rope_, "rope", at::kFloat);
  if (rope.dim() != 3 || rope.size(1) != rotary_dim / 2 || rope.size(2) != 2 || !rope.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "rope must be a contiguous [rows, %d, 2] tensor", rotary_dim / 2);
    throw Refused();
  }
  if (rope.size(0) > INT32_MAX) refuse(PyExc_ValueError, "rope", "has too many rows");
  d.same(rope, "rope");
  return {d, {nullptr, 0, 0, 0}, k, v, B, start, cu, static_cast<const float*>(rope.data_ptr()),
          static_cast<int>(rope.size(0))};
}
// q and q_out, the last of them to be looked at
gqa_bf16* queries(Tokens& t, PyObject* q_, PyObject* q_out_, int n_kv) {
  if (n_kv != t.k.heads) refuse(PyExc_ValueError, "k", "must have the KV heads of the pages");
  gqa_bf16* q_out = nullptr;
  if (q_ != Py_None) {
    const at::Tensor& qt = tensor(q_, "q", at::kBFloat16);
    t.d.same(qt, "q");
    t.q = rows(qt, "q", t.k.n);
    q_out = output(q_out_, "q_out", t.k.n, t.q.heads, t.d);
  } else if (q_out_ != Py_None) {
    refuse(PyExc_ValueError, "q_out", "needs q");
  }
  t.d.cuda("k");
  return q_out;
}

// q, k, v, start_pos, rope, k_pages, v_pages, block_table, cu_tokens, q_out, workspace, stream
int paged_append(PyObject* const* a) {
  Tokens t = tokens(a[0], a[1], a[2], a[3], a[4], a[8], DIM);
  const gqa_pages g = pages(a[5], a[6], a[7], t.B, t.d);
  gqa_bf16* q_out = queries(t, a[0], a[9], g.n_kv_heads);
  const Workspace w = workspace(a[10], t.d);
  if (t.k.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(t.d.d);
  return gqa_paged_append(t.q.p, t.q.stride, t.k.p, t.k.stride, t.v.p, t.v.stride, static_cast<int>(t.k.n),
                          static_cast<int>(t.q.heads), t.cu, static_cast<int>(t.B), t.start, t.rope, t.rope_rows, &g,
                          q_out, w.p, w.bytes, stream(a[11], t.d));
}

int rotary(PyObject* o) {
  const int r = number_of(o, "rotary_dim");
  if (r < 16 || r > DIM || r % 16) refuse(PyExc_ValueError, "rotary_dim", "must be a multiple of 16, 16 to 128");
  return r;
}

// q, k, v, start_pos, rope, k_pages, v_pages, block_table, cu_tokens, q_out, rotary_dim, halves, workspace, stream
int paged_append_rotary(PyObject* const* a) {
  const int dim = rotary(a[10]), halves = PyObject_IsTrue(a[11]);
  if (halves < 0) throw Refused();
  Tokens t = tokens(a[0], a[1], a[2], a[3], a[4], a[8], dim);
  const gqa_pages g = pages(a[5], a[6], a[7], t.B, t.d);
  gqa_bf16* q_out = queries(t, a[0], a[9], g.n_kv_heads);
  const Workspace w = workspace(a[12], t.d);
  if (t.k.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(t.d.d);
  return gqa_paged_append_rotary(t.q.p, t.q.stride, t.k.p, t.k.stride, t.v.p, t.v.stride, static_cast<int>(t.k.n),
                                 static_cast<int>(t.q.heads), t.cu, static_cast<int>(t.B), t.start, t.rope,
                                 t.rope_rows, dim, halves, &g, q_out, w.p, w.bytes, stream(a[13], t.d));
}

// q, k, v, start_pos, rope, k_pages, v_pages, k_scales, v_scales, block_table, cu_tokens, q_out, rotary_dim, halves,
// workspace, stream
int paged_append_fp8(PyObject* const* a) {
  const int dim = rotary(a[12]), halves = PyObject_IsTrue(a[13]);
  if (halves < 0) throw Refused();
  Tokens t = tokens(a[0], a[1], a[2], a[3], a[4], a[10], dim);
  const gqa_fp8_pages g = fp8_pages(a[5], a[6], a[7], a[8], a[9], t.B, t.d);
  gqa_bf16* q_out = queries(t, a[0], a[11], g.n_kv_heads);
  const Workspace w = workspace(a[14], t.d);
  if (t.k.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(t.d.d);
  return gqa_paged_append_fp8(t.q.p, t.q.stride, t.k.p, t.k.stride, t.v.p, t.v.stride, static_cast<int>(t.k.n),
                              static_cast<int>(t.q.heads), t.cu, static_cast<int>(t.B), t.start, t.rope, t.rope_rows,
                              dim, halves, &g, q_out, w.p, w.bytes, stream(a[15], t.d));
}

// rows, k_pages, v_pages, k_scales, v_scales, block_table, k_out, v_out, out_table, workspace, stream
int paged_read_fp8(PyObject* const* a) {
  const at::Tensor& rt = tensor(a[0], "rows", at::kInt);
  const Device d{rt.device()};
  int64_t B = 0;
  const int32_t* n = ints(a[0], "rows", -1, d, &B);
  const gqa_fp8_pages from = fp8_pages(a[1], a[2], a[3], a[4], a[5], B, d);
  const gqa_pages to = pages(a[6], a[7], a[8], B, d, {"k_out", "v_out", "out_table"});
  if (to.n_kv_heads != from.n_kv_heads) refuse(PyExc_ValueError, "k_out", "must have the KV heads of k_pages");
  d.cuda("rows");
  const Workspace w = workspace(a[9], d);
  if (B == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(d.d);
  return gqa_paged_read_fp8(n, static_cast<int>(B), &from, &to, w.p, w.bytes, stream(a[10], d));
}

// q, start_pos, cu_groups, prefix_rows, k_pages, v_pages, block_table, scale, out, workspace, stream
int paged_decode_shared(PyObject* const* a) {
  const at::Tensor& qt = tensor(a[0], "q", at::kBFloat16);
  const Device d{qt.device()};
  const Rows q = rows(qt, "q");
  const int32_t* start = ints(a[1], "start_pos", q.n, d);
  int64_t G = 0;
  const int32_t* prefix = ints(a[3], "prefix_rows", -1, d, &G);
  const int32_t* cu = ints(a[2], "cu_groups", G + 1, d);
  const gqa_pages g = pages(a[4], a[5], a[6], q.n, d);
  const float scale = number(a[7]);
  gqa_bf16* out = output(a[8], "out", q.n, q.heads, d);
  d.cuda("q");
  const Workspace w = workspace(a[9], d);
  if (q.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(d.d);
  if (G == 0)
    return gqa_paged_decode(q.p, q.stride, static_cast<int>(q.n), static_cast<int>(q.heads), start, &g, scale, out, w.p,
                            w.bytes, stream(a[10], d));
  return gqa_paged_decode_shared(q.p, q.stride, static_cast<int>(q.n), static_cast<int>(q.heads), start, cu,
                                 static_cast<int>(G), prefix, &g, scale, out, w.p, w.bytes, stream(a[10], d));
}

// q, start_pos, k_pages, v_pages, k_scales, v_scales, block_table, scale, out, workspace, stream
int paged_decode_fp8(PyObject* const* a) {
  const at::Tensor& qt = tensor(a[0], "q", at::kBFloat16);
  const Device d{qt.device()};
  const Rows q = rows(qt, "q");
  const int32_t* start = ints(a[1], "start_pos", q.n, d);
  const gqa_fp8_pages g = fp8_pages(a[2], a[3], a[4], a[5], a[6], q.n, d);
  const float scale = number(a[7]);
  gqa_bf16* out = output(a[8], "out", q.n, q.heads, d);
  d.cuda("q");
  const Workspace w = workspace(a[9], d);
  if (q.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(d.d);
  return gqa_paged_decode_fp8(q.p, q.stride, static_cast<int>(q.n), static_cast<int>(q.heads), start, &g, scale, out,
                              w.p, w.bytes, stream(a[10], d));
}

// q, start_pos, k_pages, v_pages, block_table, scale, out, workspace, stream
int paged_decode(PyObject* const* a) {
  const at::Tensor& qt = tensor(a[0], "q", at::kBFloat16);
  const Device d{qt.device()};
  const Rows q = rows(qt, "q");
  const int32_t* start = ints(a[1], "start_pos", q.n, d);
  const gqa_pages g = pages(a[2], a[3], a[4], q.n, d);
  const float scale = number(a[5]);
  gqa_bf16* out = output(a[6], "out", q.n, q.heads, d);
  d.cuda("q");
  const Workspace w = workspace(a[7], d);
  if (q.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(d.d);
  return gqa_paged_decode(q.p, q.stride, static_cast<int>(q.n), static_cast<int>(q.heads), start, &g, scale, out, w.p,
                          w.bytes, stream(a[8], d));
}

// q, cu_tokens, start_pos, k_pages, v_pages, block_table, scale, out, workspace, stream
int paged_prefill(PyObject* const* a) {
  const at::Tensor& qt = tensor(a[0], "q", at::kBFloat16);
  const Device d{qt.device()};
  const Rows q = rows(qt, "q");
  int64_t B = 0;
  const int32_t* start = ints(a[2], "start_pos", -1, d, &B);
  const int32_t* cu = ints(a[1], "cu_tokens", B + 1, d);
  const gqa_pages g = pages(a[3], a[4], a[5], B, d);
  const float scale = number(a[6]);
  gqa_bf16* out = output(a[7], "out", q.n, q.heads, d);
  d.cuda("q");
  const Workspace w = workspace(a[8], d);
  if (q.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(d.d);
  return gqa_paged_prefill(q.p, q.stride, static_cast<int>(q.n), static_cast<int>(q.heads), cu, static_cast<int>(B),
                           start, &g, scale, out, w.p, w.bytes, stream(a[9], d));
}

// q, k, v, cu_tokens, scale, out, workspace, stream
int packed_prefill(PyObject* const* a) {
  const at::Tensor& qt = tensor(a[0], "q", at::kBFloat16);
  const Device d{qt.device()};
  const Rows q = rows(qt, "q");
  const at::Tensor& kt = tensor(a[1], "k", at::kBFloat16);
  d.same(kt, "k");
  const Rows k = rows(kt, "k", q.n);
  const at::Tensor& vt = tensor(a[2], "v", at::kBFloat16);
  d.same(vt, "v");
  const Rows v = rows(vt, "v", q.n, k.heads);
  int64_t B1 = 0;
  const int32_t* cu = ints(a[3], "cu_tokens", -1, d, &B1);
  if (B1 < 2) refuse(PyExc_ValueError, "cu_tokens", "must have one value more than there are sequences");
  const float scale = number(a[4]);
  gqa_bf16* out = output(a[5], "out", q.n, q.heads, d);
  d.cuda("q");
  const Workspace w = workspace(a[6], d);
  if (q.n == 0) return GQA_OK;
  const c10::cuda::CUDAGuard guard(d.d);
  return gqa_packed_prefill(q.p, q.stride, k.p, k.stride, v.p, v.stride, static_cast<int>(q.n),
                            static_cast<int>(q.heads), static_cast<int>(k.heads), cu, static_cast<int>(B1 - 1), scale,
                            out, w.p, w.bytes, stream(a[7], d));
}

template <int N, int (*Call)(PyObject* const*)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<N, Call>));
}

PyMethodDef methods[] = {
    {"paged_append", fast<12, paged_append>(), METH_FASTCALL, nullptr},
    {"paged_append_rotary", fast<14, paged_append_rotary>(), METH_FASTCALL, nullptr},
    {"paged_append_fp8", fast<16, paged_append_fp8>(), METH_FASTCALL, nullptr},
    {"paged_read_fp8", fast<11, paged_read_fp8>(), METH_FASTCALL, nullptr},
    {"paged_decode_fp8", fast<11, paged_decode_fp8>(), METH_FASTCALL, nullptr},
    {"paged_decode_shared", fast<11, paged_decode_shared>(), METH_FASTCALL, nullptr},
    {"paged_decode", fast<9, paged_decode>(), METH_FASTCALL, nullptr},
    {"paged_prefill", fast<10, paged_prefill>(), METH_FASTCALL, nullptr},
    {"packed_prefill", fast<8, packed_prefill>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gqa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gqa_binding(void) { return PyModule_Create(&module); }
