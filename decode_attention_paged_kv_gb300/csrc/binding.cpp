// binding.cpp -- the Python side of libdkv's calls of a decode step: reads the
// tensors' addresses, sizes and strides, checks them, fills the C structs of
// include/dkv.h and makes the call on the tensors' device and its current stream.
// No computation happens here.
//
// A decode step's calls run for a few microseconds, less than marshalling their
// dozen tensors through Python attributes takes (16 us for exact attention, 23 us
// for an append on a Grace core); here the same checks take about 1 us.

#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "../../include/dkv.h"

namespace {

constexpr int64_t kPage = 16;

// Classes of the package, set once by setup().
PyObject* g_q4 = nullptr;
PyObject* g_paged = nullptr;
PyObject* g_fp8 = nullptr;
PyObject* g_fp8_paged = nullptr;
PyObject* g_meta8 = nullptr;
PyObject* g_error = nullptr;
PyObject* g_latent = nullptr;

struct PyError {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw PyError{};
}
[[noreturn]] void value_error(const char* text) { raise(PyExc_ValueError, text); }

bool is_none(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw PyError{};
  }
  return THPVariable_Unpack(o);
}

const at::Tensor* optional_tensor(PyObject* o, const char* name) {
  return is_none(o) ? nullptr : &tensor(o, name);
}

// Memory of which only the size counts (a workspace, a reuse state), or null: it
// is used from its first byte on, so a view must not leave any out.
const at::Tensor* scratch(PyObject* o, const char* name) {
  const at::Tensor* t = optional_tensor(o, name);
  if (t != nullptr && !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    throw PyError{};
  }
  return t;
}

int dtype_code(at::ScalarType t) {
  if (t == at::kBFloat16) return DKV_BF16;
  if (t == at::kHalf) return DKV_FP16;
  if (t == at::kFloat) return DKV_FP32;
  raise(PyExc_TypeError, "unsupported dtype");
}

at::ScalarType scalar_type(PyObject* o) {
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int64_t integer(PyObject* o) {  // as int(o)
  PyObject* n = PyNumber_Long(o);
  if (n == nullptr) throw PyError{};
  const long long v = PyLong_AsLongLong(n);
  Py_DECREF(n);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return v;
}

int cuda_index(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

int32_t int32_size(int64_t v) {
  if (v < 0 || v >= (int64_t{1} << 31)) value_error("a size is out of range");
  return static_cast<int32_t>(v);
}

// A count as the library takes it, which refuses those below 1 with its status.
int32_t int32_count(int64_t v) {
  return static_cast<int32_t>(v < -1 ? -1 : (v > INT32_MAX ? INT32_MAX : v));
}

// A K or V cache, as the package's calls take it.
struct Cache {
  dkv_kv kv{};
  int64_t B = 0, H = 0, N = 0, d = 0;
  at::ScalarType dtype = at::kBFloat16;  // of q and the page metadata
  int device = -1;
  bool fp8 = false;
  bool same_shape(const Cache& o) const { return B == o.B && H == o.H && N == o.N && d == o.d; }
};

bool is(PyObject* o, PyObject* cls) {
  return Py_TYPE(o) == reinterpret_cast<PyTypeObject*>(cls) || PyObject_IsInstance(o, cls) == 1;
}

Cache parse_cache(PyObject* o) {
  Cache c;
  dkv_kv& s = c.kv;
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != 4) value_error("K/V must be [B, Hkv, N, d]");
    c.B = t.size(0), c.H = t.size(1), c.N = t.size(2), c.d = t.size(3);
    if (t.stride(3) != 1 || t.stride(2) != c.d)
      value_error("K/V must have token stride d and channel stride 1");
    s.format = DKV_KV_DENSE;
    c.dtype = t.scalar_type();
    s.data = t.data_ptr();
    s.stride_b = t.stride(0), s.stride_h = t.stride(1);
    c.device = cuda_index(t);
  } else if (is(o, g_paged) || is(o, g_fp8_paged)) {
    c.fp8 = is(o, g_fp8_paged);
    const at::Tensor& pool = tensor(PyTuple_GET_ITEM(o, 0), "pool");
    const int at = c.fp8 ? 2 : 1;
    const at::Tensor& bt = tensor(PyTuple_GET_ITEM(o, at), "block_table");
    c.N = integer(PyTuple_GET_ITEM(o, at + 1));
    if (pool.dim() != 4 || pool.size(2) != kPage || pool.stride(3) != 1 ||
        pool.stride(2) != pool.size(3))
      value_error("pool must be [num_blocks, Hkv, 16, d] with token stride d");
    c.H = pool.size(1), c.d = pool.size(3);
    c.device = cuda_index(pool);
    if (c.fp8) {
      const at::Tensor& sc = tensor(PyTuple_GET_ITEM(o, 1), "scale");
      if (pool.scalar_type() != at::kFloat8_e4m3fn || sc.scalar_type() != at::kFloat)
        raise(PyExc_TypeError, "Fp8PagedCache wants a float8_e4m3fn pool and float32 scales");
      if (sc.dim() != 2 || sc.size(0) != pool.size(0) || sc.size(1) != c.H ||
          cuda_index(sc) != c.device)
        value_error("scale must be [num_blocks, Hkv]");
      s.scale = static_cast<const float*>(sc.data_ptr());
      s.sstride_b = sc.stride(0), s.sstride_h = sc.stride(1);
      c.dtype = scalar_type(PyTuple_GET_ITEM(o, 4));
    } else {
      c.dtype = pool.scalar_type();
    }
    if (bt.scalar_type() != at::kInt || bt.dim() != 2 || bt.stride(1) != 1)
      value_error("block_table must be int32 [B, P] with unit column stride");
    if (cuda_index(bt) != c.device) value_error("block_table must be on the pool's device");
    if (bt.size(1) < (c.N + kPage - 1) / kPage)
      value_error("block_table has fewer than ceil(seq_len / 16) columns");
    c.B = bt.size(0);
    s.format = c.fp8 ? DKV_KV_FP8_PAGED : DKV_KV_PAGED;
    s.data = pool.data_ptr();
    s.stride_b = pool.stride(0), s.stride_h = pool.stride(1);
    s.block_table = static_cast<const int32_t*>(bt.data_ptr());
    s.block_table_stride = bt.stride(0);
    s.num_blocks = int32_size(pool.size(0));
  } else if (is(o, g_fp8)) {
    c.fp8 = true;
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, 0), "codes");
    const at::Tensor& sc = tensor(PyTuple_GET_ITEM(o, 1), "scale");
    c.dtype = scalar_type(PyTuple_GET_ITEM(o, 2));
    if (t.scalar_type() != at::kFloat8_e4m3fn || sc.scalar_type() != at::kFloat)
      raise(PyExc_TypeError, "Fp8Cache wants float8_e4m3fn codes and float32 scales");
    if (t.dim() != 4 || t.stride(3) != 1 || t.stride(2) != t.size(3))
      value_error("codes must have token stride d and channel stride 1");
    c.B = t.size(0), c.H = t.size(1), c.N = t.size(2), c.d = t.size(3);
    c.device = cuda_index(t);
    const int64_t P = (c.N + kPage - 1) / kPage;
    if (sc.dim() != 3 || sc.size(0) != c.B || sc.size(1) != c.H || sc.size(2) != P ||
        (sc.stride(2) != 1 && P > 1) || cuda_index(sc) != c.device)
      value_error("scale must be [B, Hkv, ceil(N / 16)] with unit block stride");
    s.format = DKV_KV_FP8;
    s.data = t.data_ptr();
    s.stride_b = t.stride(0), s.stride_h = t.stride(1);
    s.scale = static_cast<const float*>(sc.data_ptr());
    s.sstride_b = sc.stride(0), s.sstride_h = sc.stride(1);
  } else if (is(o, g_q4)) {
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, 0), "codes");
    const at::Tensor& mn = tensor(PyTuple_GET_ITEM(o, 1), "gmin");
    const at::Tensor& mx = tensor(PyTuple_GET_ITEM(o, 2), "gmax");
    if (t.scalar_type() != at::kByte || mn.scalar_type() != at::kHalf ||
        mx.scalar_type() != at::kHalf)
      raise(PyExc_TypeError, "Q4Cache wants uint8 codes and fp16 gmin/gmax");
    if (t.dim() != 4 || t.stride(3) != 1 || t.stride(2) != t.size(3))
      value_error("codes must have token stride d/2 and channel stride 1");
    c.B = t.size(0), c.H = t.size(1), c.N = t.size(2), c.d = 2 * t.size(3);
    if (mn.strides() != mx.strides() || mn.dim() != 4 || mn.stride(3) != 1 ||
        mn.stride(2) != c.d / 64)
      value_error("gmin / gmax must share strides with token stride d/64");
    for (const at::Tensor* m : {&mn, &mx})
      if (m->dim() != 4 || m->size(0) < c.B || m->size(1) < c.H || m->size(2) < c.N ||
          m->size(3) < c.d / 64 || m->device() != t.device())
        value_error("gmin / gmax must hold [B, Hkv, N, d/64] on the codes' device");
    s.format = DKV_KV_Q4G64;
    c.dtype = at::kHalf;
    s.data = t.data_ptr();
    s.gmin = mn.data_ptr(), s.gmax = mx.data_ptr();
    s.stride_b = t.stride(0), s.stride_h = t.stride(1);
    s.gstride_b = mn.stride(0), s.gstride_h = mn.stride(1);
    c.device = cuda_index(t);
  } else {
    raise(PyExc_TypeError, "K/V must be a tensor or one of the package's cache tuples");
  }
  s.dtype = dtype_code(c.dtype);
  return c;
}

// A pair of caches of one shape.
struct Pair {
  Cache k, v;
};
Pair parse_pair(PyObject* K, PyObject* V) {
  Pair p{parse_cache(K), parse_cache(V)};
  if (!p.k.same_shape(p.v)) value_error("K and V shapes differ");
  return p;
}

// int32 lengths [B] on the device, or NULL.
const int32_t* lengths(PyObject* o, const char* name, int64_t B, int device) {
  if (is_none(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != B || !t.is_contiguous() ||
      !t.is_cuda() || t.get_device() != device) {
    PyErr_Format(PyExc_ValueError,
                 "%s must be a contiguous int32 CUDA tensor [B] on the cache's device", name);
    throw PyError{};
  }
  return static_cast<const int32_t*>(t.data_ptr());
}

dkv_params make_params(const Cache& c, int64_t page_size, PyObject* seq_lens) {
  dkv_params p{};
  p.batch = int32_size(c.B);
  p.num_q_heads = p.num_kv_heads = int32_size(c.H);
  p.head_dim = int32_size(c.d);
  p.seq_len = int32_size(c.N);
  p.page_size = int32_size(page_size);
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.d)));
  p.seq_lens = lengths(seq_lens, "seq_lens", c.B, c.device);
  return p;
}

// The query and output of an attention call.
void set_query(dkv_params* p, const Cache& c, const at::Tensor& q, PyObject* scale,
               int64_t flags) {
  if (q.dim() < 3 || q.size(0) != c.B || q.size(2) != c.d || q.stride(2) != 1)
    value_error("q's shape does not match the cache");
  p->num_q_heads = int32_size(q.size(1));
  p->q_stride_b = q.stride(0), p->q_stride_h = q.stride(1);
  if (!is_none(scale)) p->scale = static_cast<float>(number(scale));
  p->flags = static_cast<uint32_t>(flags);
}
// (A row of out may be split into more dimensions, [B, Hq, 1, d] say: d elements
// one after the other are what counts.)
void set_out(dkv_params* p, const at::Tensor& q, const at::Tensor& out) {
  bool ok = out.dim() >= 3 && out.size(0) >= q.size(0) && out.size(1) >= q.size(1);
  int64_t run = 1;  // elements of a row that follow one another
  for (int64_t i = out.dim() - 1; ok && i >= 2 && run < q.size(2); --i) {
    ok = out.stride(i) == run || out.size(i) == 1;
    run *= out.size(i);
  }
  if (!ok || run < q.size(2)) value_error("out must hold [B, Hq, d] with channel stride 1");
  p->o_stride_b = out.stride(0), p->o_stride_h = out.stride(1);
}

at::Tensor new_out(const at::Tensor& q, PyObject* dtype) {
  return at::empty({q.size(0), q.size(1), q.size(2)}, q.options().dtype(scalar_type(dtype)));
}

// The tensors of an attention call lie on one device; q has the cache's type (4-bit: fp16).
void check_tensors(const at::Tensor& q, const Pair& c,
                   std::initializer_list<const at::Tensor*> others) {
  if (q.scalar_type() != c.k.dtype) value_error("q must have the cache's dtype");
  const int dev = cuda_index(q);
  bool ok = dev >= 0 && c.k.device == dev && c.v.device == dev;
  for (const at::Tensor* t : others) ok = ok && (t == nullptr || cuda_index(*t) == dev);
  if (!ok) value_error("q, the caches and the other tensors must be on one CUDA device");
}

size_t workspace_need(const dkv_params& p, int top_k, bool fp8) {
  return fp8 ? dkv_workspace_bytes_fp8(&p, top_k) : dkv_workspace_bytes(&p, top_k);
}

// The caller's workspace, or a new one.
at::Tensor workspace_for(PyObject* o, size_t need, const at::Tensor& q) {
  if (is_none(o))
    return at::zeros({static_cast<int64_t>(need)}, q.options().dtype(at::kByte));
  const at::Tensor& t = *scratch(o, "workspace");
  if (static_cast<size_t>(t.numel()) * t.element_size() < need) value_error("workspace too small");
  return t;
}

// Other Python threads run meanwhile.  (An object, not the macro pair: a tensor
// without memory throws when its address is taken, and the exception is turned
// into a Python one, which needs the interpreter's lock.)
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// One library call on the current stream of CUDA device `dev`, which is made the
// current device for it; raises on an error status.
template <typename F>
void call(const char* where, int dev, const F& f) {
  if (dev < 0) {
    PyErr_Format(PyExc_ValueError, "%s wants CUDA tensors", where);
    throw PyError{};
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  const dkv_status st = [&] {
    const Unlocked unlocked;
    return f(stream);
  }();
  if (st != DKV_OK) {
    PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), where);
    if (e != nullptr) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw PyError{};
  }
}

PyObject* incref(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// ------------------------------------------------------------------- the calls
PyObject* setup(PyObject* const* a) {
  PyObject** to[] = {&g_q4, &g_paged, &g_fp8, &g_fp8_paged, &g_meta8, &g_error, &g_latent};
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(a[i]);
    *to[i] = a[i];
  }
  Py_RETURN_NONE;
}

// A cache's struct fields, then (B, Hkv, N, d): for callers of the C ABI.
PyObject* describe_cache(PyObject* const* a) {
  const Cache c = parse_cache(a[0]);
  const dkv_kv& s = c.kv;
  auto p = [](const void* x) { return reinterpret_cast<unsigned long long>(x); };
  return Py_BuildValue("((iiKKKLLLLKLiKLL)LLLL)", s.format, s.dtype, p(s.data), p(s.gmin),
                       p(s.gmax), (long long)s.stride_b, (long long)s.stride_h,
                       (long long)s.gstride_b, (long long)s.gstride_h, p(s.block_table),
                       (long long)s.block_table_stride, s.num_blocks, p(s.scale),
                       (long long)s.sstride_b, (long long)s.sstride_h, (long long)c.B,
                       (long long)c.H, (long long)c.N, (long long)c.d);
}

// kv_meta_build(K, page_size, seq_lens)
PyObject* kv_meta_build(PyObject* const* a) {
  const Cache c = parse_cache(a[0]);
  const int64_t S = integer(a[1]);
  const dkv_params p = make_params(c, S, a[2]);
  if (c.device < 0) value_error("dkv_kv_meta_build wants CUDA tensors");
  const int64_t P = S > 0 ? (c.N + S - 1) / S : 0;
  const auto opt = at::TensorOptions().dtype(c.dtype).device(
      at::kCUDA, static_cast<c10::DeviceIndex>(c.device));
  const at::Tensor mn = at::empty({c.B, c.H, P, c.d}, opt);
  const at::Tensor mx = at::empty({c.B, c.H, P, c.d}, opt);
  call("dkv_kv_meta_build", c.device, [&](void* stream) {
    return dkv_kv_meta_build(&p, &c.kv, mn.data_ptr(), mx.data_ptr(), stream);
  });
  return Py_BuildValue("(NN)", THPVariable_Wrap(mn), THPVariable_Wrap(mx));
}

// The two tensors of 16-bit page metadata, checked against the cache.
struct Meta {
  const at::Tensor *mn, *mx;
};
Meta meta_pair(PyObject* o, const Cache& c, int64_t P) {
  if ((!PyTuple_Check(o) && !PyList_Check(o)) || PySequence_Fast_GET_SIZE(o) != 2)
    value_error("meta must be (meta_min, meta_max)");
  const Meta m{&tensor(PySequence_Fast_GET_ITEM(o, 0), "meta_min"),
               &tensor(PySequence_Fast_GET_ITEM(o, 1), "meta_max")};
  for (const at::Tensor* t : {m.mn, m.mx}) {
    if (t->dim() != 4 || t->size(0) != c.B || t->size(1) != c.H || t->size(2) != P ||
        t->size(3) != c.d || !t->is_contiguous())
      value_error("meta must be contiguous [B, Hkv, P, d]");
    if (t->scalar_type() != c.dtype) value_error("meta must have the cache's dtype");
  }
  return m;
}

// kv_meta_append(K, meta, page_size, seq_lens, new_tokens, new_lens)
PyObject* kv_meta_append(PyObject* const* a) {
  const Cache c = parse_cache(a[0]);
  const int64_t S = integer(a[2]);
  const dkv_params p = make_params(c, S, a[3]);
  const Meta m = meta_pair(a[1], c, S > 0 ? (c.N + S - 1) / S : 0);
  if (cuda_index(*m.mn) != c.device || cuda_index(*m.mx) != c.device)
    value_error("meta must be on the cache's device");
  const int32_t* news = lengths(a[5], "new_lens", c.B, c.device);
  if (news != nullptr && is_none(a[4])) value_error("new_lens needs new_tokens");
  const int32_t fresh = is_none(a[4]) ? 1 : int32_count(integer(a[4]));
  call("dkv_kv_meta_append", c.device, [&](void* stream) {
    return dkv_kv_meta_append_tokens(&p, &c.kv, fresh, news, m.mn->data_ptr(), m.mx->data_ptr(),
                                     stream);
  });
  Py_RETURN_NONE;
}

// Rows [B, T, H, d] of new tokens: address and (batch, token, head) strides.
struct Rows {
  void* p = nullptr;
  int64_t sb = 0, st = 0, sh = 0;
};
Rows rows(const at::Tensor& t, const char* name, const Cache& c, int64_t T, int64_t H) {
  if (t.dim() != 4 || t.size(0) != c.B || t.size(1) != T || t.size(2) != H || t.size(3) != c.d ||
      t.stride(3) != 1 || t.scalar_type() != c.dtype || cuda_index(t) != c.device) {
    PyErr_Format(PyExc_ValueError,
                 "%s must be [B, T, heads, d] with channel stride 1, in the caches' dtype and on "
                 "their device",
                 name);
    throw PyError{};
  }
  return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

// kv_append(k, v, K, V, seq_lens, new_lens, q, q_out, rope, interleaved, workspace)
PyObject* kv_append(PyObject* const* a) {
  const Pair c = parse_pair(a[2], a[3]);
  if (c.k.device < 0 || c.v.device != c.k.device)
    value_error("K and V must be on one CUDA device");
  const int dev = c.k.device;
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  if (k.dim() != 4) value_error("k must be [B, T, Hkv, d]");
  const int64_t T = k.size(1);
  dkv_append p{};
  p.batch = int32_size(c.k.B);
  p.num_kv_heads = int32_size(c.k.H);
  p.head_dim = int32_size(c.k.d);
  p.seq_len = int32_size(c.k.N);
  p.new_tokens = int32_size(T);
  const Rows rk = rows(k, "k", c.k, T, c.k.H), rv = rows(v, "v", c.k, T, c.k.H);
  p.k = rk.p, p.k_stride_b = rk.sb, p.k_stride_t = rk.st, p.k_stride_h = rk.sh;
  p.v = rv.p, p.v_stride_b = rv.sb, p.v_stride_t = rv.st, p.v_stride_h = rv.sh;
  std::optional<at::Tensor> made;
  if (!is_none(a[6])) {
    const at::Tensor& q = tensor(a[6], "q");
    if (q.dim() != 4) value_error("q must be [B, T, Hq, d]");
    const int64_t Hq = q.size(2);
    const Rows rq = rows(q, "q", c.k, T, Hq);
    // (rows that no token has are left as they are)
    if (is_none(a[7])) made = at::empty({c.k.B, T, Hq, c.k.d}, q.options());
    const Rows ro = rows(made ? *made : tensor(a[7], "q_out"), "q_out", c.k, T, Hq);
    p.num_q_heads = int32_size(Hq);
    p.q = rq.p, p.q_stride_b = rq.sb, p.q_stride_t = rq.st, p.q_stride_h = rq.sh;
    p.q_out = ro.p, p.o_stride_b = ro.sb, p.o_stride_t = ro.st, p.o_stride_h = ro.sh;
  } else if (!is_none(a[7])) {
    value_error("q_out without q");
  }
  if (!is_none(a[8])) {
    if ((!PyTuple_Check(a[8]) && !PyList_Check(a[8])) || PySequence_Fast_GET_SIZE(a[8]) != 2)
      value_error("rope must be (cos, sin)");
    const at::Tensor& cs = tensor(PySequence_Fast_GET_ITEM(a[8], 0), "cos");
    const at::Tensor& sn = tensor(PySequence_Fast_GET_ITEM(a[8], 1), "sin");
    if (cs.dim() != 2 || cs.sizes() != sn.sizes() || cs.scalar_type() != at::kFloat ||
        sn.scalar_type() != at::kFloat || cuda_index(cs) != dev || cuda_index(sn) != dev ||
        !cs.is_contiguous() || !sn.is_contiguous())
      value_error("rope must be two contiguous float32 [positions, r / 2] tables");
    p.rope_len = int32_size(cs.size(0));
    p.rotary_dim = int32_size(2 * cs.size(1));
    p.cos = static_cast<const float*>(cs.data_ptr());
    p.sin = static_cast<const float*>(sn.data_ptr());
  }
  const int il = PyObject_IsTrue(a[9]);
  if (il < 0) throw PyError{};
  p.interleaved = il;
  p.seq_lens = lengths(a[4], "seq_lens", c.k.B, dev);
  p.new_lens = lengths(a[5], "new_lens", c.k.B, dev);
  void* ws = nullptr;
  if (const at::Tensor* t = scratch(a[10], "workspace")) {
    if (cuda_index(*t) != dev ||
        static_cast<size_t>(t->numel()) * t->element_size() < DKV_WORKSPACE_HEADER_BYTES)
      value_error("workspace must hold 256 bytes on the caches' device");
    ws = t->data_ptr();
  }
  if (T > 0)  // (an empty tensor has no address)
    call("dkv_kv_append", dev,
         [&](void* stream) { return dkv_kv_append(&p, &c.k.kv, &c.v.kv, ws, stream); });
  if (made) return THPVariable_Wrap(*made);
  return incref(is_none(a[7]) ? Py_None : a[7]);
}

// decode_attn_full(q, K, V, scale, out_dtype, out, workspace, flags, seq_lens)
PyObject* decode_attn_full(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const Pair c = parse_pair(a[1], a[2]);
  const at::Tensor* given = optional_tensor(a[5], "out");
  check_tensors(q, c, {given, scratch(a[6], "workspace")});
  dkv_params p = make_params(c.k, kPage, a[8]);
  set_query(&p, c.k, q, a[3], integer(a[7]));
  const int dev = cuda_index(q);
  const at::Tensor out = given ? *given : new_out(q, a[4]);
  set_out(&p, q, out);
  const size_t need = workspace_need(p, 0, c.k.fp8);
  const at::Tensor ws = workspace_for(a[6], need, q);
  const int code = dtype_code(out.scalar_type());
  call("dkv_decode_attn_full", dev, [&](void* stream) {
    return dkv_decode_attn_full(&p, q.data_ptr(), &c.k.kv, &c.v.kv, out.data_ptr(), code,
                                ws.data_ptr(), need, stream);
  });
  return given ? incref(a[5]) : THPVariable_Wrap(out);
}

// decode_attn_select(q, K, V, meta, top_k, scale, out_dtype, out, return_selected, selected,
//                    workspace, flags, seq_lens, page_size, hot, step)
PyObject* decode_attn_select(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const Pair c = parse_pair(a[1], a[2]);
  const int64_t S = integer(a[13]);
  const int32_t top_k = int32_count(integer(a[4]));
  const int64_t P = S > 0 ? (c.k.N + S - 1) / S : 0;
  const at::Tensor* given = optional_tensor(a[7], "out");
  const at::Tensor* chosen = optional_tensor(a[9], "selected");
  const at::Tensor* hot = scratch(a[14], "hot");
  const bool m8 = is(a[3], g_meta8);
  if (m8 && hot != nullptr) value_error("cross-step reuse takes 16-bit metadata");
  Meta m{};
  const at::Tensor* part[4] = {};  // Meta8: code_min, code_max, lo, step
  if (m8) {
    for (int i = 0; i < 4; ++i) {
      part[i] = &tensor(PyTuple_GET_ITEM(a[3], i), "Meta8");
      const at::Tensor& t = *part[i];
      if (t.dim() != (i < 2 ? 4 : 3) || t.size(0) != c.k.B || t.size(1) != c.k.H ||
          t.size(2) != P || (i < 2 && t.size(3) != c.k.d) || !t.is_contiguous())
        value_error("Meta8 must hold contiguous [B, Hkv, P, d] codes, [B, Hkv, P] grid");
      if (t.scalar_type() != (i < 2 ? at::kByte : at::kFloat))
        value_error("Meta8 must have the dtypes uint8 (codes) and float32 (grid)");
    }
  } else {
    m = meta_pair(a[3], c.k, P);
  }
  check_tensors(q, c, {given, scratch(a[10], "workspace"), chosen, hot, m.mn, m.mx,
                       part[0], part[1], part[2], part[3]});
  dkv_params p = make_params(c.k, S, a[12]);
  set_query(&p, c.k, q, a[5], integer(a[11]));
  const int dev = cuda_index(q);
  const at::Tensor out = given ? *given : new_out(q, a[6]);
  set_out(&p, q, out);
  const int64_t kk = top_k < 0 ? 0 : (top_k < P ? top_k : P);
  const int wanted = PyObject_IsTrue(a[8]);
  if (wanted < 0) throw PyError{};
  std::optional<at::Tensor> made;
  if (chosen != nullptr) {
    if (chosen->scalar_type() != at::kInt || !chosen->is_contiguous() ||
        chosen->numel() < c.k.B * q.size(1) * kk)
      value_error("selected must hold a contiguous int32 [B, Hq, min(top_k, P)]");
  } else if (wanted) {
    made = at::empty({c.k.B, q.size(1), kk}, q.options().dtype(at::kInt));
    chosen = &*made;
  }
  const size_t need = workspace_need(p, top_k, c.k.fp8);
  const at::Tensor ws = workspace_for(a[10], need, q);
  const int code = dtype_code(out.scalar_type());
  int32_t* sel = chosen != nullptr ? static_cast<int32_t*>(chosen->data_ptr()) : nullptr;
  const void* qp = q.data_ptr();
  void *op = out.data_ptr(), *wp = ws.data_ptr();
  if (m8) {
    call("dkv_decode_attn_select_meta8", dev, [&](void* stream) {
      return dkv_decode_attn_select_meta8(&p, qp, &c.k.kv, &c.v.kv, part[0]->data_ptr(),
                                          part[1]->data_ptr(), part[2]->data_ptr(),
                                          part[3]->data_ptr(), top_k, op, code, sel, wp, need,
                                          stream);
    });
  } else if (hot != nullptr) {
    const int32_t step = int32_count(integer(a[15]));
    const size_t bytes = static_cast<size_t>(hot->numel()) * hot->element_size();
    call("dkv_decode_attn_select_hot", dev, [&](void* stream) {
      return dkv_decode_attn_select_hot(&p, qp, &c.k.kv, &c.v.kv, m.mn->data_ptr(),
                                        m.mx->data_ptr(), top_k, op, code, sel, hot->data_ptr(),
                                        bytes, step, wp, need, stream);
    });
  } else {
    call("dkv_decode_attn_select", dev, [&](void* stream) {
      return dkv_decode_attn_select(&p, qp, &c.k.kv, &c.v.kv, m.mn->data_ptr(), m.mx->data_ptr(),
                                    top_k, op, code, sel, wp, need, stream);
    });
  }
  PyObject* o = given ? incref(a[7]) : THPVariable_Wrap(out);
  if (!wanted) return o;
  return Py_BuildValue("(NN)", o, made ? THPVariable_Wrap(*made) : incref(a[9]));
}

// ----------------------------------------------------------------- latent caches
struct Latent {
  dkv_latent_cache c{};
  at::ScalarType dtype = at::kBFloat16;
  int64_t B = 0, N = 0, width = 0;
  int device = -1;
};

// A dense tensor [B, N, dc + 64] or a LatentCache.
Latent parse_latent(PyObject* o) {
  Latent l;
  dkv_latent_cache& c = l.c;
  const at::Tensor* t;
  if (THPVariable_Check(o)) {
    t = &THPVariable_Unpack(o);
    if (t->dim() != 3 || t->stride(2) != 1)
      value_error("a latent cache must be [B, N, latent + rope] with channel stride 1");
    l.B = t->size(0), l.N = t->size(1);
  } else if (is(o, g_latent)) {
    t = &tensor(PyTuple_GET_ITEM(o, 0), "pool");
    const at::Tensor& bt = tensor(PyTuple_GET_ITEM(o, 1), "block_table");
    l.N = integer(PyTuple_GET_ITEM(o, 2));
    if (t->dim() != 3 || t->stride(2) != 1)
      value_error("pool must be [num_blocks, block_size, latent + rope] with channel stride 1");
    if (bt.scalar_type() != at::kInt || bt.dim() != 2 || (bt.stride(1) != 1 && bt.size(1) > 1))
      value_error("block_table must be int32 [B, P] with unit column stride");
    if (cuda_index(bt) != cuda_index(*t)) value_error("block_table must be on the pool's device");
    c.block_size = int32_size(t->size(1));
    if (c.block_size != 16 && c.block_size != 32 && c.block_size != 64)
      value_error("a latent pool's blocks hold 16, 32 or 64 tokens");
    if (l.N < 1 || bt.size(1) < (l.N + c.block_size - 1) / c.block_size)
      value_error("block_table has fewer than ceil(seq_len / block_size) columns");
    l.B = bt.size(0);
    c.num_blocks = int32_size(t->size(0));
    c.block_table = static_cast<const int32_t*>(bt.data_ptr());
    c.block_table_stride = bt.stride(0);
  } else {
    raise(PyExc_TypeError, "a latent cache is a tensor or a LatentCache");
  }
  l.width = t->size(2);
  l.dtype = t->scalar_type();
  l.device = cuda_index(*t);
  c.dtype = dtype_code(l.dtype);
  c.rope_dim = 64;
  c.latent_dim = int32_size(l.width - 64 < 0 ? 0 : l.width - 64);
  c.seq_len = int32_size(l.N);
  c.data = t->data_ptr();
  // (the stride of a dimension of size 1 says nothing)
  c.stride_t = t->size(1) > 1 ? t->stride(1) : l.width;
  c.stride_b = t->size(0) > 1 ? t->stride(0) : 0;
  return l;
}

// A tensor of an exact shape with channel stride 1, in the given dtype and on the device.
const at::Tensor& shaped(PyObject* o, const char* name, at::IntArrayRef shape,
                         at::ScalarType dtype, int device) {
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || t.scalar_type() != dtype || cuda_index(t) != device ||
      (t.numel() > 0 && t.size(-1) > 1 && t.stride(-1) != 1)) {
    PyErr_Format(PyExc_ValueError,
                 "%s has another shape, dtype or device than the call's other tensors, or no "
                 "channel stride of 1",
                 name);
    throw PyError{};
  }
  return t;
}

// The stride of dimension i, 0 where it has one element.
int64_t stride_of(const at::Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// The 256 bytes where a call records what it refused on the device, or NULL.
void* status_word(PyObject* o, int device) {
  const at::Tensor* t = scratch(o, "workspace");
  if (t == nullptr) return nullptr;
  if (cuda_index(*t) != device ||
      static_cast<size_t>(t->numel()) * t->element_size() < DKV_WORKSPACE_HEADER_BYTES)
    value_error("workspace must hold 256 bytes on the caches' device");
  return t->data_ptr();
}

// latent_append(c, k_rope, cache, seq_lens, new_lens, q_rope, q_out, rope, norm, eps,
//               interleaved, workspace)
PyObject* latent_append(PyObject* const* a) {
  const Latent l = parse_latent(a[2]);
  const int dev = l.device;
  if (dev < 0) value_error("latent_append wants CUDA tensors");
  const int64_t dc = l.c.latent_dim;
  const at::Tensor& c0 = tensor(a[0], "c");
  if (c0.dim() != 3) value_error("c must be [B, T, latent]");
  const int64_t T = c0.size(1);
  const at::Tensor& c = shaped(a[0], "c", {l.B, T, dc}, l.dtype, dev);
  const at::Tensor& k = shaped(a[1], "k_rope", {l.B, T, 64}, l.dtype, dev);
  dkv_latent_append_args p{};
  p.batch = int32_size(l.B);
  p.new_tokens = int32_size(T);
  p.c = c.data_ptr(), p.c_stride_b = stride_of(c, 0), p.c_stride_t = stride_of(c, 1);
  p.k = k.data_ptr(), p.k_stride_b = stride_of(k, 0), p.k_stride_t = stride_of(k, 1);
  std::optional<at::Tensor> made;
  if (!is_none(a[5])) {
    const at::Tensor& q0 = tensor(a[5], "q_rope");
    if (q0.dim() != 4) value_error("q_rope must be [B, T, H, 64]");
    const int64_t H = q0.size(2);
    const at::Tensor& q = shaped(a[5], "q_rope", {l.B, T, H, 64}, l.dtype, dev);
    // (rows that no token has are left as they are)
    if (is_none(a[6])) made = at::empty({l.B, T, H, 64}, q.options());
    const at::Tensor& o = made ? *made : shaped(a[6], "q_out", {l.B, T, H, 64}, l.dtype, dev);
    p.num_q_heads = int32_size(H);
    p.q = q.data_ptr();
    p.q_stride_b = stride_of(q, 0), p.q_stride_t = stride_of(q, 1), p.q_stride_h = stride_of(q, 2);
    p.q_out = o.data_ptr();
    p.o_stride_b = stride_of(o, 0), p.o_stride_t = stride_of(o, 1), p.o_stride_h = stride_of(o, 2);
  } else if (!is_none(a[6])) {
    value_error("q_out without q_rope");
  }
  if (!is_none(a[7])) {
    if ((!PyTuple_Check(a[7]) && !PyList_Check(a[7])) || PySequence_Fast_GET_SIZE(a[7]) != 2)
      value_error("rope must be (cos, sin)");
    const at::Tensor& cs = tensor(PySequence_Fast_GET_ITEM(a[7], 0), "cos");
    const at::Tensor& sn = tensor(PySequence_Fast_GET_ITEM(a[7], 1), "sin");
    if (cs.dim() != 2 || cs.size(1) != 32 || cs.size(0) < 1 || cs.sizes() != sn.sizes() ||
        cs.scalar_type() != at::kFloat || sn.scalar_type() != at::kFloat || cuda_index(cs) != dev ||
        cuda_index(sn) != dev || !cs.is_contiguous() || !sn.is_contiguous())
      value_error("rope must be two contiguous float32 [positions, 32] tables");
    p.rope_len = int32_size(cs.size(0));
    p.cos = static_cast<const float*>(cs.data_ptr());
    p.sin = static_cast<const float*>(sn.data_ptr());
  }
  if (!is_none(a[8])) {
    const at::Tensor& w = shaped(a[8], "norm", {dc}, l.dtype, dev);
    p.norm = w.data_ptr();
  }
  p.eps = static_cast<float>(number(a[9]));
  const int il = PyObject_IsTrue(a[10]);
  if (il < 0) throw PyError{};
  p.interleaved = il;
  p.seq_lens = lengths(a[3], "seq_lens", l.B, dev);
  p.new_lens = lengths(a[4], "new_lens", l.B, dev);
  void* ws = status_word(a[11], dev);
  if (T > 0)  // (an empty tensor has no address)
    call("dkv_latent_append", dev,
         [&](void* stream) { return dkv_latent_append(&p, &l.c, ws, stream); });
  if (made) return THPVariable_Wrap(*made);
  return incref(is_none(a[6]) ? Py_None : a[6]);
}

// latent_decode_attn(q_latent, q_rope, cache, scale, seq_lens, new_lens, out_dtype, out,
//                    workspace, flags)
PyObject* latent_decode_attn(PyObject* const* a) {
  const Latent l = parse_latent(a[2]);
  const int dev = l.device;
  if (dev < 0) value_error("latent_decode_attn wants CUDA tensors");
  const int64_t dc = l.c.latent_dim;
  const at::Tensor& q0 = tensor(a[0], "q_latent");
  if (q0.dim() != 4) value_error("q_latent must be [B, T, H, latent]");
  const int64_t T = q0.size(1), H = q0.size(2);
  const at::Tensor& ql = shaped(a[0], "q_latent", {l.B, T, H, dc}, l.dtype, dev);
  const at::Tensor& qr = shaped(a[1], "q_rope", {l.B, T, H, 64}, l.dtype, dev);
  at::Tensor out;
  if (is_none(a[7])) {
    // (rows that no token has are left as they are: here 0)
    const auto opt = ql.options().dtype(scalar_type(a[6]));
    out = is_none(a[5]) ? at::empty({l.B, T, H, dc}, opt) : at::zeros({l.B, T, H, dc}, opt);
  } else {
    out = tensor(a[7], "out");
    shaped(a[7], "out", {l.B, T, H, dc}, out.scalar_type(), dev);
  }
  dkv_latent_attn p{};
  p.batch = int32_size(l.B);
  p.num_heads = int32_size(H);
  p.new_tokens = int32_size(T);
  p.flags = static_cast<uint32_t>(integer(a[9]));
  p.scale = static_cast<float>(number(a[3]));
  p.out_dtype = dtype_code(out.scalar_type());
  p.q_latent = ql.data_ptr(), p.q_rope = qr.data_ptr(), p.out = out.data_ptr();
  p.ql_stride_b = stride_of(ql, 0), p.ql_stride_t = stride_of(ql, 1), p.ql_stride_h = stride_of(ql, 2);
  p.qr_stride_b = stride_of(qr, 0), p.qr_stride_t = stride_of(qr, 1), p.qr_stride_h = stride_of(qr, 2);
  p.o_stride_b = stride_of(out, 0), p.o_stride_t = stride_of(out, 1), p.o_stride_h = stride_of(out, 2);
  p.seq_lens = lengths(a[4], "seq_lens", l.B, dev);
  p.new_lens = lengths(a[5], "new_lens", l.B, dev);
  const size_t need = dkv_latent_workspace_bytes(&p, &l.c);
  const at::Tensor ws = workspace_for(a[8], need, ql);
  if (cuda_index(ws) != dev) value_error("workspace must be on the cache's device");
  call("dkv_latent_decode_attn", dev, [&](void* stream) {
    return dkv_latent_decode_attn(&p, &l.c, ws.data_ptr(), need, stream);
  });
  return is_none(a[7]) ? THPVariable_Wrap(out) : incref(a[7]);
}

// latent_prompt_attn(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale, causal, out_dtype,
//                    out, workspace, flags)
PyObject* latent_prompt_attn(PyObject* const* a) {
  const at::Tensor &q0 = tensor(a[0], "q_nope"), &k0 = tensor(a[2], "k_nope");
  if (q0.dim() != 3 || k0.dim() != 3) value_error("q_nope and k_nope must be [rows, H, nope]");
  const int dev = cuda_index(q0);
  if (dev < 0) value_error("latent_prompt_attn wants CUDA tensors");
  const at::ScalarType dt = q0.scalar_type();
  const int64_t Tq = q0.size(0), H = q0.size(1), dn = q0.size(2), Tk = k0.size(0);
  const at::Tensor& qn = shaped(a[0], "q_nope", {Tq, H, dn}, dt, dev);
  const at::Tensor& qr = shaped(a[1], "q_rope", {Tq, H, 64}, dt, dev);
  const at::Tensor& kn = shaped(a[2], "k_nope", {Tk, H, dn}, dt, dev);
  const at::Tensor& kr = shaped(a[3], "k_rope", {Tk, 64}, dt, dev);
  const at::Tensor& v = shaped(a[4], "v", {Tk, H, dn}, dt, dev);
  const at::Tensor& cu = tensor(a[5], "cu_q");
  if (cu.dim() != 1 || cu.size(0) < 2) value_error("cu_q must be int32 [B + 1]");
  const int64_t n = cu.size(0);
  dkv_prompt p{};
  p.cu_q = lengths(a[5], "cu_q", n, dev);
  p.cu_k = is_none(a[6]) ? p.cu_q : lengths(a[6], "cu_k", n, dev);
  at::Tensor out;
  if (is_none(a[10])) {  // (rows outside the sequences are left as they are: here 0)
    out = at::zeros({Tq, H, dn}, qn.options().dtype(scalar_type(a[9])));
  } else {
    out = tensor(a[10], "out");
    shaped(a[10], "out", {Tq, H, dn}, out.scalar_type(), dev);
  }
  p.batch = int32_size(n - 1);
  p.num_heads = int32_size(H);
  p.nope_dim = int32_size(dn);
  p.rope_dim = 64;
  p.dtype = dtype_code(dt);
  p.out_dtype = dtype_code(out.scalar_type());
  const int causal = PyObject_IsTrue(a[8]);
  if (causal < 0) throw PyError{};
  p.causal = causal;
  p.flags = static_cast<uint32_t>(integer(a[12]));
  p.scale = static_cast<float>(number(a[7]));
  p.total_q = int32_size(Tq);
  p.total_k = int32_size(Tk);
  p.q_nope = qn.data_ptr(), p.q_rope = qr.data_ptr(), p.out = out.data_ptr();
  p.k_nope = kn.data_ptr(), p.k_rope = kr.data_ptr(), p.v = v.data_ptr();
  p.qn_stride_t = stride_of(qn, 0), p.qn_stride_h = stride_of(qn, 1);
  p.qr_stride_t = stride_of(qr, 0), p.qr_stride_h = stride_of(qr, 1);
  p.kn_stride_t = stride_of(kn, 0), p.kn_stride_h = stride_of(kn, 1);
  p.v_stride_t = stride_of(v, 0), p.v_stride_h = stride_of(v, 1);
  p.kr_stride_t = stride_of(kr, 0);
  p.o_stride_t = stride_of(out, 0), p.o_stride_h = stride_of(out, 1);
  void* ws = status_word(a[11], dev);
  if (Tq > 0 && H > 0)
    call("dkv_latent_prompt_attn", dev,
         [&](void* stream) { return dkv_latent_prompt_attn(&p, ws, stream); });
  return is_none(a[10]) ? THPVariable_Wrap(out) : incref(a[10]);
}

// ------------------------------------------------------------------------- pages
// Caches whose block table and pools a call changes.
struct Pages {
  dkv_pages p{};
  const at::Tensor* table = nullptr;
  int device = -1;
};

void add_pool(Pages* g, const at::Tensor& t) {
  dkv_pages& p = g->p;
  if (p.num_pools == DKV_MAX_POOLS) value_error("too many caches");
  if (p.num_pools == 0) p.num_blocks = int32_size(t.size(0));
  if (t.size(0) != p.num_blocks) value_error("the caches' pools have different numbers of blocks");
  int64_t run = 1;  // the elements of a block follow one another
  for (int64_t i = t.dim() - 1; i > 0; --i) {
    if (t.stride(i) != run && t.size(i) != 1) value_error("a pool's blocks must be contiguous");
    run *= t.size(i);
  }
  const int64_t size = t.element_size();
  const int64_t stride = t.size(0) > 1 ? t.stride(0) : run;
  p.pools[p.num_pools++] = {t.data_ptr(), stride * size, run * size};
}

Pages parse_pages(PyObject* o, const char* where) {
  Pages g;
  if ((!PyTuple_Check(o) && !PyList_Check(o)) || is(o, g_paged) || is(o, g_fp8_paged) ||
      is(o, g_latent) || PySequence_Fast_GET_SIZE(o) < 1)
    value_error("caches must be a list of paged caches");
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(o); ++i) {
    PyObject* c = PySequence_Fast_GET_ITEM(o, i);
    const bool latent = is(c, g_latent), eight = is(c, g_fp8_paged);
    const at::Tensor* table;
    int device;
    int32_t block = kPage;
    if (latent) {
      const Latent l = parse_latent(c);
      block = l.c.block_size;
      device = l.device;
    } else if (eight || is(c, g_paged)) {
      device = parse_cache(c).device;
    } else {
      raise(PyExc_TypeError, "caches must be PagedCache, Fp8PagedCache or LatentCache objects");
    }
    if (device < 0) {
      PyErr_Format(PyExc_ValueError, "%s wants CUDA tensors", where);
      throw PyError{};
    }
    table = &tensor(PyTuple_GET_ITEM(c, eight ? 2 : 1), "block_table");
    if (i == 0) {
      g.table = table;
      g.device = device;
      g.p.block_size = block;
    } else if (table->data_ptr() != g.table->data_ptr() || table->sizes() != g.table->sizes() ||
               table->strides() != g.table->strides() || device != g.device ||
               block != g.p.block_size) {
      value_error("the caches must share one block table, block size and device");
    }
    add_pool(&g, tensor(PyTuple_GET_ITEM(c, 0), "pool"));
    if (eight) add_pool(&g, tensor(PyTuple_GET_ITEM(c, 1), "scale"));
  }
  g.p.rows = int32_size(g.table->size(0));
  g.p.cols = int32_size(g.table->size(1));
  g.p.block_table = static_cast<int32_t*>(g.table->data_ptr());
  g.p.table_stride = g.table->stride(0);
  return g;
}

int32_t* block_ints(PyObject* o, const char* name, const Pages& g) {
  return const_cast<int32_t*>(lengths(o, name, g.p.num_blocks, g.device));
}

at::Tensor pages_workspace(PyObject* o, const Pages& g, size_t* need) {
  *need = dkv_pages_workspace_bytes(g.p.rows, g.p.cols, g.p.num_blocks);
  if (*need == 0) *need = DKV_WORKSPACE_HEADER_BYTES;  // (the call refuses the sizes)
  const at::Tensor t = workspace_for(o, *need, *g.table);
  if (cuda_index(t) != g.device) value_error("workspace must be on the caches' device");
  return t;
}

// kv_pages_fork(caches, refs, seq_lens, parents, new_lens, workspace)
PyObject* kv_pages_fork(PyObject* const* a) {
  Pages g = parse_pages(a[0], "kv_pages_fork");
  if (is_none(a[1]) || is_none(a[2])) value_error("refs and seq_lens are needed");
  g.p.refs = block_ints(a[1], "refs", g);
  const int32_t* lens = lengths(a[2], "seq_lens", g.p.rows, g.device);
  const int32_t* parents = lengths(a[3], "parents", g.p.rows, g.device);
  const int32_t* news = lengths(a[4], "new_lens", g.p.rows, g.device);
  size_t need;
  const at::Tensor ws = pages_workspace(a[5], g, &need);
  call("dkv_kv_pages_fork", g.device, [&](void* stream) {
    return dkv_kv_pages_fork(&g.p, lens, parents, news, ws.data_ptr(), need, stream);
  });
  Py_RETURN_NONE;
}

// kv_pages_compact(caches, refs, refs_out, block_table_out, workspace)
PyObject* kv_pages_compact(PyObject* const* a) {
  Pages g = parse_pages(a[0], "kv_pages_compact");
  if (is_none(a[1])) value_error("refs are needed");
  g.p.refs = block_ints(a[1], "refs", g);
  int32_t* refs_out = is_none(a[2]) ? g.p.refs : block_ints(a[2], "refs_out", g);
  int32_t* table_out = g.p.block_table;
  int64_t stride = g.p.table_stride;
  if (!is_none(a[3])) {
    const at::Tensor& t = shaped(a[3], "block_table_out", g.table->sizes(), at::kInt, g.device);
    table_out = static_cast<int32_t*>(t.data_ptr());
    stride = t.stride(0);
  }
  const at::Tensor map = at::empty({g.p.num_blocks}, g.table->options());
  size_t need;
  const at::Tensor ws = pages_workspace(a[4], g, &need);
  call("dkv_kv_pages_compact", g.device, [&](void* stream) {
    return dkv_kv_pages_compact(&g.p, table_out, stride, refs_out,
                                static_cast<int32_t*>(map.data_ptr()), ws.data_ptr(), need, stream);
  });
  return THPVariable_Wrap(map);
}

// A call of N positional arguments; C++ exceptions become Python ones.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyError&) {
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<setup, 7>("setup"),
                           method<describe_cache, 1>("describe_cache"),
                           method<kv_meta_build, 3>("kv_meta_build"),
                           method<kv_meta_append, 6>("kv_meta_append"),
                           method<kv_append, 11>("kv_append"),
                           method<decode_attn_full, 9>("decode_attn_full"),
                           method<decode_attn_select, 16>("decode_attn_select"),
                           method<latent_append, 12>("latent_append"),
                           method<latent_decode_attn, 10>("latent_decode_attn"),
                           method<latent_prompt_attn, 13>("latent_prompt_attn"),
                           method<kv_pages_fork, 6>("kv_pages_fork"),
                           method<kv_pages_compact, 5>("kv_pages_compact"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
