// Native marshalling of the tensor wrappers of the cache operators and of attention
// with modified scores.
//
// A decoding step makes the former calls once per layer on a few rows, where the
// kernels take 3 to 10 us; checking tensors and building arguments in Python
// took 20 to 30.  Here the same checks read the tensors directly, outputs come
// from the framework's allocator, and the library is called through its C ABI
// (fa.h).  Nothing is computed.
//
// Each function returns its outputs, or an int fa_status that the Python side
// raises; a bad tensor raises ValueError or TypeError here.  All of them run on
// the current stream of the current device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "../../include/fa.h"

namespace {

using at::Tensor;

struct BadValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct BadType : std::runtime_error {
  using std::runtime_error::runtime_error;
};

void require(bool ok, const char* what) {
  if (!ok) throw BadValue(what);
}

// Arguments of one call.
struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  const Tensor& tensor(int i, const char* name) const {
    if (!THPVariable_Check(v[i])) throw BadType(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(v[i]);
  }
  // nullptr for None
  const Tensor* maybe(int i, const char* name) const { return v[i] == Py_None ? nullptr : &tensor(i, name); }
  int64_t integer(int i) const {
    const long long x = PyLong_AsLongLong(v[i]);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
  }
  double real(int i) const {
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
  }
  bool flag(int i) const {
    const int x = PyObject_IsTrue(v[i]);
    if (x < 0) throw python_error();
    return x != 0;
  }
};

fa_dtype dtype_code(const Tensor& x) {
  if (x.scalar_type() == at::kHalf) return FA_FP16;
  if (x.scalar_type() == at::kBFloat16) return FA_BF16;
  throw BadType("unsupported dtype; use float16 or bfloat16");
}

// All tensors on one device, the current one (kernels launch there).
struct OneDevice {
  int device;
  explicit OneDevice(const Tensor& x) : device(x.get_device()) {
    require(device >= 0, "the tensors must be on a CUDA device");
    require(device == c10::cuda::current_device(), "the tensors are not on the current CUDA device");
  }
  void also(const Tensor& x) const { require(x.get_device() == device, "all tensors must be on one CUDA device"); }
  void also(const Tensor* x) const {
    if (x) also(*x);
  }
};

// Token stride of [T, heads, D] rows with dense heads.
int64_t rows(const Tensor& x, at::IntArrayRef shape, at::ScalarType type, const char* name) {
  if (x.scalar_type() != type || x.sizes() != shape ||
      (x.stride(2) != 1 && shape[2] > 1) || (x.stride(1) != shape[2] && shape[1] > 1))
    throw BadValue(std::string(name) +
                   " must have the other rows' dtype and shape, with dense heads (any stride between tokens)");
  return shape[0] > 1 ? x.stride(0) : shape[1] * shape[2];
}

const void* ints(const Tensor& x, at::ScalarType type, int64_t n, const char* name) {
  if (x.scalar_type() != type || x.dim() != 1 || x.size(0) != n || !x.is_contiguous())
    throw BadValue(std::string(name) + " must be a contiguous 1-D " + (type == at::kInt ? "int32" : "int64") +
                   " tensor of " + std::to_string(n) + " entries");
  return x.const_data_ptr();
}

const void* floats(const Tensor& x, int64_t n, const char* name) {
  if (x.scalar_type() != at::kFloat || x.dim() != 1 || x.size(0) != n || !x.is_contiguous())
    throw BadValue(std::string(name) + " must be a contiguous 1-D float32 tensor of " + std::to_string(n) + " entries");
  return x.const_data_ptr();
}

int64_t offsets(const Tensor& cu) {
  require(cu.scalar_type() == at::kInt && cu.dim() == 1 && cu.size(0) >= 1 && cu.is_contiguous(),
          "cu_seqlens must be a contiguous 1-D int32 tensor [batch + 1]");
  return cu.size(0) - 1;
}

fa_paged_cache paged_cache(const Tensor& k, const Tensor& v, const Tensor& table, const Tensor& kv_lens, int64_t batch,
                           int64_t heads, int64_t D, at::ScalarType type) {
  require(k.dim() == 4 && k.size(2) == heads && k.size(3) == D && k.scalar_type() == type && v.scalar_type() == type &&
              v.sizes() == k.sizes() && v.strides() == k.strides() && (k.stride(3) == 1 || D <= 1),
          "k_cache and v_cache must be [pages, page_size, H_kv, D] of the rows' heads, head dimension and dtype, with "
          "the same strides and the last dimension dense");
  require(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == batch && (batch == 0 || table.size(1) >= 1) &&
              (table.stride(1) == 1 || table.size(1) <= 1) && (batch <= 1 || table.stride(0) >= table.size(1)),
          "block_table must be an int32 tensor [batch, pages per sequence] with dense rows");
  fa_paged_cache c;
  c.k = k.mutable_data_ptr();
  c.v = v.mutable_data_ptr();
  c.block_table = static_cast<const int32_t*>(table.const_data_ptr());
  c.kv_lens = static_cast<const int32_t*>(ints(kv_lens, at::kInt, batch, "kv_lens"));
  c.table_stride = batch > 1 ? table.stride(0) : table.size(1);
  c.table_pages = table.size(1);
  c.num_pages = k.size(0);
  c.page_size = k.size(1);
  // The stride of a dimension of one entry is never used; it may be any number in torch.
  c.page_stride = c.num_pages > 1 ? k.stride(0) : D;
  c.row_stride = c.page_size > 1 ? k.stride(1) : D;
  c.head_stride = heads > 1 ? k.stride(2) : D;
  return c;
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
}

// Scratch of forward_paged, one per device and stream: calls on a stream run
// one after another, so they can share it.  A call that is being captured gets
// its own (the graph may run beside this stream's later calls).  Kept for the
// life of the process, and never destroyed, so that no tensor outlives the
// CUDA context's end.
Tensor scratch(int64_t bytes, const Tensor& like, cudaStream_t stream) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return empty({std::max<int64_t>(bytes, 256)}, at::kByte, like);
  static auto* kept = new std::map<std::pair<int, cudaStream_t>, Tensor>;  // (under the interpreter's lock)
  Tensor& t = (*kept)[{like.get_device(), stream}];
  if (!t.defined() || t.numel() < bytes) t = empty({std::max<int64_t>(bytes, 1 << 20)}, at::kByte, like);
  return t;
}

// Held while a call that uses kept scratch issues its launches: between two
// threads that share a stream, one call's launches must not fall between the
// other's.  Taken without the interpreter's lock.
std::mutex& scratch_order() {
  static auto* m = new std::mutex;
  return *m;
}

// The interpreter's lock, given up for the scope's life.  Inside it nothing of a
// tensor is asked for: its pointers can throw (no storage behind it) or allocate
// (a lazy copy), so they are read before.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Calls f() and turns its exceptions into Python's.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const BadType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
  PyObject* t = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// rope(back, q, k, positions, steps, interleaved, magnitude, q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 9, "rope: nine arguments");
    const Args a{argv, n};
    const Tensor &q = a.tensor(1, "q"), &k = a.tensor(2, "k"), &pos = a.tensor(3, "positions"),
                 &steps = a.tensor(4, "steps");
    const Tensor *qo = a.maybe(7, "q_out"), *ko = a.maybe(8, "k_out");
    const OneDevice dev(q);
    dev.also(k);
    dev.also(pos);
    dev.also(steps);
    dev.also(qo);
    dev.also(ko);
    require(q.dim() == 3 && k.dim() == 3, "q and k must be [T, heads, D]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), hk = k.size(1);
    const auto type = q.scalar_type();
    require(k.size(0) == T && k.size(2) == D, "k must have q's tokens and head dimension");
    const int64_t qs = rows(q, q.sizes(), type, "q"), ks = rows(k, k.sizes(), type, "k");
    const void* p = ints(pos, at::kInt, T, "positions");
    const int64_t pairs = steps.numel();
    const void* s = ints(steps, at::kLong, pairs, "steps");
    const int64_t qos = qo ? rows(*qo, q.sizes(), type, "the q output") : H * D;
    const int64_t kos = ko ? rows(*ko, k.sizes(), type, "the k output") : hk * D;
    const fa_dtype code = dtype_code(q);
    const Tensor q_out = qo ? *qo : empty(q.sizes(), type, q), k_out = ko ? *ko : empty(k.sizes(), type, q);
    const bool back = a.flag(0), inter = a.flag(5);
    const float mag = static_cast<float>(a.real(6));
    void* stream = c10::cuda::getCurrentCUDAStream().stream();
    const void *q_at = q.const_data_ptr(), *k_at = k.const_data_ptr();
    void *qo_at = q_out.mutable_data_ptr(), *ko_at = k_out.mutable_data_ptr();
    fa_status st;
    {
      const Unlocked unlocked;
      st = (back ? fa_rope_bwd : fa_rope)(q_at, qs, k_at, ks, qo_at, qos, ko_at, kos, static_cast<const int32_t*>(p),
                                          static_cast<const uint64_t*>(s), T, H, hk, D, 2 * pairs, inter, mag, code,
                                          stream);
    }
    return st == FA_OK ? pair(q_out, k_out) : PyLong_FromLong(st);
  });
}

// paged_append(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_seqlen, q, positions, steps,
//              interleaved, magnitude, q_out)
PyObject* paged_append(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 14, "paged_append: fourteen arguments");
    const Args a{argv, n};
    const Tensor &k = a.tensor(0, "k"), &v = a.tensor(1, "v"), &kc = a.tensor(2, "k_cache"),
                 &vc = a.tensor(3, "v_cache"), &table = a.tensor(4, "block_table"), &lens = a.tensor(5, "kv_lens"),
                 &cu = a.tensor(6, "cu_seqlens");
    const Tensor *q = a.maybe(8, "q"), *pos = a.maybe(9, "positions"), *steps = a.maybe(10, "steps"),
                 *qo = a.maybe(13, "q_out");
    const OneDevice dev(k);
    for (const Tensor* x : {&v, &kc, &vc, &table, &lens, &cu}) dev.also(*x);
    for (const Tensor* x : {q, pos, steps, qo}) dev.also(x);
    require(k.dim() == 3, "k must be [T, H_kv, D]");
    const int64_t T = k.size(0), hk = k.size(1), D = k.size(2);
    const auto type = k.scalar_type();
    const int64_t batch = offsets(cu);
    const fa_paged_cache cache = paged_cache(kc, vc, table, lens, batch, hk, D, type);
    const int64_t ks = rows(k, k.sizes(), type, "k"), vs = rows(v, k.sizes(), type, "v");
    const int64_t pairs = steps ? steps->numel() : 0;
    const void* s = steps ? ints(*steps, at::kLong, pairs, "steps") : nullptr;
    const void* p = pos ? ints(*pos, at::kInt, T, "positions") : nullptr;
    const fa_dtype code = dtype_code(k);
    int64_t H = 0, qs = 0, qos = 0;
    Tensor q_out;
    if (q) {
      require(q->dim() == 3 && q->size(0) == T && q->size(2) == D, "q must be [T, H, D] of k's tokens and head dimension");
      H = q->size(1);
      qs = rows(*q, q->sizes(), type, "q");
      qos = qo ? rows(*qo, q->sizes(), type, "q_out") : H * D;
      q_out = qo ? *qo : empty(q->sizes(), type, k);
    }
    const int64_t max_len = a.integer(7);
    const bool inter = a.flag(11);
    const float mag = static_cast<float>(a.real(12));
    void* stream = c10::cuda::getCurrentCUDAStream().stream();
    const void *q_at = q ? q->const_data_ptr() : nullptr, *k_at = k.const_data_ptr(), *v_at = v.const_data_ptr(),
               *cu_at = cu.const_data_ptr();
    void* qo_at = q ? q_out.mutable_data_ptr() : nullptr;
    fa_status st;
    {
      const Unlocked unlocked;
      st = fa_paged_append(q_at, qs, qo_at, qos, k_at, ks, v_at, vs, &cache, static_cast<const int32_t*>(cu_at),
                           static_cast<const int32_t*>(p), static_cast<const uint64_t*>(s), batch, max_len, T, H, hk, D,
                           2 * pairs, inter, mag, code, stream);
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    if (q) return THPVariable_Wrap(q_out);
    Py_RETURN_NONE;
  });
}

// forward_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_seqlen_q, max_seqlen_k, causal, left,
//               right, scale, out, lse, workspace, softcap, slopes, tree, positions)
PyObject* forward_paged(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 19, "forward_paged: nineteen arguments");
    const Args a{argv, n};
    const Tensor &q = a.tensor(0, "q"), &kc = a.tensor(1, "k_cache"), &vc = a.tensor(2, "v_cache"),
                 &table = a.tensor(3, "block_table"), &lens = a.tensor(4, "kv_lens"), &cu = a.tensor(5, "cu_seqlens");
    const Tensor *o = a.maybe(12, "out"), *l = a.maybe(13, "lse"), *ws = a.maybe(14, "workspace"),
                 *slopes = a.maybe(16, "slopes"), *tree = a.maybe(17, "tree"), *pos = a.maybe(18, "positions");
    const OneDevice dev(q);
    for (const Tensor* x : {&kc, &vc, &table, &lens, &cu}) dev.also(*x);
    for (const Tensor* x : {o, l, ws, slopes, tree, pos}) dev.also(x);
    require(q.dim() == 3 && q.is_contiguous(), "q must be a contiguous tensor [T, H, D]");
    require(kc.dim() == 4, "k_cache must be [pages, page_size, H_kv, D]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), hk = kc.size(2);
    require(hk >= 1 && H % hk == 0, "q's heads must be a multiple of the cache's");
    const auto type = q.scalar_type();
    const int64_t batch = offsets(cu);
    const fa_paged_cache cache = paged_cache(kc, vc, table, lens, batch, hk, D, type);
    const fa_dtype code = dtype_code(q);
    require(!o || (o->sizes() == q.sizes() && o->scalar_type() == type && o->is_contiguous()), "out must be like q");
    require(!l || (l->dim() == 2 && l->size(0) == H && l->size(1) == T && l->scalar_type() == at::kFloat &&
                   l->is_contiguous()),
            "lse must be contiguous fp32 [H, T]");
    require(!ws || ws->is_contiguous(), "workspace must be contiguous");
    const int64_t max_q = a.integer(6), max_k = a.integer(7), left = a.integer(9), right = a.integer(10);
    const bool causal = a.flag(8);
    fa_scores scores = {};
    if (argv[15] != Py_None) {
      scores.softcap = static_cast<float>(a.real(15));
      require(scores.softcap > 0, "softcap must be positive (None: no cap)");
    }
    if (slopes) scores.slopes = static_cast<const float*>(floats(*slopes, H, "slopes"));
    const bool modified = scores.softcap > 0 || slopes;
    require(!tree == !pos, "tree and positions belong together");
    int64_t words = 0, row_stride = 0;
    if (tree) {
      require(causal, "a tree's rows say what its tokens see: causal stays true");
      require(right <= 0, "a tree has the window's left side alone");
      require(tree->scalar_type() == at::kInt && tree->dim() == 2 && tree->size(0) == T &&
                  (tree->stride(1) == 1 || tree->size(1) <= 1) && (T <= 1 || tree->stride(0) >= tree->size(1)),
              "tree must be an int32 tensor [T, words] with dense rows");
      words = tree->size(1);
      row_stride = T > 1 ? tree->stride(0) : words;
      ints(*pos, at::kInt, T, "positions");
    }
    const float scale = argv[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                            : static_cast<float>(a.real(11));
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream().stream();
    const int64_t need = static_cast<int64_t>(fa_fwd_paged_workspace_size(batch, max_q, max_k, H, hk, D));
    const Tensor work = ws ? *ws : scratch(need, q, stream);
    const Tensor out = o ? *o : empty(q.sizes(), type, q), lse = l ? *l : empty({H, T}, at::kFloat, q);
    const void *q_at = q.const_data_ptr(), *cu_at = cu.const_data_ptr();
    void *o_at = out.mutable_data_ptr(), *l_at = lse.mutable_data_ptr(), *work_at = work.mutable_data_ptr();
    const void *tree_at = tree ? tree->const_data_ptr() : nullptr, *pos_at = tree ? pos->const_data_ptr() : nullptr;
    const size_t work_bytes = work.nbytes();
    fa_status st;
    {
      const Unlocked unlocked;
      std::unique_lock<std::mutex> turn(scratch_order(), std::defer_lock);  // (ends before the interpreter's is taken)
      if (!ws) turn.lock();
      const auto* offs = static_cast<const int32_t*>(cu_at);
      float* l_out = static_cast<float*>(l_at);
      if (tree)
        st = fa_fwd_paged_tree(q_at, o_at, l_out, &cache, offs, static_cast<const int32_t*>(pos_at),
                               static_cast<const uint32_t*>(tree_at), row_stride, words, batch, max_q, max_k, T, H, hk,
                               D, left, &scores, scale, code, work_at, work_bytes, stream);
      else if (modified)
        st = fa_fwd_paged_scores(q_at, o_at, l_out, &cache, offs, batch, max_q, max_k, T, H, hk, D, causal, left, right,
                                 &scores, scale, code, work_at, work_bytes, stream);
      else
        st = fa_fwd_paged(q_at, o_at, l_out, &cache, offs, batch, max_q, max_k, T, H, hk, D, causal, left, right, scale,
                          code, work_at, work_bytes, stream);
    }
    return st == FA_OK ? pair(out, lse) : PyLong_FromLong(st);
  });
}

// Whole sequences with modified scores: [B, heads, S, D] (or [B, S, D], one head), or
// packed [T, heads, D] with offsets.
struct Whole {
  bool packed, squeezed;
  int64_t B, H, hk, S, D, T;  // packed: B sequences of up to S of the T tokens
  at::ScalarType type;
  fa_dtype code;
  const int32_t* cu = nullptr;
  std::vector<int64_t> q_shape, kv_shape, lse_shape;
  Whole(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor* offs, int64_t max_seqlen, const OneDevice& dev)
      : packed(offs != nullptr), type(q.scalar_type()), code(dtype_code(q)) {
    squeezed = !packed && q.dim() == 3;
    const int64_t dims = packed || squeezed ? 3 : 4;
    require(q.dim() == dims && k.dim() == dims,
            packed ? "q and k must be [T, heads, D]" : "q and k must be [B, heads, S, D] (or both [B, S, D])");
    if (packed) {
      T = q.size(0), H = q.size(1), D = q.size(2), hk = k.size(1);
      B = offsets(*offs);
      S = max_seqlen;
      dev.also(*offs);
      cu = static_cast<const int32_t*>(offs->const_data_ptr());
      q_shape = {T, H, D}, kv_shape = {T, hk, D}, lse_shape = {H, T};
    } else if (squeezed) {
      B = q.size(0), S = q.size(1), D = q.size(2), H = hk = 1, T = 0;
      q_shape = kv_shape = {B, S, D}, lse_shape = {B, S};
    } else {
      B = q.size(0), H = q.size(1), S = q.size(2), D = q.size(3), hk = k.size(1), T = 0;
      q_shape = {B, H, S, D}, kv_shape = {B, hk, S, D}, lse_shape = {B, H, S};
    }
    require((hk >= 1 && H % hk == 0) || (H == 0 && hk == 0), "q's heads must be a multiple of k's and v's");
    like(q, q_shape, type, "q", dev);
    like(k, kv_shape, type, "k", dev);
    like(v, kv_shape, type, "v", dev);
  }
  static void like(const Tensor& x, at::IntArrayRef shape, at::ScalarType t, const char* name, const OneDevice& dev) {
    dev.also(x);
    if (x.sizes() != shape || x.scalar_type() != t || !x.is_contiguous())
      throw BadValue(std::string(name) + " must be a contiguous tensor of the call's shape and dtype");
  }
  static Tensor given(const Tensor* x, at::IntArrayRef shape, at::ScalarType t, const char* name, const Tensor& q,
                      const OneDevice& dev) {
    if (!x) return empty(shape, t, q);
    like(*x, shape, t, name, dev);
    return *x;
  }
  fa_scores scores(const Args& a, int at, const OneDevice& dev) const {  // softcap, slopes, prefix
    fa_scores s = {};
    if (a.v[at] != Py_None) {
      s.softcap = static_cast<float>(a.real(at));
      require(s.softcap > 0, "softcap must be positive (None: no cap)");
    }
    const Tensor *slopes = a.maybe(at + 1, "slopes"), *prefix = a.maybe(at + 2, "prefix");
    dev.also(slopes);
    dev.also(prefix);
    if (slopes) s.slopes = static_cast<const float*>(floats(*slopes, H, "slopes"));
    if (prefix) s.prefix = static_cast<const int32_t*>(ints(*prefix, at::kInt, B, "prefix"));
    return s;
  }
  float scale(const Args& a, int at) const {
    return a.v[at] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                              : static_cast<float>(a.real(at));
  }
};

// attend(q, k, v, cu_seqlens, max_seqlen, causal, left, right, softcap, slopes, prefix, scale, out, lse)
PyObject* attend(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 14, "attend: fourteen arguments");
    const Args a{argv, n};
    const Tensor &q = a.tensor(0, "q"), &k = a.tensor(1, "k"), &v = a.tensor(2, "v");
    const OneDevice dev(q);
    const Tensor* cu = a.maybe(3, "cu_seqlens");
    const Whole w(q, k, v, cu, cu ? a.integer(4) : 0, dev);
    const bool causal = a.flag(5);
    const int64_t left = a.integer(6), right = a.integer(7);
    const fa_scores scores = w.scores(a, 8, dev);
    const float scale = w.scale(a, 11);
    const Tensor out = Whole::given(a.maybe(12, "out"), w.q_shape, w.type, "out", q, dev);
    const Tensor lse = Whole::given(a.maybe(13, "lse"), w.lse_shape, at::kFloat, "lse", q, dev);
    void* stream = c10::cuda::getCurrentCUDAStream().stream();
    const void *q_at = q.const_data_ptr(), *k_at = k.const_data_ptr(), *v_at = v.const_data_ptr();
    void* o_at = out.mutable_data_ptr();
    float* l_at = static_cast<float*>(lse.mutable_data_ptr());
    fa_status st;
    {
      const Unlocked unlocked;
      st = w.packed ? fa_fwd_scores_varlen(q_at, k_at, v_at, o_at, l_at, w.cu, w.B, w.S, w.T, w.H, w.hk, w.D, causal,
                                           left, right, &scores, scale, w.code, stream)
                    : fa_fwd_scores(q_at, k_at, v_at, o_at, l_at, w.B, w.H, w.hk, w.S, w.D, causal, left, right,
                                    &scores, scale, w.code, stream);
    }
    return st == FA_OK ? pair(out, lse) : PyLong_FromLong(st);
  });
}

// attend_backward(q, k, v, o, do, lse, cu_seqlens, max_seqlen, causal, left, right, softcap, slopes, prefix, scale,
//                 dq, dk, dv, workspace)
PyObject* attend_backward(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 19, "attend_backward: nineteen arguments");
    const Args a{argv, n};
    const Tensor &q = a.tensor(0, "q"), &k = a.tensor(1, "k"), &v = a.tensor(2, "v"), &o = a.tensor(3, "o"),
                 &dout = a.tensor(4, "do"), &lse = a.tensor(5, "lse");
    const OneDevice dev(q);
    const Tensor* cu = a.maybe(6, "cu_seqlens");
    const Whole w(q, k, v, cu, cu ? a.integer(7) : 0, dev);
    Whole::like(o, w.q_shape, w.type, "o", dev);
    Whole::like(dout, w.q_shape, w.type, "do", dev);
    Whole::like(lse, w.lse_shape, at::kFloat, "lse", dev);
    const bool causal = a.flag(8);
    const int64_t left = a.integer(9), right = a.integer(10);
    const fa_scores scores = w.scores(a, 11, dev);
    const float scale = w.scale(a, 14);
    const Tensor dq = Whole::given(a.maybe(15, "dq"), w.q_shape, w.type, "dq", q, dev);
    const Tensor dk = Whole::given(a.maybe(16, "dk"), w.kv_shape, w.type, "dk", q, dev);
    const Tensor dv = Whole::given(a.maybe(17, "dv"), w.kv_shape, w.type, "dv", q, dev);
    const Tensor* ws = a.maybe(18, "workspace");
    dev.also(ws);
    require(!ws || ws->is_contiguous(), "workspace must be contiguous");
    const size_t need = w.packed ? fa_bwd_varlen_workspace_size(w.B, w.S, w.T, w.H, w.hk, w.D)
                                 : fa_bwd_gqa_workspace_size(w.B, w.H, w.hk, w.S, w.D);
    const Tensor work = ws ? *ws : empty({std::max<int64_t>(static_cast<int64_t>(need), 256)}, at::kByte, q);
    void* stream = c10::cuda::getCurrentCUDAStream().stream();
    const void *q_at = q.const_data_ptr(), *k_at = k.const_data_ptr(), *v_at = v.const_data_ptr(),
               *o_at = o.const_data_ptr(), *do_at = dout.const_data_ptr();
    const float* l_at = static_cast<const float*>(lse.const_data_ptr());
    void *dq_at = dq.mutable_data_ptr(), *dk_at = dk.mutable_data_ptr(), *dv_at = dv.mutable_data_ptr(),
         *work_at = work.mutable_data_ptr();
    const size_t work_bytes = work.nbytes();
    fa_status st;
    {
      const Unlocked unlocked;
      st = w.packed ? fa_bwd_scores_varlen(q_at, k_at, v_at, o_at, do_at, l_at, dq_at, dk_at, dv_at, w.cu, w.B, w.S,
                                           w.T, w.H, w.hk, w.D, causal, left, right, &scores, scale, w.code, work_at,
                                           work_bytes, stream)
                    : fa_bwd_scores(q_at, k_at, v_at, o_at, do_at, l_at, dq_at, dk_at, dv_at, w.B, w.H, w.hk, w.S, w.D,
                                    causal, left, right, &scores, scale, w.code, work_at, work_bytes, stream);
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject *x = THPVariable_Wrap(dq), *y = x ? THPVariable_Wrap(dk) : nullptr, *z = y ? THPVariable_Wrap(dv) : nullptr;
    PyObject* t = z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return t;
  });
}

// paged_keep(k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_seqlen, path, path_lens)
PyObject* paged_keep(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 8, "paged_keep: eight arguments");
    const Args a{argv, n};
    const Tensor &kc = a.tensor(0, "k_cache"), &vc = a.tensor(1, "v_cache"), &table = a.tensor(2, "block_table"),
                 &lens = a.tensor(3, "kv_lens"), &cu = a.tensor(4, "cu_seqlens"), &path = a.tensor(6, "path"),
                 &path_lens = a.tensor(7, "path_lens");
    const OneDevice dev(kc);
    for (const Tensor* x : {&vc, &table, &lens, &cu, &path, &path_lens}) dev.also(*x);
    require(kc.dim() == 4, "k_cache must be [pages, page_size, H_kv, D]");
    const int64_t hk = kc.size(2), D = kc.size(3), batch = offsets(cu);
    const fa_dtype code = dtype_code(kc);
    const fa_paged_cache cache = paged_cache(kc, vc, table, lens, batch, hk, D, kc.scalar_type());
    require(path.scalar_type() == at::kInt && path.dim() == 2 && path.size(0) == batch &&
                (path.stride(1) == 1 || path.size(1) <= 1) && (batch <= 1 || path.stride(0) >= path.size(1)),
            "path must be an int32 tensor [batch, tokens] with dense rows");
    const int64_t cols = path.size(1), stride = batch > 1 ? path.stride(0) : cols;
    const void *path_at = path.const_data_ptr(), *cu_at = cu.const_data_ptr(),
               *lens_at = ints(path_lens, at::kInt, batch, "path_lens");
    const int64_t max_len = a.integer(5);
    void* stream = c10::cuda::getCurrentCUDAStream().stream();
    fa_status st;
    {
      const Unlocked unlocked;
      st = fa_paged_keep(&cache, static_cast<const int32_t*>(cu_at), static_cast<const int32_t*>(path_at), stride, cols,
                         static_cast<const int32_t*>(lens_at), batch, max_len, hk, D, code, stream);
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_append)), METH_FASTCALL, nullptr},
    {"forward_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(forward_paged)), METH_FASTCALL,
     nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"attend_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend_backward)), METH_FASTCALL,
     nullptr},
    {"paged_keep", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_keep)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&module); }
