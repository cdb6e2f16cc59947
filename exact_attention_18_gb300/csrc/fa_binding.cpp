// Native marshalling of the cache operators' tensor wrappers.
//
// A decoding step makes these calls once per layer on a few rows, where the
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
//               right, scale, out, lse, workspace)
PyObject* forward_paged(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    require(n == 15, "forward_paged: fifteen arguments");
    const Args a{argv, n};
    const Tensor &q = a.tensor(0, "q"), &kc = a.tensor(1, "k_cache"), &vc = a.tensor(2, "v_cache"),
                 &table = a.tensor(3, "block_table"), &lens = a.tensor(4, "kv_lens"), &cu = a.tensor(5, "cu_seqlens");
    const Tensor *o = a.maybe(12, "out"), *l = a.maybe(13, "lse"), *ws = a.maybe(14, "workspace");
    const OneDevice dev(q);
    for (const Tensor* x : {&kc, &vc, &table, &lens, &cu}) dev.also(*x);
    for (const Tensor* x : {o, l, ws}) dev.also(x);
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
    const float scale = argv[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                            : static_cast<float>(a.real(11));
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream().stream();
    const int64_t need = static_cast<int64_t>(fa_fwd_paged_workspace_size(batch, max_q, max_k, H, hk, D));
    const Tensor work = ws ? *ws : scratch(need, q, stream);
    const Tensor out = o ? *o : empty(q.sizes(), type, q), lse = l ? *l : empty({H, T}, at::kFloat, q);
    const void *q_at = q.const_data_ptr(), *cu_at = cu.const_data_ptr();
    void *o_at = out.mutable_data_ptr(), *l_at = lse.mutable_data_ptr(), *work_at = work.mutable_data_ptr();
    const size_t work_bytes = work.nbytes();
    fa_status st;
    {
      const Unlocked unlocked;
      std::unique_lock<std::mutex> turn(scratch_order(), std::defer_lock);  // (ends before the interpreter's is taken)
      if (!ws) turn.lock();
      st = fa_fwd_paged(q_at, o_at, static_cast<float*>(l_at), &cache, static_cast<const int32_t*>(cu_at), batch, max_q,
                        max_k, T, H, hk, D, causal, left, right, scale, code, work_at, work_bytes, stream);
    }
    return st == FA_OK ? pair(out, lse) : PyLong_FromLong(st);
  });
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_append)), METH_FASTCALL, nullptr},
    {"forward_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(forward_paged)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&module); }
