// C-ABI entry points: argument validation, tensor-map encoding and launches.
// Nothing here computes attention; every arithmetic step runs in the kernels.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <atomic>
#include <cstring>
#include <mutex>

#include "../../include/fa.h"
#include "fa_internal.cuh"
#include "fa_paged.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// One error word per device; kernels receive its address.
static __device__ int g_fa_device_error = 0;

int* device_error_word() {
  static int* addr[64] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* a = nullptr;
    if (cudaGetSymbolAddress(&a, g_fa_device_error) != cudaSuccess) return nullptr;
    addr[dev] = static_cast<int*>(a);
  }
  return addr[dev];
}

// Limit of each pipeline wait in the kernels launched from now on.
static std::atomic<unsigned long long> g_wait_limit_ns{ptx::kWaitLimitNs};

unsigned long long wait_limit_ns() { return g_wait_limit_ns.load(std::memory_order_relaxed); }

}  // namespace fa

// ---------------------------------------------------------------------------
// Scratch for fa_bwd_noalloc.  Some callers cannot allocate device memory at
// the point where they need the backward pass (a custom allocator that must
// not be re-entered, a memory pool that is already fully carved up, code
// running under a framework that forbids cudaMalloc on its hot path).  For
// them the backward's one scratch buffer, the fp32 row vector D, lives in this
// fixed array instead of a caller workspace.  Every GPU that loads the library
// holds it (8 MiB) until the process exits.
namespace fa {
constexpr int64_t kNoAllocMaxRows = int64_t(1) << 21;  // B*H*S rows: 2 Mi floats = 8 MiB
static __device__ __align__(256) float g_noalloc_delta[kNoAllocMaxRows];

// Device address of g_noalloc_delta on the current device.  In host code the
// array's name only stands for the symbol, so the address is looked up once
// per device (with that device current) and cached.
float* noalloc_delta_address(cudaError_t* err) {
  static float* addr[64] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= 64) {
    *err = cudaErrorInvalidDevice;
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* a = nullptr;
    *err = cudaGetSymbolAddress(&a, g_noalloc_delta);
    if (*err != cudaSuccess) return nullptr;
    addr[dev] = static_cast<float*>(a);
  }
  return addr[dev];
}
}  // namespace fa

namespace {

thread_local char g_detail[256] = "";

fa_status fail(fa_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fa_status fail(fa_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_detail, sizeof(g_detail), fmt, ap);
  va_end(ap);
  return s;
}

// cuTensorMapEncodeTiled, fetched from the driver through the runtime so the
// library does not link against libcuda directly.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// [BH, S, D] 16-bit tensor as a 3-D map {D, S, BH}; box {row_bytes/2, box_rows, 1}.
// Rows past S read as zero.
fa_status encode_qkv_map(CUtensorMap* map, const void* base, bool bf16, int64_t D, int64_t S, int64_t BH,
                         const char* name, unsigned box_rows = 128) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int rb = fa::row_bytes_for(static_cast<int>(D));
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D * 2), static_cast<cuuint64_t>(S * D * 2)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(rb / 2), static_cast<cuuint32_t>(box_rows), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUtensorMapSwizzle swz = rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : (rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "tensor map for %s: cuTensorMapEncodeTiled error %d", name, (int)r);
  return FA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fa_status check_common(int64_t B, int64_t H, int64_t S, int64_t D, float scale, fa_dtype dtype) {
  if (B < 0 || H < 0 || S < 0) return fail(FA_ERR_INVALID_ARG, "negative size: B=%lld H=%lld S=%lld",
                                           (long long)B, (long long)H, (long long)S);
  if (dtype != FA_FP16 && dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (!std::isfinite(scale)) return fail(FA_ERR_INVALID_ARG, "scale must be finite");
  if (D != 16 && D != 32 && D != 64 && D != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dimension D=%lld is not one of 16, 32, 64, 128", (long long)D);
  if (B > 0 && H > (int64_t(1) << 31) / B) return fail(FA_ERR_UNSUPPORTED, "B*H must be below 2^31");
  if (S >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "S must be below 2^31");
  if ((S + 127) / 128 > 65535) return fail(FA_ERR_UNSUPPORTED, "S=%lld exceeds 65535 tiles of 128", (long long)S);
  // element count must fit comfortably in 64-bit byte offsets
  if (B * H > 0 && S * D > (int64_t(1) << 60) / (B * H)) return fail(FA_ERR_UNSUPPORTED, "tensor too large");
  return FA_OK;
}

fa_status check_ptr(const void* p, const char* name) {
  if (!p) return fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(FA_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  return FA_OK;
}

fa_status from_cuda(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FA_OK;
  return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr float kLog2e = 1.4426950408889634f;

// Grouped heads: H_kv K/V heads, each shared by H / H_kv consecutive query
// heads.  H_kv = H is ordinary multi-head attention.
fa_status check_heads(int64_t H, int64_t H_kv) {
  if (H_kv < 0 || H_kv > H) return fail(FA_ERR_INVALID_ARG, "H_kv=%lld must lie in [0, H=%lld]",
                                        (long long)H_kv, (long long)H);
  if (H > 0 && (H_kv == 0 || H % H_kv != 0))
    return fail(FA_ERR_INVALID_ARG, "H=%lld is not a multiple of H_kv=%lld", (long long)H, (long long)H_kv);
  if (H == 0 && H_kv != 0) return fail(FA_ERR_INVALID_ARG, "H_kv=%lld with H=0", (long long)H_kv);
  return FA_OK;
}

// One call's problem.  Fixed length: B entries of S rows, tensors [B, H(_kv), S, D].
// Packed batch (cu != nullptr): B samples over T = total tokens, tensors
// [T, H(_kv), D], S = the largest sample length; L is [H, T].
struct Shape {
  int64_t B, H, H_kv, S, D;
  const int32_t* cu;
  int64_t total;
  bool is_packed;
  int64_t win_left = -1, win_right = -1;  // window band; negative = unlimited
  bool packed() const { return is_packed; }
  // Kernel window sides (fa::kNoWindow = unlimited; causal fixes the right side at 0).
  int kernel_left() const { return win_left < 0 || win_left >= S ? fa::kNoWindow : static_cast<int>(win_left); }
  int kernel_right(bool causal) const {
    if (causal) return 0;
    return win_right < 0 || win_right >= S ? fa::kNoWindow : static_cast<int>(win_right);
  }
  // The general kernels serve packed batches and windows that cut the band;
  // fixed-length full/causal calls take the specialised ones.
  bool general(bool causal) const {
    return is_packed || kernel_left() != fa::kNoWindow || (!causal && kernel_right(false) != fa::kNoWindow);
  }
  int64_t q_rows() const { return packed() ? total * H : B * H * S; }      // rows of Q, O, dO, L, Delta
  int64_t kv_rows() const { return packed() ? total * H_kv : B * H_kv * S; }  // rows of K, V, dK, dV
  bool empty() const { return B * H == 0 || S == 0 || (packed() && total == 0); }
};

fa_status check_shape(const Shape& sh, float scale, fa_dtype dtype) {
  fa_status st = check_common(sh.B, sh.H, sh.S, sh.D, scale, dtype);
  if (st != FA_OK) return st;
  if ((st = check_heads(sh.H, sh.H_kv))) return st;
  if (sh.packed()) {
    if (sh.total < 0) return fail(FA_ERR_INVALID_ARG, "negative total tokens %lld", (long long)sh.total);
    if (sh.total >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "total tokens must be below 2^31");
    if (sh.H > 0 && sh.total * sh.H >= (int64_t(1) << 31))
      return fail(FA_ERR_UNSUPPORTED, "total tokens * H must be below 2^31");
    if (sh.cu && (reinterpret_cast<uintptr_t>(sh.cu) & 3u) != 0)
      return fail(FA_ERR_ALIGNMENT, "cu_seqlens is not 4-byte aligned");
  }
  return FA_OK;
}

// The tensor map of one input for the call's layout: {D, S, B*heads} (fixed
// length; rows past S read zero) or {D, heads, T} (packed; tokens past T read
// zero), box {row_bytes/2, box_rows, 1} or {row_bytes/2, 1, box_rows}.
fa_status encode_input(CUtensorMap* map, const void* base, bool bf16, const Shape& sh, int64_t heads,
                       const char* name, unsigned box_rows = 128) {
  if (!sh.packed()) return encode_qkv_map(map, base, bf16, sh.D, sh.S, sh.B * heads, name, box_rows);
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int rb = fa::row_bytes_for(static_cast<int>(sh.D));
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(sh.D), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(sh.total)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(sh.D * 2), static_cast<cuuint64_t>(heads * sh.D * 2)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(rb / 2), 1u, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUtensorMapSwizzle swz = rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : (rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "tensor map for %s: cuTensorMapEncodeTiled error %d", name, (int)r);
  return FA_OK;
}

// The constants of a cap.  tanh(v) / v on |v| <= 1.25 is a polynomial in v^2 (minimax
// of degree 6, by Remez exchange; relative error 6.2e-7); with v = scale x / cap it
// becomes tanh(v) = x * sum_k poly[k] x^(2k), off by 7.4e-7 to 8.4e-7 with fp32's
// roundings, as they fall for the scale / cap (1286 of them, 1e-8 to 1e7; 2^-20 is 9.5e-7).
// Coefficients that leave fp32's normal range bound the |x| it is used for: below it
// to where the terms left out are under 2^-22 of the value, above it to none.  (So a cap
// of 400 scales or more has its polynomial up to 0.49 of the cap: 50 at D = 64 and 128.)
// Range and degree were measured (us; scores of deviation 4 under 50 B2 H32/4 S4096
// D128, of 8 under 30 B7 H16/2 up to 2500 D64): degree 5 to 1.05 (error 9.5e-7) 335,
// 157, to 1.1 (1.5e-6) 336, 143; degree 6 to 1.25 349, 124.  A block that holds a score
// beyond takes the longer way.
void tanh_poly(float scale, float cap, fa::ScoreParams* p) {
  constexpr double kC[fa::kTanhTerms] = {0.999999376, -0.333293396, 0.132906482, -0.0522054417,
                                          0.0182291227, -0.00462690537, 0.00058449404};
  constexpr double kMax = 1.25;
  const double in = static_cast<double>(scale) / cap;
  p->cap = static_cast<float>(cap * 1.4426950408889634074);
  p->in2 = static_cast<float>(2 * 1.4426950408889634074 * in);
  double vmax = kMax, f = in;
  for (int k = 0; k < fa::kTanhTerms; ++k, f *= in * in) {
    p->poly[k] = static_cast<float>(kC[k] * f);
    const double size = std::fabs(kC[k] * f);
    if (size > 1e37) vmax = -1;  // no score is small, 0 neither: 0 * inf
    if (k > 0 && size < 1e-37) {
      p->poly[k] = 0.f;
      vmax = std::fmin(vmax, std::pow(2.4e-7 / (2 * std::fabs(kC[k])), 1.0 / (2 * k)));
    }
  }
  const double small = in == 0 ? 1e18 : std::fmin(vmax / std::fabs(in), 1e18);
  p->small = vmax < 0 ? -1.f : static_cast<float>(small);
}

// Modified scores of a call; *on: they need their own kernels.  (A packed call that
// may have them takes those whatever they are: they clear what lies behind a sample.)
fa_status check_scores(const fa_scores* in, float scale, bool prefix_ok, bool packed, bool* on,
                       fa::ScoreParams* out) {
  *on = false;
  *out = fa::ScoreParams{};
  const float scale_log2 = scale * kLog2e;
  const bool by_scale = scale_log2 >= 1e-4f;
  out->unit = by_scale ? scale_log2 : 1.f;
  out->pre = scale_log2;
  out->premul = by_scale ? 0 : 1;
  out->per_unit = 1.f / out->unit;
  if (!in) return FA_OK;
  if (!std::isfinite(in->softcap) || in->softcap < 0)
    return fail(FA_ERR_INVALID_ARG, "softcap must be finite and not negative (0: none)");
  if (in->prefix && !prefix_ok) return fail(FA_ERR_UNSUPPORTED, "a prefix is for whole sequences, not for a cache");
  if ((reinterpret_cast<uintptr_t>(in->slopes) & 3u) != 0) return fail(FA_ERR_ALIGNMENT, "slopes is not 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(in->prefix) & 3u) != 0) return fail(FA_ERR_ALIGNMENT, "prefix is not 4-byte aligned");
  if (in->softcap > 0) {
    // (beyond these the cap's own arithmetic leaves the range of fp32)
    if (in->softcap < 1e-10f || in->softcap > 1e10f || !std::isfinite(scale / in->softcap * 3.f))
      return fail(FA_ERR_UNSUPPORTED, "softcap must be between 1e-10 and 1e10, and scale / softcap finite");
    tanh_poly(scale, in->softcap, out);
    out->unit = out->cap;
    out->premul = 0;
    out->per_unit = 1.f / out->unit;
  }
  out->slopes = in->slopes;
  out->prefix = in->prefix;
  *on = packed || in->softcap > 0 || in->slopes || in->prefix;
  return FA_OK;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Split-KV: keys per shard (a multiple of 128) and shard count for a request of n splits.
void splitkv_layout(int64_t S, int64_t n, int* chunk, int* shards) {
  const int64_t per = (S + n - 1) / n;
  const int64_t c = ((per + 127) / 128) * 128;
  *chunk = static_cast<int>(c);
  *shards = static_cast<int>((S + c - 1) / c);
}

size_t splitkv_bytes(const Shape& sh, int shards) {
  return round256(static_cast<size_t>(shards) * static_cast<size_t>(sh.B * sh.H * sh.S) *
                  static_cast<size_t>(sh.D + 1) * sizeof(float));
}

// Forward; with split > 0 (general kernels, fixed layout) the keys are cut
// into shards whose fp32 partials go to `workspace`, then merged by L.
fa_status fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, const Shape& sh, int causal,
                   float scale, fa_dtype dtype, void* stream, int64_t split = 0, void* workspace = nullptr,
                   size_t workspace_bytes = 0, const fa_scores* scores = nullptr) {
  g_detail[0] = 0;
  fa_status st = check_shape(sh, scale, dtype);
  if (st != FA_OK) return st;
  bool scored = false;
  fa::WithScores<fa::FwdParams> p;
  if ((st = check_scores(scores, scale, true, sh.packed(), &scored, &p.sc))) return st;
  if (sh.empty()) return FA_OK;  // empty: nothing is read or written, pointers may be NULL
  if ((st = check_ptr(q, "q")) || (st = check_ptr(k, "k")) || (st = check_ptr(v, "v")) ||
      (st = check_ptr(o, "o")) || (st = check_ptr(lse, "lse")))
    return st;
  if (sh.packed() && !sh.cu) return fail(FA_ERR_INVALID_ARG, "cu_seqlens is NULL");
  int chunk = 0, shards = 1;
  if (split > 0) {
    splitkv_layout(sh.S, split, &chunk, &shards);
    const size_t need = splitkv_bytes(sh, shards);
    if (!workspace) return fail(FA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (workspace_bytes < need) return fail(FA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return fail(FA_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    if (static_cast<int64_t>(shards) * sh.B * sh.H > 65535 * 65535LL)
      return fail(FA_ERR_UNSUPPORTED, "too many shards");
    if (shards > 65535) return fail(FA_ERR_UNSUPPORTED, "at most 65535 shards");
  }
  const bool bf16 = dtype == FA_BF16;
  // Q in 128-row boxes (a CTA's own tiles); K and V in 64-row boxes.
  CUtensorMap tq, tk, tv;
  if ((st = encode_input(&tq, q, bf16, sh, sh.H, "q")) || (st = encode_input(&tk, k, bf16, sh, sh.H_kv, "k", 64)) ||
      (st = encode_input(&tv, v, bf16, sh, sh.H_kv, "v", 64)))
    return st;
  p.o = o;
  p.lse = lse;
  p.S = static_cast<int>(sh.S);
  p.cu_seqlens = sh.cu;
  p.heads = static_cast<int>(sh.H);
  p.total = static_cast<int>(sh.packed() ? sh.total : 0);
  const int rows_per_cta = fa::fwd_rows_per_cta(static_cast<int>(sh.D));
  p.n_m_tiles = static_cast<int>((sh.S + rows_per_cta - 1) / rows_per_cta);  // CTAs per (b, h)
  p.causal = causal ? 1 : 0;
  p.win_left = sh.kernel_left();
  p.win_right = sh.kernel_right(causal != 0);
  p.group = static_cast<int>(sh.H / sh.H_kv);
  p.kv_chunk = chunk;
  const int64_t rows = sh.B * sh.H * sh.S;
  p.o_part = split > 0 ? static_cast<float*>(workspace) : nullptr;
  p.lse_part = split > 0 ? static_cast<float*>(workspace) + static_cast<size_t>(shards) * rows * sh.D : nullptr;
  p.scale_log2 = scale * kLog2e;
  p.err = fa::device_error_word();
  if (!p.err) return fail(FA_ERR_CUDA, "cannot resolve the device error word on the current device");
  p.wait_ns = fa::wait_limit_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (scored)
    return from_cuda(fa::launch_fwd_scored(static_cast<int>(sh.D), bf16, tq, tk, tv, p,
                                           static_cast<int>(sh.B * sh.H), s),
                     "forward launch");
  if ((st = from_cuda(fa::launch_fwd(static_cast<int>(sh.D), bf16, split > 0 || sh.general(causal != 0), tq, tk, tv,
                                     p, static_cast<int>(sh.B * sh.H), s),
                      "forward launch")))
    return st;
  if (split > 0)
    return from_cuda(fa::launch_merge_lse(static_cast<int>(sh.D), bf16, p.o_part, p.lse_part, shards, rows, o, lse, s),
                     "split-KV merge launch");
  return FA_OK;
}

// Backward workspace: the fp32 row vector Delta of every query row, then, when
// the dK/dV pass splits a K/V head's query heads over several CTAs, their fp32
// partial [dV | dK] rows.  Heads must already be validated (H_kv divides H).
size_t bwd_workspace_layout(const Shape& sh, int* splits, size_t* delta_bytes) {
  *splits = 1;
  *delta_bytes = 0;
  if (sh.B <= 0 || sh.H <= 0 || sh.S <= 0 || sh.H_kv <= 0 || (sh.packed() && sh.total <= 0)) return 0;
  *delta_bytes = round256(static_cast<size_t>(sh.q_rows()) * sizeof(float));
  *splits = fa::bwd_kv_splits(sh.B * sh.H_kv, (sh.S + 127) / 128, static_cast<int>(sh.H / sh.H_kv));
  if (*splits == 1) return *delta_bytes;
  return *delta_bytes + round256(static_cast<size_t>(*splits) * static_cast<size_t>(sh.kv_rows()) *
                                 static_cast<size_t>(2 * sh.D) * sizeof(float));
}

fa_status bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                   void* dq, void* dk, void* dv, const Shape& sh, int causal, float scale, fa_dtype dtype,
                   void* workspace, size_t workspace_bytes, void* stream, void* const* marks,
                   const fa_scores* scores = nullptr) {
  g_detail[0] = 0;
  fa_status st = check_shape(sh, scale, dtype);
  if (st != FA_OK) return st;
  bool scored = false;
  fa::WithScores<fa::BwdParams> p;
  if ((st = check_scores(scores, scale, true, sh.packed(), &scored, &p.sc))) return st;
  if (sh.empty()) return FA_OK;  // empty: nothing is read or written, pointers may be NULL
  if ((st = check_ptr(q, "q")) || (st = check_ptr(k, "k")) || (st = check_ptr(v, "v")) ||
      (st = check_ptr(o, "o")) || (st = check_ptr(dout, "dout")) || (st = check_ptr(lse, "lse")) ||
      (st = check_ptr(dq, "dq")) || (st = check_ptr(dk, "dk")) || (st = check_ptr(dv, "dv")))
    return st;
  if (sh.packed() && !sh.cu) return fail(FA_ERR_INVALID_ARG, "cu_seqlens is NULL");
  int splits = 1;
  size_t delta_bytes = 0;
  const size_t need = bwd_workspace_layout(sh, &splits, &delta_bytes);
  if (!workspace) return fail(FA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (workspace_bytes < need)
    return fail(FA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(FA_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  const bool bf16 = dtype == FA_BF16;
  fa::BwdMaps maps;
  if ((st = encode_input(&maps.q128, q, bf16, sh, sh.H, "q")) ||
      (st = encode_input(&maps.k128, k, bf16, sh, sh.H_kv, "k")) ||
      (st = encode_input(&maps.v128, v, bf16, sh, sh.H_kv, "v")) ||
      (st = encode_input(&maps.do128, dout, bf16, sh, sh.H, "dout")) ||
      (st = encode_input(&maps.q64, q, bf16, sh, sh.H, "q", 64)) ||
      (st = encode_input(&maps.k64, k, bf16, sh, sh.H_kv, "k", 64)) ||
      (st = encode_input(&maps.v64, v, bf16, sh, sh.H_kv, "v", 64)) ||
      (st = encode_input(&maps.do64, dout, bf16, sh, sh.H, "dout", 64)))
    return st;
  p.o = o;
  p.dout = dout;
  p.lse = lse;
  p.delta = static_cast<float*>(workspace);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.S = static_cast<int>(sh.S);
  p.cu_seqlens = sh.cu;
  p.heads = static_cast<int>(sh.H);
  p.total = static_cast<int>(sh.packed() ? sh.total : 0);
  p.BH = static_cast<int>(sh.B * sh.H);
  p.group = static_cast<int>(sh.H / sh.H_kv);
  p.kv_splits = splits;
  p.dkv_part = splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + delta_bytes) : nullptr;
  p.n_tiles = static_cast<int>((sh.S + 127) / 128);
  p.causal = causal ? 1 : 0;
  p.win_left = sh.kernel_left();
  p.win_right = sh.kernel_right(causal != 0);
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.err = fa::device_error_word();
  if (!p.err) return fail(FA_ERR_CUDA, "cannot resolve the device error word on the current device");
  p.wait_ns = fa::wait_limit_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int Di = static_cast<int>(sh.D);
  const int64_t q_rows = sh.q_rows(), kv_rows = sh.kv_rows();
  auto mark = [&](int i) -> fa_status {
    if (!marks || !marks[i]) return FA_OK;
    return from_cuda(cudaEventRecord(static_cast<cudaEvent_t>(marks[i]), s), "event record");
  };
  const bool general = scored || sh.general(causal != 0);
  auto pass = [&](bool kv_outer, bool dependent) {
    if (scored) return fa::launch_bwd_scored(Di, bf16, kv_outer, maps, p, s);
    return kv_outer ? fa::launch_bwd_dkdv(Di, bf16, general, maps, p, s, dependent)
                    : fa::launch_bwd_dq(Di, bf16, general, maps, p, s, dependent);
  };
  const bool fused_delta = fa::bwd_dq_computes_delta(Di, general);
  // Delta then dK/dV then dQ; or, when the dQ kernel computes Delta, dQ then dK/dV.
  // With modified scores Delta, dQ (which makes it exact), dK/dV.
  if ((st = mark(0))) return st;
  if (fused_delta) {
    if ((st = from_cuda(pass(false, false), "backward dQ launch"))) return st;
  } else if ((st = from_cuda(fa::launch_bwd_preprocess(Di, bf16, p, q_rows, s), "backward preprocess launch"))) {
    return st;
  }
  if ((st = mark(1))) return st;
  if (scored && (st = from_cuda(pass(false, true), "backward dQ launch"))) return st;
  // The second and third kernels are programmatic dependent launches: their
  // first CTAs start as the previous kernel's last ones finish.
  if ((st = from_cuda(pass(true, true), "backward dK/dV launch"))) return st;
  if (splits > 1 &&
      (st = from_cuda(fa::launch_bwd_dkv_reduce(Di, bf16, p, kv_rows, s), "backward dK/dV reduce launch")))
    return st;
  if ((st = mark(2))) return st;
  if (!fused_delta && !scored && (st = from_cuda(pass(false, true), "backward dQ launch"))) return st;
  return mark(3);
}

Shape fixed(int64_t B, int64_t H, int64_t H_kv, int64_t S, int64_t D) {
  return Shape{B, H, H_kv, S, D, nullptr, 0, false};
}

Shape windowed(int64_t B, int64_t H, int64_t H_kv, int64_t S, int64_t D, int64_t left, int64_t right) {
  Shape sh{B, H, H_kv, S, D, nullptr, 0, false};
  sh.win_left = left;
  sh.win_right = right;
  return sh;
}

Shape packed(const int32_t* cu, int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv,
             int64_t D) {
  return Shape{batch, H, H_kv, max_seqlen, D, cu, total, true};
}

// ---------------------------------------------------------------------------
// Rotary positions and the paged cache.

fa_status check_dtype_d(int64_t D, fa_dtype dtype) {
  if (dtype != FA_FP16 && dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (D != 16 && D != 32 && D != 64 && D != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dimension D=%lld is not one of 16, 32, 64, 128", (long long)D);
  return FA_OK;
}

fa_status check_tokens(int64_t total, int64_t H, int64_t H_kv) {
  if (total < 0 || H < 0 || H_kv < 0)
    return fail(FA_ERR_INVALID_ARG, "negative size: total=%lld H=%lld H_kv=%lld", (long long)total, (long long)H,
                (long long)H_kv);
  // total, H, H_kv < 2^31 each, so their products with 128 fit 64 bits
  if (total >= (int64_t(1) << 31) || H >= (int64_t(1) << 20) || H_kv >= (int64_t(1) << 20))
    return fail(FA_ERR_UNSUPPORTED, "total must be below 2^31, H and H_kv below 2^20");
  return FA_OK;
}

// Rows of `heads` dense heads, `stride` elements between tokens.
fa_status check_rows(const void* p, int64_t stride, int64_t heads, int64_t D, const char* name) {
  fa_status st = check_ptr(p, name);
  if (st != FA_OK) return st;
  if (stride % 8 != 0) return fail(FA_ERR_ALIGNMENT, "%s: stride %lld is not a multiple of 8 elements", name, (long long)stride);
  if (stride < heads * D || stride > (int64_t(1) << 40))
    return fail(FA_ERR_INVALID_ARG, "%s: stride %lld does not hold %lld heads of %lld", name, (long long)stride,
                (long long)heads, (long long)D);
  return FA_OK;
}

fa_status check_ints(const void* p, const char* name, unsigned bytes) {
  if (!p) return fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0)
    return fail(FA_ERR_ALIGNMENT, "%s is not %u-byte aligned", name, bytes);
  return FA_OK;
}

fa_status check_rotation(int64_t rot_dim, int64_t D, int64_t least, float magnitude, const void* steps) {
  if (rot_dim < least || rot_dim > D || rot_dim % 2 != 0)
    return fail(FA_ERR_INVALID_ARG, "rot_dim=%lld must be even, between %lld and D=%lld", (long long)rot_dim,
                (long long)least, (long long)D);
  if (!std::isfinite(magnitude)) return fail(FA_ERR_INVALID_ARG, "magnitude must be finite");
  return rot_dim > 0 ? check_ints(steps, "steps", 8) : FA_OK;
}

fa_status check_cache(const fa_paged_cache* c, int64_t H_kv, int64_t D) {
  if (!c) return fail(FA_ERR_INVALID_ARG, "cache is NULL");
  fa_status st;
  if ((st = check_ptr(c->k, "cache.k")) || (st = check_ptr(c->v, "cache.v")) ||
      (st = check_ints(c->block_table, "cache.block_table", 4)) || (st = check_ints(c->kv_lens, "cache.kv_lens", 4)))
    return st;
  const int64_t ps = c->page_size;
  if (ps < 16 || (ps & (ps - 1)) != 0 || ps > (int64_t(1) << 30))
    return fail(FA_ERR_UNSUPPORTED, "page_size=%lld is not a power of two from 16 to 2^30", (long long)ps);
  if (c->num_pages < 1 || c->num_pages >= (int64_t(1) << 31) - 1 || c->table_stride < 1 ||
      c->table_stride >= (int64_t(1) << 31))
    return fail(FA_ERR_INVALID_ARG, "num_pages=%lld and table_stride=%lld must be positive, below 2^31 - 1",
                (long long)c->num_pages, (long long)c->table_stride);
  if (c->table_pages < 0 || c->table_pages > c->table_stride)
    return fail(FA_ERR_INVALID_ARG, "table_pages=%lld must be between 0 and table_stride=%lld",
                (long long)c->table_pages, (long long)c->table_stride);
  const int64_t sp = c->page_stride, sr = c->row_stride, sh = c->head_stride;
  if (sp <= 0 || sr <= 0 || sh <= 0) return fail(FA_ERR_INVALID_ARG, "cache strides must be positive");
  if (sp % 8 != 0 || sr % 8 != 0 || sh % 8 != 0)
    return fail(FA_ERR_ALIGNMENT, "cache strides must be multiples of 8 elements");
  // 40 bits of bytes is what a tensor map's strides hold.
  if (sp >= (int64_t(1) << 39) || sr >= (int64_t(1) << 39) || sh >= (int64_t(1) << 39))
    return fail(FA_ERR_UNSUPPORTED, "cache strides must be below 2^39 elements");
  if (sh < D || sr < D || sp < D) return fail(FA_ERR_INVALID_ARG, "cache strides must be at least D");
  // Rows are apart when, sorted by stride, each dimension spans what is inside it.
  struct Dim { int64_t stride, n; } d[3] = {{sh, H_kv}, {sr, ps}, {sp, c->num_pages}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (d[j].n == 1 ? false : (d[j + 1].n == 1 || d[j].stride > d[j + 1].stride)) {
        const Dim t = d[j];
        d[j] = d[j + 1];
        d[j + 1] = t;
      }
  int64_t span = D;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    if (x.stride < span) return fail(FA_ERR_INVALID_ARG, "cache strides make rows overlap");
    if (x.n - 1 > ((int64_t(1) << 60) - span) / x.stride) return fail(FA_ERR_UNSUPPORTED, "cache too large");
    span += (x.n - 1) * x.stride;
  }
  return FA_OK;
}

int log2_of(int64_t x) {
  int s = 0;
  while ((int64_t(1) << s) < x) ++s;
  return s;
}

// Keys a row of the block table can hold (at most kMaxPagedLen).
int64_t table_keys(const fa_paged_cache* c) {
  const int64_t pages = c->table_pages ? c->table_pages : c->table_stride;
  return pages > fa::kMaxPagedLen / c->page_size ? fa::kMaxPagedLen : pages * c->page_size;
}

fa_status rope_impl(const void* q, int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                    int64_t q_out_stride, void* k_out, int64_t k_out_stride, const int32_t* positions,
                    const uint64_t* steps, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                    int interleaved, float magnitude, float sign, fa_dtype dtype, void* stream) {
  g_detail[0] = 0;
  fa_status st;
  if ((st = check_dtype_d(D, dtype)) || (st = check_tokens(total, H, H_kv))) return st;
  if (total == 0 || H + H_kv == 0) return FA_OK;
  if (H > 0 && ((st = check_rows(q, q_stride, H, D, "q")) || (st = check_rows(q_out, q_out_stride, H, D, "q_out"))))
    return st;
  if (H_kv > 0 &&
      ((st = check_rows(k, k_stride, H_kv, D, "k")) || (st = check_rows(k_out, k_out_stride, H_kv, D, "k_out"))))
    return st;
  if ((st = check_ints(positions, "positions", 4)) || (st = check_rotation(rot_dim, D, 2, magnitude, steps))) return st;
  if ((H > 0 && q == q_out && q_stride != q_out_stride) || (H_kv > 0 && k == k_out && k_stride != k_out_stride))
    return fail(FA_ERR_INVALID_ARG, "in place needs equal strides");
  fa::RopeParams p = {};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.positions = positions;
  p.steps = reinterpret_cast<const unsigned long long*>(steps);
  p.total = static_cast<int>(total);
  p.H = static_cast<int>(H);
  p.H_kv = static_cast<int>(H_kv);
  p.D = static_cast<int>(D);
  p.r = static_cast<int>(rot_dim / 2);
  p.interleaved = interleaved ? 1 : 0;
  p.mag = magnitude;
  p.mag_sin = sign * magnitude;
  return from_cuda(fa::launch_rope(p, dtype == FA_BF16, false, 1, static_cast<cudaStream_t>(stream)), "rope launch");
}

// One of the two paged-attention kernels in a call: its tiling, and its share
// of the workspace.
struct PagedPart {
  bool used = false;
  int N;               // fa_paged_kernel: rows it is instantiated for
  int tok_tile, tiles, grid, part_rows;
  int tok_lo, tok_hi, small;
  size_t o_at, lse_at, desc_at;  // byte offsets in the workspace
};
struct PagedPlan {
  PagedPart few, tile;
  size_t go_at;  // calls of both kernels: byte offset of their word (PagedParams::go)
  size_t bytes;
};

// The tiling of a call; false when it is empty or, with `launch`, has too many
// units.  The workspace never grows as max_q or max_k get smaller, so a launch
// may plan with tighter bounds than those its workspace was sized for.
bool paged_plan(int64_t batch, int64_t max_q, int64_t max_k, int64_t H, int64_t H_kv, int64_t D, bool launch,
                PagedPlan* plan) {
  if (batch <= 0 || max_q <= 0 || max_k < 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || H / H_kv > 128 ||
      batch >= (int64_t(1) << 31) || max_q > fa::kMaxPagedLen || max_k > fa::kMaxPagedLen ||
      H >= (int64_t(1) << 20))
    return false;
  const int64_t G = H / H_kv;
  plan->bytes = 0;
  auto add = [&](PagedPart* part, int64_t tok, int64_t longest, int64_t block, int64_t slot_rows,
                 int64_t ctas, int64_t cost) -> bool {
    part->used = true;
    part->tok_tile = static_cast<int>(tok < longest ? tok : longest);
    part->tiles = static_cast<int>((longest + part->tok_tile - 1) / part->tok_tile);
    part->part_rows = static_cast<int>(slot_rows);
    if (launch && batch > (int64_t(1) << 30) / part->tiles) return false;
    const int64_t units = batch * part->tiles;               // at most 2^30 in a launch
    const int64_t blocks = (max_k + block - 1) / block + 1;  // of a unit, at most
    const bool many = units > (int64_t(1) << 37) / (blocks * H_kv);
    if (launch && many) return false;  // a CTA's run of blocks fits 31 bits
    const int64_t most = many ? int64_t(1) << 37 : units * H_kv * blocks;
    part->grid = static_cast<int>(most < ctas ? most : ctas);
    part->small = most * cost < (int64_t(1) << 31) / 304;  // (share x CTA stays below 2^31 too)
    part->o_at = plan->bytes;
    part->lse_at = part->o_at + round256(static_cast<size_t>(2) * part->grid * part->part_rows * D * sizeof(float));
    part->desc_at = part->lse_at + round256(static_cast<size_t>(2) * part->grid * part->part_rows * sizeof(float));
    // (not by the grid: a call of fewer rows a unit may have twice the CTAs)
    plan->bytes = part->desc_at + round256(static_cast<size_t>(2 * fa::kPagedSms) * sizeof(int4));
    return true;
  };
  const bool chunks = max_q * G > fa::kFewRows;
  // Sequences of few rows: all of them, or those of a mixed batch.
  if (!chunks || (batch > 1 && G <= fa::kFewRows)) {
    const int64_t longest = chunks ? fa::kFewRows / G : max_q;
    plan->few.N = fa::paged_rows(longest * G);
    plan->few.tok_lo = 0;
    plan->few.tok_hi = static_cast<int>(longest);
    const int64_t ctas = fa::kPagedSms * fa::paged_ctas(static_cast<int>(D), plan->few.N);
    if (!add(&plan->few, longest, longest, 128, plan->few.N, ctas, 1)) return false;
  }
  if (chunks) {
    const int Di = static_cast<int>(D);
    plan->tile.tok_lo = plan->few.used ? plan->few.tok_hi + 1 : 0;
    plan->tile.tok_hi = static_cast<int>(max_q);
    const int64_t tok = fa::paged_tile_tiles(Di) * (128 / G);
    if (!add(&plan->tile, tok, max_q, fa::paged_tile_block(Di), tok * G, fa::kPagedSms,
             fa::kMaxBlockCost))
      return false;
  }
  plan->go_at = plan->bytes;
  if (plan->few.used && plan->tile.used) plan->bytes += 256;
  return true;
}

// A number that no other launch of the process has, and that other contents of a
// workspace hardly are (an odd multiple, modulo 2^64, of a count).
unsigned long long launch_ticket() {
  static std::atomic<unsigned long long> count{0};
  return (count.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull;
}

// Tensor map of a packed [T, H, D] Q, box {row chunk, G heads, tok_tile tokens}.
fa_status encode_paged_q(CUtensorMap* map, const void* q, bool bf16, int64_t total, int64_t H, int64_t D, int64_t G,
                         int tok_tile) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int rb = fa::row_bytes_for(static_cast<int>(D));
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(total)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D * 2), static_cast<cuuint64_t>(H * D * 2)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(rb / 2), static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tok_tile)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUtensorMapSwizzle swz = rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : (rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "tensor map for q: cuTensorMapEncodeTiled error %d", (int)r);
  return FA_OK;
}

// Tensor map of the cache's K or V: {D, H_kv, page_size, num_pages}, box
// {row chunk, 1, min(page_size, block), 1}.  Pages from num_pages on read zero.
fa_status encode_paged_kv(CUtensorMap* map, const void* base, bool bf16, const fa_paged_cache* c, int64_t H_kv,
                          int64_t D, int64_t block, const char* name) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int rb = fa::row_bytes_for(static_cast<int>(D));
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_kv),
                        static_cast<cuuint64_t>(c->page_size), static_cast<cuuint64_t>(c->num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c->head_stride * 2), static_cast<cuuint64_t>(c->row_stride * 2),
                           static_cast<cuuint64_t>(c->page_stride * 2)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(rb / 2), 1u,
                       static_cast<cuuint32_t>(c->page_size < block ? c->page_size : block), 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  CUtensorMapSwizzle swz = rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : (rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  // L2 lines fetched along with a miss: no more than lies contiguous in the
  // cache (a row of one head, unless a head's rows follow one another).
  const int64_t run = c->row_stride == D ? 256 : D * 2;
  const CUtensorMapL2promotion promote = run >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : run == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                         : run == 64  ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_NONE;
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "tensor map for %s: cuTensorMapEncodeTiled error %d", name, (int)r);
  return FA_OK;
}

// The drafted trees of a call.
struct Tree {
  const int32_t* positions;
  const uint32_t* rows;
  int64_t stride, words;
};

fa_status paged_fwd_impl(const void* q, void* o, float* lse, const fa_paged_cache* cache, const int32_t* cu_seqlens,
                         int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t total, int64_t H,
                         int64_t H_kv, int64_t D, int causal, int64_t window_left, int64_t window_right, float scale,
                         fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream,
                         const fa_scores* scores, const Tree* tree) {
  g_detail[0] = 0;
  fa_status st;
  if ((st = check_dtype_d(D, dtype)) || (st = check_tokens(total, H, H_kv)) || (st = check_heads(H, H_kv))) return st;
  if (!std::isfinite(scale)) return fail(FA_ERR_INVALID_ARG, "scale must be finite");
  fa::PagedScoredParams p = {};
  bool scored = false;
  if ((st = check_scores(scores, scale, false, false, &scored, &p.sc))) return st;
  scored = scored || tree;
  if (batch < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(FA_ERR_INVALID_ARG, "negative size: batch=%lld max_seqlen_q=%lld max_seqlen_k=%lld", (long long)batch,
                (long long)max_seqlen_q, (long long)max_seqlen_k);
  if (batch == 0 || max_seqlen_q == 0 || total == 0 || H == 0) return FA_OK;
  if (max_seqlen_q > fa::kMaxPagedLen || max_seqlen_k > fa::kMaxPagedLen)
    return fail(FA_ERR_UNSUPPORTED, "max_seqlen_q and max_seqlen_k must be at most 2^29");
  if (H / H_kv > 128) return fail(FA_ERR_UNSUPPORTED, "more than 128 query heads to a K/V head");
  if ((st = check_ptr(q, "q")) || (st = check_ptr(o, "o")) || (st = check_ptr(lse, "lse")) ||
      (st = check_cache(cache, H_kv, D)) || (st = check_ints(cu_seqlens, "cu_seqlens", 4)))
    return st;
  if (tree) {
    if ((st = check_ints(tree->positions, "positions", 4)) || (st = check_ints(tree->rows, "tree", 4))) return st;
    const int64_t most = max_seqlen_q < total ? max_seqlen_q : total;
    if (tree->words < (most + 31) / 32 || tree->stride < tree->words)
      return fail(FA_ERR_INVALID_ARG, "tree rows of %lld words, %lld apart, for up to %lld new tokens",
                  (long long)tree->words, (long long)tree->stride, (long long)most);
    if (tree->stride >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "tree_stride must be below 2^31");
    p.tree = tree->rows;
    p.positions = tree->positions;
    p.tree_stride = tree->stride;
    p.tree_words = static_cast<int>(tree->words);
  }
  // No sequence has more new tokens than there are, or more keys than its row of
  // the table holds, however loose the bounds.
  const int64_t most_q = max_seqlen_q < total ? max_seqlen_q : total;
  const int64_t most_k = max_seqlen_k < table_keys(cache) ? max_seqlen_k : table_keys(cache);
  PagedPlan plan;
  if (!paged_plan(batch, most_q, most_k, H, H_kv, D, true, &plan))
    return fail(FA_ERR_UNSUPPORTED, "batch and lengths too large");
  const int shift = log2_of(cache->page_size);
  if (!workspace) return fail(FA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", plan.bytes);
  if (workspace_bytes < plan.bytes)
    return fail(FA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, plan.bytes);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(FA_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  const bool bf16 = dtype == FA_BF16;
  const int64_t G = H / H_kv;
  p.o = o;
  p.lse = lse;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = cache->kv_lens;
  p.block_table = cache->block_table;
  p.table_stride = cache->table_stride;
  p.batch = static_cast<int>(batch);
  p.H = static_cast<int>(H);
  p.H_kv = static_cast<int>(H_kv);
  p.G = static_cast<int>(G);
  p.total = static_cast<int>(total);
  p.max_q = static_cast<int>(max_seqlen_q);
  p.max_k = static_cast<int>(most_k);
  p.win_left = window_left < 0 || window_left >= max_seqlen_k ? fa::kNoWindow : static_cast<int>(window_left);
  p.win_right =
      causal ? 0 : (window_right < 0 || window_right >= max_seqlen_k + max_seqlen_q ? fa::kNoWindow : static_cast<int>(window_right));
  p.page_shift = shift;
  p.num_pages = static_cast<int>(cache->num_pages);
  p.scale_log2 = scale * kLog2e;
  p.err = fa::device_error_word();
  if (!p.err) return fail(FA_ERR_CUDA, "cannot resolve the device error word on the current device");
  p.wait_ns = fa::wait_limit_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  fa::PagedMergeParams mp = {};
  mp.o = o;
  mp.lse = lse;
  mp.G = p.G;
  mp.H = p.H;
  mp.total = p.total;
  if (plan.few.used && plan.tile.used) {
    p.go = mp.go = reinterpret_cast<unsigned long long*>(ws + plan.go_at);
    p.ticket = launch_ticket();
  }
  int sets = 0, grid = 0;
  auto run = [&](const PagedPart& part, bool tile) -> fa_status {
    p.tok_tile = part.tok_tile;
    p.tiles = part.tiles;
    p.tok_lo = part.tok_lo;
    p.tok_hi = part.tok_hi;
    p.small = part.small;
    p.sub_tok = static_cast<int>(128 / G);
    p.costs = fa::paged_costs(static_cast<int>(D));
    p.part_rows = part.part_rows;
    p.after_tile = !tile && plan.tile.used;
    p.o_part = reinterpret_cast<float*>(ws + part.o_at);
    p.lse_part = reinterpret_cast<float*>(ws + part.lse_at);
    p.desc = reinterpret_cast<int4*>(ws + part.desc_at);
    mp.parts[sets++] = fa::PagedParts{p.o_part, p.lse_part, p.desc, part.part_rows, part.grid, tile ? 1 : 0};
    if (part.grid > grid) grid = part.grid;
    const int Di = static_cast<int>(D);
    const int64_t block = tile ? fa::paged_tile_block(Di) : 128;
    CUtensorMap tq, tk, tv;
    fa_status r;
    if ((r = encode_paged_q(&tq, q, bf16, total, H, D, G, tile ? static_cast<int>(128 / G) : part.tok_tile)) ||
        (r = encode_paged_kv(&tk, cache->k, bf16, cache, H_kv, D, block, "cache.k")) ||
        (r = encode_paged_kv(&tv, cache->v, bf16, cache, H_kv, D, block, "cache.v")))
      return r;
    cudaError_t e = cudaErrorInvalidValue;
    if (scored) {
      switch (D) {
        case 16: e = fa::launch_paged_scored_d16(part.N, tile, bf16, tq, tk, tv, p, part.grid, s); break;
        case 32: e = fa::launch_paged_scored_d32(part.N, tile, bf16, tq, tk, tv, p, part.grid, s); break;
        case 64: e = fa::launch_paged_scored_d64(part.N, tile, bf16, tq, tk, tv, p, part.grid, s); break;
        case 128: e = fa::launch_paged_scored_d128(part.N, tile, bf16, tq, tk, tv, p, part.grid, s); break;
      }
    } else if (tile) {
      switch (D) {
        case 16: e = fa::launch_paged_tile_d16(bf16, tq, tk, tv, p, part.grid, s); break;
        case 32: e = fa::launch_paged_tile_d32(bf16, tq, tk, tv, p, part.grid, s); break;
        case 64: e = fa::launch_paged_tile_d64(bf16, tq, tk, tv, p, part.grid, s); break;
        case 128: e = fa::launch_paged_tile_d128(bf16, tq, tk, tv, p, part.grid, s); break;
      }
    } else {
      switch (D) {
        case 16: e = fa::launch_paged_d16(part.N, bf16, tq, tk, tv, p, part.grid, s); break;
        case 32: e = fa::launch_paged_d32(part.N, bf16, tq, tk, tv, p, part.grid, s); break;
        case 64: e = fa::launch_paged_d64(part.N, bf16, tq, tk, tv, p, part.grid, s); break;
        case 128: e = fa::launch_paged_d128(part.N, bf16, tq, tk, tv, p, part.grid, s); break;
      }
    }
    return from_cuda(e, "paged attention launch");
  };
  // The long sequences first: the few-row kernel's CTAs start as theirs end.
  if (plan.tile.used && (st = run(plan.tile, true))) return st;
  if (plan.few.used && (st = run(plan.few, false))) return st;
  return from_cuda(fa::launch_paged_merge(static_cast<int>(D), bf16, mp, grid, sets, s), "paged merge launch");
}

}  // namespace

extern "C" {

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H, int64_t S,
                 int64_t D, int causal, float scale, fa_dtype dtype, void* stream) {
  return fwd_impl(q, k, v, o, lse, fixed(B, H, H, S, D), causal, scale, dtype, stream);
}

fa_status fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                     int64_t H_kv, int64_t S, int64_t D, int causal, float scale, fa_dtype dtype, void* stream) {
  return fwd_impl(q, k, v, o, lse, fixed(B, H, H_kv, S, D), causal, scale, dtype, stream);
}

fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                        int64_t H_kv, int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right,
                        float scale, fa_dtype dtype, void* stream) {
  return fwd_impl(q, k, v, o, lse, windowed(B, H, H_kv, S, D, window_left, window_right), causal, scale, dtype,
                  stream);
}

fa_status fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                         int64_t H_kv, int64_t S, int64_t D, int causal, int64_t num_splits, float scale,
                         fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_splits < 1) {
    g_detail[0] = 0;
    return fail(FA_ERR_INVALID_ARG, "num_splits=%lld must be at least 1", (long long)num_splits);
  }
  return fwd_impl(q, k, v, o, lse, fixed(B, H, H_kv, S, D), causal, scale, dtype, stream, num_splits, workspace,
                  workspace_bytes);
}

size_t fa_fwd_splitkv_workspace_size(int64_t B, int64_t H, int64_t S, int64_t D, int64_t num_splits) {
  if (B <= 0 || H <= 0 || S <= 0 || num_splits < 1) return 0;
  int chunk = 0, shards = 1;
  splitkv_layout(S, num_splits, &chunk, &shards);
  return splitkv_bytes(fixed(B, H, H, S, D), shards);
}

int64_t fa_splitkv_num_splits(int64_t B, int64_t H, int64_t S, int64_t D) {
  // Enough shards to give every SM of a 152-SM GPU two CTAs, no more than one
  // shard per 128 keys.
  if (B <= 0 || H <= 0 || S <= 0 || (D != 16 && D != 32 && D != 64 && D != 128)) return 1;
  const int64_t rows_per_cta = fa::fwd_rows_per_cta(static_cast<int>(D));
  const int64_t ctas = B * H * ((S + rows_per_cta - 1) / rows_per_cta);
  const int64_t want = (2 * 152 + ctas - 1) / ctas;
  const int64_t cap = (S + 127) / 128;
  return want < 1 ? 1 : (want > cap ? cap : want);
}

fa_status fa_merge_lse(const float* o_part, const float* lse_part, void* o, float* lse, int64_t shards,
                       int64_t rows, int64_t D, fa_dtype dtype, void* stream) {
  g_detail[0] = 0;
  if (shards < 1 || rows < 0) return fail(FA_ERR_INVALID_ARG, "shards must be >= 1 and rows >= 0");
  if (dtype != FA_FP16 && dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (D != 16 && D != 32 && D != 64 && D != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dimension D=%lld is not one of 16, 32, 64, 128", (long long)D);
  if (shards > (int64_t(1) << 31) || (rows > 0 && shards > (int64_t(1) << 60) / (rows * (D + 1))))
    return fail(FA_ERR_UNSUPPORTED, "partials too large");
  if (rows == 0) return FA_OK;
  fa_status st;
  if ((st = check_ptr(o_part, "o_part")) || (st = check_ptr(lse_part, "lse_part")) || (st = check_ptr(o, "o")) ||
      (st = check_ptr(lse, "lse")))
    return st;
  return from_cuda(fa::launch_merge_lse(static_cast<int>(D), dtype == FA_BF16, o_part, lse_part,
                                        static_cast<int>(shards), rows, o, lse, static_cast<cudaStream_t>(stream)),
                   "merge launch");
}

fa_status fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                        const int32_t* cu_seqlens, int64_t batch, int64_t max_seqlen, int64_t total, int64_t H,
                        int64_t H_kv, int64_t D, int causal, float scale, fa_dtype dtype, void* stream) {
  return fwd_impl(q, k, v, o, lse, packed(cu_seqlens, batch, max_seqlen, total, H, H_kv, D), causal, scale, dtype,
                  stream);
}

size_t fa_bwd_workspace_size(int64_t B, int64_t H, int64_t S, int64_t D) {
  int splits = 1;
  size_t delta_bytes = 0;
  if (B < 0 || H < 0 || S < 0) return 0;
  return bwd_workspace_layout(fixed(B, H, H, S, D), &splits, &delta_bytes);
}

size_t fa_bwd_gqa_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S, int64_t D) {
  if (B < 0 || S < 0 || H_kv <= 0 || H <= 0 || H % H_kv != 0) return 0;
  int splits = 1;
  size_t delta_bytes = 0;
  return bwd_workspace_layout(fixed(B, H, H_kv, S, D), &splits, &delta_bytes);
}

size_t fa_bwd_varlen_workspace_size(int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv,
                                    int64_t D) {
  if (batch < 0 || max_seqlen < 0 || total < 0 || H_kv <= 0 || H <= 0 || H % H_kv != 0) return 0;
  int splits = 1;
  size_t delta_bytes = 0;
  return bwd_workspace_layout(packed(nullptr, batch, max_seqlen, total, H, H_kv, D), &splits, &delta_bytes);
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                 void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t S, int64_t D, int causal, float scale,
                 fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, fixed(B, H, H, S, D), causal, scale, dtype, workspace,
                  workspace_bytes, stream, nullptr);
}

fa_status fa_bwd_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t S, int64_t D,
                        int causal, float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                        void* stream, void* const* marks) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, fixed(B, H, H, S, D), causal, scale, dtype, workspace,
                  workspace_bytes, stream, marks);
}

fa_status fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                     void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv, int64_t S, int64_t D,
                     int causal, float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                     void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, fixed(B, H, H_kv, S, D), causal, scale, dtype, workspace,
                  workspace_bytes, stream, nullptr);
}

fa_status fa_bwd_gqa_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                            const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                            int64_t S, int64_t D, int causal, float scale, fa_dtype dtype, void* workspace,
                            size_t workspace_bytes, void* stream, void* const* marks) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, fixed(B, H, H_kv, S, D), causal, scale, dtype, workspace,
                  workspace_bytes, stream, marks);
}

fa_status fa_bwd_window_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                               int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right,
                               float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream,
                               void* const* marks) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, windowed(B, H, H_kv, S, D, window_left, window_right), causal,
                  scale, dtype, workspace, workspace_bytes, stream, marks);
}

fa_status fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                        int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right, float scale,
                        fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return fa_bwd_window_marked(q, k, v, o, dout, lse, dq, dk, dv, B, H, H_kv, S, D, causal, window_left,
                              window_right, scale, dtype, workspace, workspace_bytes, stream, nullptr);
}

fa_status fa_bwd_varlen_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens,
                               int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D,
                               int causal, float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                               void* stream, void* const* marks) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, packed(cu_seqlens, batch, max_seqlen, total, H, H_kv, D),
                  causal, scale, dtype, workspace, workspace_bytes, stream, marks);
}

fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens, int64_t batch,
                        int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D, int causal,
                        float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return fa_bwd_varlen_marked(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, batch, max_seqlen, total, H, H_kv, D,
                              causal, scale, dtype, workspace, workspace_bytes, stream, nullptr);
}

fa_status fa_fwd_scores(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                        int64_t H_kv, int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right,
                        const fa_scores* scores, float scale, fa_dtype dtype, void* stream) {
  return fwd_impl(q, k, v, o, lse, windowed(B, H, H_kv, S, D, window_left, window_right), causal, scale, dtype, stream,
                  0, nullptr, 0, scores);
}

fa_status fa_bwd_scores(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv, int64_t S,
                        int64_t D, int causal, int64_t window_left, int64_t window_right, const fa_scores* scores,
                        float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, windowed(B, H, H_kv, S, D, window_left, window_right), causal,
                  scale, dtype, workspace, workspace_bytes, stream, nullptr, scores);
}

fa_status fa_fwd_scores_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                               const int32_t* cu_seqlens, int64_t batch, int64_t max_seqlen, int64_t total, int64_t H,
                               int64_t H_kv, int64_t D, int causal, int64_t window_left, int64_t window_right,
                               const fa_scores* scores, float scale, fa_dtype dtype, void* stream) {
  Shape sh = packed(cu_seqlens, batch, max_seqlen, total, H, H_kv, D);
  sh.win_left = window_left;
  sh.win_right = window_right;
  const fa_scores plain = {};
  return fwd_impl(q, k, v, o, lse, sh, causal, scale, dtype, stream, 0, nullptr, 0, scores ? scores : &plain);
}

fa_status fa_bwd_scores_varlen(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens,
                               int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D,
                               int causal, int64_t window_left, int64_t window_right, const fa_scores* scores,
                               float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  Shape sh = packed(cu_seqlens, batch, max_seqlen, total, H, H_kv, D);
  sh.win_left = window_left;
  sh.win_right = window_right;
  const fa_scores plain = {};
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, sh, causal, scale, dtype, workspace, workspace_bytes, stream,
                  nullptr, scores ? scores : &plain);
}

fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dout,
                         const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t S,
                         int64_t D, int causal, float scale, fa_dtype dtype, void* stream) {
  g_detail[0] = 0;
  fa_status st = check_common(B, H, S, D, scale, dtype);
  if (st != FA_OK) return st;
  const int64_t BH = B * H;
  if (BH == 0 || S == 0) return FA_OK;
  if (BH > fa::kNoAllocMaxRows / S)
    return fail(FA_ERR_UNSUPPORTED, "fa_bwd_noalloc: B*H*S = %lld rows exceeds its fixed scratch of %lld rows",
                (long long)(BH * S), (long long)fa::kNoAllocMaxRows);
  cudaError_t e = cudaSuccess;
  float* delta = fa::noalloc_delta_address(&e);
  if (!delta) return from_cuda(e, "fa_bwd_noalloc: address of the scratch array");
  // The same kernels as fa_bwd, with the scratch array as the workspace.
  // Every row's Delta is written (by the Delta kernel or the dQ pass) before it
  // is read, so nothing needs clearing.
  return fa_bwd_marked(q, k, v, o, dout, lse, dq, dk, dv, B, H, S, D, causal, scale, dtype, delta,
                       static_cast<size_t>(fa::kNoAllocMaxRows) * sizeof(float), stream, nullptr);
}

fa_status fa_rope_inv_freq(int64_t rot_dim, double base, fa_rope_scaling scaling, double factor, double original_len,
                           double fast_turns, double slow_turns, double* inv_freq, float* magnitude) {
  g_detail[0] = 0;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > (1 << 20))
    return fail(FA_ERR_INVALID_ARG, "rot_dim=%lld must be even and at least 2", (long long)rot_dim);
  if (!inv_freq) return fail(FA_ERR_INVALID_ARG, "inv_freq is NULL");
  if (!std::isfinite(base) || base <= 0) return fail(FA_ERR_INVALID_ARG, "base must be finite and positive");
  if (scaling != FA_ROPE_NONE && scaling != FA_ROPE_LINEAR && scaling != FA_ROPE_BASE && scaling != FA_ROPE_PARTS)
    return fail(FA_ERR_INVALID_ARG, "unknown scaling %d", (int)scaling);
  if (scaling != FA_ROPE_NONE && (!std::isfinite(factor) || factor <= 0))
    return fail(FA_ERR_INVALID_ARG, "factor must be finite and positive");
  const bool parts = scaling == FA_ROPE_PARTS;
  if (parts && !(original_len > 0 && slow_turns > 0 && fast_turns > slow_turns && std::isfinite(original_len) &&
                 std::isfinite(fast_turns) && base > 1))
    return fail(FA_ERR_INVALID_ARG, "scaling by parts needs original_len > 0, fast_turns > slow_turns > 0, base > 1");
  const double rot = static_cast<double>(rot_dim);
  // (rot_dim = 2 has one pair, of frequency 1 whatever the base)
  if (scaling == FA_ROPE_BASE && rot_dim > 2) base *= std::pow(factor, rot / (rot - 2.0));
  double lo = 0, hi = 0;
  if (parts) {
    // Pair index (a real number) that makes `turns` turns in original_len positions.
    constexpr double kTwoPi = 6.283185307179586476925;
    auto pair_of = [&](double turns) {
      return rot * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(fast_turns)), 0.0);
    hi = std::fmin(std::ceil(pair_of(slow_turns)), rot - 1.0);
    // The ramp's end (before pair 0) or its start (past the last) may lie beyond
    // every pair: all are then slow, or all fast.
    if (pair_of(slow_turns) < 0) lo = hi - 1.0;
    else if (lo >= hi) hi = lo + 0.001;
  }
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * static_cast<double>(i) / rot);
    if (scaling == FA_ROPE_LINEAR) f /= factor;
    if (parts) {
      const double ramp = std::fmin(std::fmax((static_cast<double>(i) - lo) / (hi - lo), 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    inv_freq[i] = f;
  }
  if (magnitude) *magnitude = parts && factor > 1 ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return FA_OK;
}

fa_status fa_rope_steps(const double* inv_freq, int64_t n, uint64_t* steps) {
  g_detail[0] = 0;
  if (n < 0) return fail(FA_ERR_INVALID_ARG, "n=%lld is negative", (long long)n);
  if (n > 0 && (!inv_freq || !steps)) return fail(FA_ERR_INVALID_ARG, "inv_freq or steps is NULL");
  for (int64_t i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return fail(FA_ERR_INVALID_ARG, "inv_freq[%lld] is not finite", (long long)i);
  for (int64_t i = 0; i < n; ++i) {
    const double turns = inv_freq[i] / 6.283185307179586476925;
    const double frac = turns - std::floor(turns);  // [0, 1]; 1 when a tiny negative rounds up
    steps[i] = frac >= 1.0 ? 0 : static_cast<uint64_t>(std::ldexp(frac, 64));
  }
  return FA_OK;
}

fa_status fa_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                  int64_t q_out_stride, void* k_out, int64_t k_out_stride, const int32_t* positions,
                  const uint64_t* steps, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                  int interleaved, float magnitude, fa_dtype dtype, void* stream) {
  return rope_impl(q, q_stride, k, k_stride, q_out, q_out_stride, k_out, k_out_stride, positions, steps, total, H,
                   H_kv, D, rot_dim, interleaved, magnitude, 1.f, dtype, stream);
}

fa_status fa_rope_bwd(const void* dq_out, int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride, void* dq,
                      int64_t dq_stride, void* dk, int64_t dk_stride, const int32_t* positions,
                      const uint64_t* steps, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                      int interleaved, float magnitude, fa_dtype dtype, void* stream) {
  return rope_impl(dq_out, dq_out_stride, dk_out, dk_out_stride, dq, dq_stride, dk, dk_stride, positions, steps, total,
                   H, H_kv, D, rot_dim, interleaved, magnitude, -1.f, dtype, stream);
}

fa_status fa_paged_append(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const fa_paged_cache* cache,
                          const int32_t* cu_seqlens, const int32_t* positions, const uint64_t* steps, int64_t batch,
                          int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                          int interleaved, float magnitude, fa_dtype dtype, void* stream) {
  g_detail[0] = 0;
  fa_status st;
  if ((st = check_dtype_d(D, dtype)) || (st = check_tokens(total, H, H_kv))) return st;
  if (batch < 0 || max_seqlen < 0)
    return fail(FA_ERR_INVALID_ARG, "negative size: batch=%lld max_seqlen=%lld", (long long)batch, (long long)max_seqlen);
  if (batch >= (int64_t(1) << 31) || max_seqlen >= (int64_t(1) << 31))
    return fail(FA_ERR_UNSUPPORTED, "batch and max_seqlen must be below 2^31");
  if (H > 0 && H_kv == 0) return fail(FA_ERR_INVALID_ARG, "H_kv=0 with H=%lld", (long long)H);
  if (batch == 0 || max_seqlen == 0 || total == 0 || H_kv == 0) return FA_OK;
  if (H > 0 && ((st = check_rows(q, q_stride, H, D, "q")) || (st = check_rows(q_out, q_out_stride, H, D, "q_out"))))
    return st;
  if (H > 0 && q == q_out && q_stride != q_out_stride) return fail(FA_ERR_INVALID_ARG, "in place needs equal strides");
  if ((st = check_rows(k, k_stride, H_kv, D, "k")) || (st = check_rows(v, v_stride, H_kv, D, "v")) ||
      (st = check_cache(cache, H_kv, D)) || (st = check_ints(cu_seqlens, "cu_seqlens", 4)) ||
      (st = check_rotation(rot_dim, D, 0, magnitude, steps)))
    return st;
  if (positions && (st = check_ints(positions, "positions", 4))) return st;
  fa::RopeParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_out = cache->k;
  p.v_out = cache->v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.positions = positions;
  p.steps = reinterpret_cast<const unsigned long long*>(steps);
  p.total = static_cast<int>(total);
  p.H = static_cast<int>(H);
  p.H_kv = static_cast<int>(H_kv);
  p.D = static_cast<int>(D);
  p.r = static_cast<int>(rot_dim / 2);
  p.interleaved = interleaved ? 1 : 0;
  p.mag = p.mag_sin = magnitude;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = cache->kv_lens;
  p.block_table = cache->block_table;
  p.table_stride = cache->table_stride;
  p.page_stride = cache->page_stride;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.page_shift = log2_of(cache->page_size);
  p.num_pages = static_cast<int>(cache->num_pages);
  p.max_len = static_cast<int>(max_seqlen);
  p.max_kv = static_cast<int>(table_keys(cache));
  p.err = fa::device_error_word();
  if (!p.err) return fail(FA_ERR_CUDA, "cannot resolve the device error word on the current device");
  return from_cuda(
      fa::launch_rope(p, dtype == FA_BF16, true, static_cast<int>(batch), static_cast<cudaStream_t>(stream)),
      "append launch");
}

size_t fa_fwd_paged_workspace_size(int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t H,
                                   int64_t H_kv, int64_t D) {
  if (D != 16 && D != 32 && D != 64 && D != 128) return 0;
  PagedPlan plan;
  return paged_plan(batch, max_seqlen_q, max_seqlen_k, H, H_kv, D, false, &plan) ? plan.bytes : 0;
}

fa_status fa_fwd_paged(const void* q, void* o, float* lse, const fa_paged_cache* cache, const int32_t* cu_seqlens,
                       int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t total, int64_t H,
                       int64_t H_kv, int64_t D, int causal, int64_t window_left, int64_t window_right, float scale,
                       fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return paged_fwd_impl(q, o, lse, cache, cu_seqlens, batch, max_seqlen_q, max_seqlen_k, total, H, H_kv, D, causal,
                        window_left, window_right, scale, dtype, workspace, workspace_bytes, stream, nullptr, nullptr);
}

fa_status fa_fwd_paged_scores(const void* q, void* o, float* lse, const fa_paged_cache* cache,
                              const int32_t* cu_seqlens, int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k,
                              int64_t total, int64_t H, int64_t H_kv, int64_t D, int causal, int64_t window_left,
                              int64_t window_right, const fa_scores* scores, float scale, fa_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  return paged_fwd_impl(q, o, lse, cache, cu_seqlens, batch, max_seqlen_q, max_seqlen_k, total, H, H_kv, D, causal,
                        window_left, window_right, scale, dtype, workspace, workspace_bytes, stream, scores, nullptr);
}

fa_status fa_fwd_paged_tree(const void* q, void* o, float* lse, const fa_paged_cache* cache,
                            const int32_t* cu_seqlens, const int32_t* positions, const uint32_t* tree,
                            int64_t tree_stride, int64_t tree_words, int64_t batch, int64_t max_seqlen_q,
                            int64_t max_seqlen_k, int64_t total, int64_t H, int64_t H_kv, int64_t D,
                            int64_t window_left, const fa_scores* scores, float scale, fa_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const Tree t{positions, tree, tree_stride, tree_words};
  return paged_fwd_impl(q, o, lse, cache, cu_seqlens, batch, max_seqlen_q, max_seqlen_k, total, H, H_kv, D, 0,
                        window_left, -1, scale, dtype, workspace, workspace_bytes, stream, scores, &t);
}

fa_status fa_paged_keep(const fa_paged_cache* cache, const int32_t* cu_seqlens, const int32_t* path,
                        int64_t path_stride, int64_t path_cols, const int32_t* path_lens, int64_t batch,
                        int64_t max_seqlen, int64_t H_kv, int64_t D, fa_dtype dtype, void* stream) {
  g_detail[0] = 0;
  fa_status st;
  if ((st = check_dtype_d(D, dtype)) || (st = check_tokens(0, 0, H_kv))) return st;
  if (batch < 0 || max_seqlen < 0 || path_cols < 0)
    return fail(FA_ERR_INVALID_ARG, "negative size: batch=%lld max_seqlen=%lld path_cols=%lld", (long long)batch,
                (long long)max_seqlen, (long long)path_cols);
  if (batch >= (int64_t(1) << 31) || max_seqlen >= (int64_t(1) << 31) || path_cols >= (int64_t(1) << 31) ||
      path_stride >= (int64_t(1) << 40))
    return fail(FA_ERR_UNSUPPORTED, "batch, max_seqlen and path_cols must be below 2^31, path_stride below 2^40");
  if (path_stride < path_cols)
    return fail(FA_ERR_INVALID_ARG, "path rows of %lld entries, %lld apart", (long long)path_cols, (long long)path_stride);
  if (batch == 0 || max_seqlen == 0 || path_cols == 0 || H_kv == 0) return FA_OK;
  if ((st = check_cache(cache, H_kv, D)) || (st = check_ints(cu_seqlens, "cu_seqlens", 4)) ||
      (st = check_ints(path, "path", 4)) || (st = check_ints(path_lens, "path_lens", 4)))
    return st;
  if ((2 * (D / 8) * H_kv + 127) / 128 > ((int64_t(1) << 31) - 1) / batch)
    return fail(FA_ERR_UNSUPPORTED, "batch times H_kv * D too large");
  fa::KeepParams p = {};
  p.k = cache->k;
  p.v = cache->v;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = cache->kv_lens;
  p.block_table = cache->block_table;
  p.path = path;
  p.path_lens = path_lens;
  p.table_stride = cache->table_stride;
  p.path_stride = path_stride;
  p.page_stride = cache->page_stride;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.path_cols = static_cast<int>(path_cols);
  p.page_shift = log2_of(cache->page_size);
  p.num_pages = static_cast<int>(cache->num_pages);
  p.H_kv = static_cast<int>(H_kv);
  p.D = static_cast<int>(D);
  p.max_len = static_cast<int>(max_seqlen);
  p.max_kv = static_cast<int>(table_keys(cache));
  p.err = fa::device_error_word();
  if (!p.err) return fail(FA_ERR_CUDA, "cannot resolve the device error word on the current device");
  return from_cuda(fa::launch_keep(p, static_cast<int>(batch), static_cast<cudaStream_t>(stream)), "keep launch");
}

const char* fa_status_string(fa_status status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_ALIGNMENT: return "FA_ERR_ALIGNMENT";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
  }
  return "FA_ERR_UNKNOWN";
}

const char* fa_last_error_detail(void) { return g_detail; }

uint64_t fa_set_wait_limit_ns(uint64_t ns) {
  const unsigned long long v = ns == 0 ? fa::ptx::kWaitLimitNs : static_cast<unsigned long long>(ns);
  return static_cast<uint64_t>(fa::g_wait_limit_ns.exchange(v));
}

fa_status fa_check_device_errors(void* stream) {
  g_detail[0] = 0;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return from_cuda(e, "stream synchronize");
  int code = 0;
  e = cudaMemcpyFromSymbol(&code, fa::g_fa_device_error, sizeof(int));
  if (e != cudaSuccess) return from_cuda(e, "read device error word");
  if (code != 0) {
    const int zero = 0;
    cudaMemcpyToSymbol(fa::g_fa_device_error, &zero, sizeof(int));
    if (code == fa::kErrBadSeqlens)
      return fail(FA_ERR_INVALID_ARG, "cu_seqlens contradicts max_seqlen or the token count (checked on the device)");
    if (code == fa::kErrBadCache)
      return fail(FA_ERR_INVALID_ARG, "a paged cache length contradicts the call (checked on the device)");
    if (code == fa::kErrBadPage)
      return fail(FA_ERR_INVALID_ARG, "a block table entry in use is not a page (checked on the device)");
    if (code == fa::kErrBadPath)
      return fail(FA_ERR_INVALID_ARG, "a kept path contradicts the call (checked on the device)");
    return fail(FA_ERR_TIMEOUT, "device pipeline wait timed out (code %d)", code);
  }
  return FA_OK;
}

}  // extern "C"
