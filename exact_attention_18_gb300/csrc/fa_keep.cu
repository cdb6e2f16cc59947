// Keeps the accepted path of a drafted tree: rows of the paged cache move to the
// slots right behind the sequence's context.
//
//   slot f + i  <-  slot f + path[i],  i = 0 .. m - 1,  f = kv_len - n
//
// path increases strictly, so path[i] >= i: row i's source lies at or behind its
// slot, and no slot written for i is a source of a later one.  A thread owns one
// 16-byte column of the rows (of K or V, one head) and takes the path's rows in
// order, a batch of kBatch loaded before it is stored; that is all the order the
// move needs, so there is no barrier and no scratch.
//
// What bounds it: latency.  A few rows a sequence are 0.1 to 3 MB in all; the chain
// offsets -> path -> block table -> row -> store and the launch are the time.  The
// loads of a batch are independent, and the grid starts as a programmatic dependent
// of the kernel before it.  48 sequences that keep up to 9 of 64 tokens, 8 heads of 128:
// 3.8 us in a stream of calls (1.2 MB: 0.4 us at the copy rate); one sequence 2.8.
#include "fa_kernel_common.cuh"
#include "fa_paged.cuh"

namespace fa {
using namespace ptx;

namespace {

constexpr int kKeepThreads = 128;
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kKeepThreads) fa_keep_kernel(const KeepParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int cols = p.D / 8 * p.H_kv;  // 16-byte columns of a row of one cache
  const int parts = (2 * cols + kKeepThreads - 1) / kKeepThreads;  // CTAs of a sequence
  const int b = blockIdx.x / parts, part = blockIdx.x - b * parts;
  const int a = p.cu_seqlens[b], e = p.cu_seqlens[b + 1], kv = p.kv_lens[b], m = p.path_lens[b];
  const int n = e - a, first = kv - n;
  const int* path = p.path + b * p.path_stride;
  int code = 0;
  if (a < 0 || e < a || n > p.max_len) code = kErrBadSeqlens;
  else if (kv < n || kv > p.max_kv) code = kErrBadCache;
  else if (m < 0 || m > n || m > p.path_cols) code = kErrBadPath;
  bool bad = false;
  if (code == 0)
    for (int i = threadIdx.x; i < m; i += kKeepThreads)
      bad |= path[i] >= n || path[i] <= (i == 0 ? -1 : path[i - 1]);
  if (__syncthreads_or(bad) && code == 0) code = kErrBadPath;
  if (code != 0) {
    if (threadIdx.x == 0 && part == 0) record_error(p.err, code);
    return;
  }
  const int col = part * kKeepThreads + threadIdx.x;
  if (col >= 2 * cols) return;
  const int c = col < cols ? col : col - cols;
  const int head = c / (p.D / 8);
  char* base = static_cast<char*>(col < cols ? p.k : p.v) +
               (head * p.head_stride + static_cast<int64_t>(c - head * (p.D / 8)) * 8) * 2;
  const int* table = p.block_table + b * p.table_stride;
  const int mask = (1 << p.page_shift) - 1;
  // The column's 16 bytes of key `key`; nullptr where its page is none.
  auto at = [&](int key) -> uint4* {
    const int page = table[key >> p.page_shift];
    if (page < 0 || page >= p.num_pages) {
      record_error(p.err, kErrBadPage);
      return nullptr;
    }
    return reinterpret_cast<uint4*>(base + (page * p.page_stride + (key & mask) * p.row_stride) * 2);
  };
  for (int i0 = 0; i0 < m; i0 += kBatch) {
    uint4 x[kBatch];
    int from[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) from[k] = i0 + k < m ? path[i0 + k] : i0 + k;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      x[k] = make_uint4(0, 0, 0, 0);
      if (from[k] == i0 + k) continue;  // in its place already (or past the path)
      const uint4* src = at(first + from[k]);
      if (src) x[k] = *src;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (from[k] == i0 + k) continue;
      uint4* dst = at(first + i0 + k);
      if (dst) *dst = x[k];
    }
  }
}

}  // namespace

cudaError_t launch_keep(const KeepParams& p, int batch, cudaStream_t stream) {
  const int64_t parts = (2 * static_cast<int64_t>(p.D / 8) * p.H_kv + kKeepThreads - 1) / kKeepThreads;
  if (parts * batch >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  return launch_dependent(fa_keep_kernel, dim3(static_cast<unsigned>(parts * batch)), kKeepThreads, 0, stream, p);
}

}  // namespace fa
