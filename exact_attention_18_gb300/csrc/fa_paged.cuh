// Parameters and launchers of the paged-cache operators: rotary positions,
// the append of new tokens to the cache, and their attention over it.
#pragma once

#include "fa_internal.cuh"

namespace fa {

// Codes of these kernels for the device error word, after DeviceErrorCode's.
constexpr int kErrBadCache = 6;  // a length below the new tokens', or past what the call allows
constexpr int kErrBadPage = 7;   // a block table entry in use is not a page

// Longest cache length (and largest window side): positions and their sums
// with a window side stay inside 32 bits.
constexpr int kMaxPagedLen = 1 << 29;

// Launches as a programmatic dependent of whatever precedes it on the stream:
// the grid may start while that kernel's last CTAs run.  Every kernel launched
// this way waits for the grids before it (griddep_wait, in every thread) ahead
// of its first access to the caller's memory, so it also never completes
// before them.  What the caller's earlier kernels may have written is read with
// plain loads, never through the read-only path (__ldg): that path may serve a
// line that was cached before the wait.  One grid may do without its wait at the
// front: the few-row kernel behind the tile kernel, where it has acquired that
// kernel's word that the grids before the call are done (say_go); it waits at
// its end, so that it does not complete before that kernel.
template <typename... Params, typename... Args>
inline cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Row t of q starts at q + t * q_stride (elements), its head h at + h * D;
// likewise k, v and the outputs.  Append: k_out and v_out are the caches'
// bases, rows at page * page_stride + row * row_stride + head * head_stride.
struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;
  void* v_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  const int* positions;  // [total]; append: may be nullptr (the cache position is the angle's)
  const unsigned long long* steps;  // [r] phase steps in 2^-64 turns a position
  int total;             // tokens
  int H, H_kv, D;
  int r;                 // rotated pairs
  int interleaved;
  int log2_items;        // threads a row, log2 (set by the launcher)
  int tok_per_cta;       // set by the launcher
  int tiles;             // append: CTAs per sequence (set by the launcher)
  int batch;             // append: sequences (set by the launcher)
  float mag, mag_sin;    // factors of cos and sin (mag_sin = -mag turns back)
  // append
  const int* cu_seqlens;
  const int* kv_lens;
  const int* block_table;
  int64_t table_stride;
  int64_t page_stride, row_stride, head_stride;
  int page_shift, num_pages;
  int max_len;           // largest number of new tokens of a sequence
  int max_kv;            // largest cache length the block table can hold
  int* err;
};

cudaError_t launch_rope(RopeParams p, bool bf16, bool append, int batch, cudaStream_t stream);

// Attention over the cache.  A "unit" is one (sequence, tile of tok_tile
// tokens, K/V head): its rows are tok_tile tokens x G query heads, its work the
// blocks of keys its rows can see.
struct PagedParams {
  void* o;               // [T, H, D]
  float* lse;            // [H, T] natural log
  const int* cu_seqlens;
  const int* kv_lens;
  const int* block_table;
  int64_t table_stride;
  int batch, H, H_kv, G;
  int total;             // T
  int max_q, max_k;
  int tok_tile;          // tokens of a tile
  int tiles;             // tiles of the longest sequence: ceil(max_q / tok_tile)
  int win_left, win_right;  // key j visible to position i iff i - win_left <= j <= i + win_right (and j < kv_len)
  int page_shift, num_pages;
  int tok_lo, tok_hi;    // sequences of tok_lo .. tok_hi new tokens are this kernel's
  int small;             // the cost of all blocks of the call is below 2^31 / 304
  int sub_tok;           // tile kernel: tokens of one of a unit's tiles
  unsigned costs;        // tile kernel: byte i is the cost of a block of a unit that fills i + 1 tiles
  int after_tile;        // few-row kernel: launched behind the tile kernel of the same call
  unsigned long long* go;    // calls of both kernels: the tile kernel writes `ticket` here when the grids before the
  unsigned long long ticket; // call have completed; the join clears it.  A number of the launch's own.
  float scale_log2;
  int part_rows;         // rows of a partial's slot
  float* o_part;         // [2 grid][part_rows x D] fp32, laid out as in PagedParts
  float* lse_part;       // [2 grid][part_rows] fp32, base 2
  int4* desc;            // [grid] unit whose first blocks CTA c computed without finishing it:
                         // {first token, tokens (0 = none), K/V head, last CTA}
  int* err;
  unsigned long long wait_ns;
};

// One main kernel's partials; parts[z] is joined by grid slice z.
struct PagedParts {
  const float* o_part;
  const float* lse_part;
  const int4* desc;
  int rows;  // of a slot
  int grid;  // CTAs of the main kernel
  int by_chunk;  // o_part is [slot][D / 4][rows][4] (the tile kernel's), else [slot][rows][D]
};
struct PagedMergeParams {
  PagedParts parts[2];
  void* o;
  float* lse;
  int G, H, total;
  unsigned long long* go;  // cleared (nullptr: none)
};

// Query rows (new tokens x G) of a sequence up to which the few-row kernel takes
// it, and rows of a unit it is instantiated for: the smallest that holds `rows`.
// Both kernels measured (us, few-row / tile; 16 sequences of 8192 keys, 4 K/V
// heads, G = 8, pages of 16), D = 16, 32, 64, 128: 40 rows 36.2 / 39.2, 35.0 /
// 42.8, 36.5 / 51.8, 53.8 / 71.2; 64 rows 36.6 / 39.6, 35.5 / 42.3, 37.4 / 51.5,
// 55.5 / 71.9.  With an instantiation for 128 rows that was tried, D = 64 and 128:
// 80 rows 58.7 / 47.3, 86.5 / 70.7; 128 rows 56.7 / 48.8, 68.5 / 73.4; 160 rows
// 92.2 / 57.9, 111 / 78.0.
constexpr int kFewRows = 64;
inline int paged_rows(int64_t rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64); }
constexpr int kPagedSms = 152;
// Costs of the tile kernel's blocks by the row tiles of their unit.  256 units of
// 8192 keys, 1 .. 4 tiles: D = 64 125, 171, 283, 301 us, D = 32 112, 149, 243, 275,
// D = 16 106, 141, 225, 260; D = 128, 1 and 2 tiles: 203, 248.  One table for
// D <= 64, a little above the first for short units' joins.  With 3, 5, 7, 8 / 3,
// 4, 7, 8 / 4, 5, 7, 8 / 4, 5, 8, 8 (D = 64): ragged chunks of 16 heads 86.7 / 84.7 /
// 84.4 / 85.0 us, 16 chunks of up to 1000 tokens 114 / 132 / 117 / 119, prompts of
// 40 and 20 tokens 36.4 / 31.7 / 32.1 / 32.1.
constexpr int kMaxBlockCost = 8;
constexpr unsigned paged_costs(int D) { return D == 128 ? 0x0807u : 0x08080504u; }
// CTAs per SM of the few-row kernel.
constexpr int paged_ctas(int D, int N) { return D <= 64 && N == 16 ? 2 : 1; }
// Rows of a unit of the tile kernel (tiles of 128 rows) and keys of its blocks.
inline int paged_tile_tiles(int D) { return D == 128 ? 2 : 4; }
inline int paged_tile_block(int D) { return D == 128 ? 128 : 64; }

cudaError_t launch_paged_tile_d16(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_tile_d32(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_tile_d64(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_tile_d128(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, int grid, cudaStream_t stream);
// `sets` of parts.
cudaError_t launch_paged_merge(int D, bool bf16, const PagedMergeParams& p, int grid, int sets, cudaStream_t stream);
cudaError_t launch_paged_d16(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_d32(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_d64(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_d128(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PagedParams& p, int grid, cudaStream_t stream);

}  // namespace fa
