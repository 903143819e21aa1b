// fa2_paged.h -- declarations shared by the paged-cache translation units: the
// parameters their kernels read and the launchers.  Not part of the public
// interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fa2 {

// Bit of the device status word a paged kernel sets when a step's lengths, a
// slot or a page of a block table is out of range.
constexpr uint32_t kStatusBadPages = 4u;

// Largest batch of fa2_paged_plan: its kernel keeps two prefix sums of it in
// shared memory (128 KB).
constexpr int kPagedPlanMaxBatch = 16384;

// Rows of one query tile: group (query heads of one K/V head) x tokens.
constexpr int kPagedTileRows = 128;
constexpr int kPagedKeyTile = 64;

// Where a cache tensor's boxes lie in its 5-D map (64 columns, 8 rows, d / 64
// column blocks, then): ratio > 0: 8-row groups of a page, and page * ratio +
// head (the page stride is `ratio` head strides); ratio = 0: heads, pages.
struct PagedSide {
  int ratio;
  int extent;   // ratio > 0: the last coordinate's extent (out of range: zeros)
};

constexpr int kPagedMergeBytes = 32;   // sizeof(PagedMerge)

struct PagedParams {
  void* o;                // 16-bit output [total_q][heads_q][d] by strides
  float* lse;             // [heads_q][total_q], head stride lse_hs
  uint32_t* status;       // device status word (library-owned)
  const int* table;       // block table, rows of max_pages entries, table_stride apart
  const int* cu_q;        // [batch + 1] row offsets of the sequences' queries
  const int* lens_k;      // [batch] key counts
  long long table_stride, o_rs, o_hs, lse_hs;
  int batch, heads_kv, group;
  int tile_tokens;        // tokens of a query tile: 128 / group
  int total_q, max_q;
  int num_pages, page_size;
  int max_keys;           // a sequence's keys at most: max_pages * page_size
  unsigned page_magic, page_shift;   // k / page_size = (umulhi(k, magic) + k) >> shift for 0 <= k < 2^31
  int box_rows;           // key rows of a box: 8, 16, 32 or 64
  PagedSide k_side, v_side;
  int window_left, window_right, prefix;   // as KernelParams
  float scale_log2_mag;   // as KernelParams
  uint32_t qk_negate;     // as KernelParams
  int ctas;               // pieces the line of work is cut into
  int pair_ctas;          // most pairs that may run whole (the grid holds that many
                          // CTAs, rounded up to whole waves), or 0: up to ctas
  int cached_keys;        // keys (of one K/V head) whose K and V stay in the L2 cache
  int overhead;           // a pair's fixed cost on the line, in keys (whole key tiles)
  int min_share;          // keys of a piece at least (whole key tiles)
  int merge_cost;         // what a merge costs, in keys of one CTA's work (whole key tiles)
  int slot_rows;          // rows of a Q load and of a partial state: group x tokens
  float* ws_o;            // [2 * ctas][d / 4][slot_rows][4] partial O~
  float* ws_ml;           // [2 * ctas][slot_rows][2] partial (m, l), exp2 domain
  struct PagedMerge* merges;   // [ctas] pairs to merge, kPagedMergeBytes each
  int sinks;              // first keys a row sees as far as its band's right edge (0 without a left window)
};

struct PagedLaunchArgs {
  CUtensorMap tm_q;       // (d, group, heads_kv, total_q), boxes of 64 columns x group x 1 x tokens
  CUtensorMap tm_k, tm_v; // see PagedSide; boxes of 64 columns x 8 rows x d / 64 x (box_rows / 8 groups)
  PagedParams p;
  bool bf16;
  bool band;              // window_left >= 0 or prefix > 0
  bool wide;              // more than 64 rows in a query tile, or a line of 2^31 key tiles
  cudaStream_t stream;
};

int launch_paged_d64(const PagedLaunchArgs& a);
int launch_paged_d128(const PagedLaunchArgs& a);
int launch_paged_d256(const PagedLaunchArgs& a);

struct PagedPlanArgs {
  const int* context_lens;
  const int* query_lens;
  const int* free_pages;
  const int* free_count;
  int* table;
  int* cu_q;
  int* lens_k;
  int* slots;
  int* free_left;
  uint32_t* status;
  long long table_stride;
  int batch, max_pages, num_pages, page_size, total_q, num_free;
};

int launch_paged_plan(const PagedPlanArgs& a, cudaStream_t stream);

// One of K and V: new rows [total][heads][d] and cache [page][head][row][d],
// strides in 16-byte units.
struct PagedAppendSide {
  const uint4* src;
  uint4* dst;
  long long src_rs, src_hs;          // token, head
  long long dst_ps, dst_hs, dst_rs;  // page, head, row of a page
};

struct PagedAppendArgs {
  PagedAppendSide k, v;
  const int* slots;
  uint32_t* status;
  int total, heads, num_slots, page_size;
  int row_chunks_log2;    // 16-byte chunks of a head's row: d / 8 = 1 << row_chunks_log2
};

int launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);

// Launches a kernel as a programmatic dependent of what precedes it on the
// stream: it may be scheduled before that is done, and calls
// grid_dependency_wait before it touches memory.  What the kernel before may
// still be writing when this one starts is not constant for this one's
// lifetime, so it is read with ordinary loads, which stay behind the wait:
// a read-only load (__ldg, ld.global.nc) may be moved across it.
template <class... Params, class... Args>
int launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                     const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();   // returned here, not left for the next call that asks
  return (int)e;
}

// Services of the C-ABI translation unit: the current device's status word
// (checks the device), and a tensor map of a 16-bit tensor whose innermost
// dimension is contiguous (strides of the others in elements; 128-byte
// swizzle, rank <= 5).
int paged_device_status(uint32_t** status);
int encode_map_nd(CUtensorMap* m, const void* base, int rank, const long long* dims, const long long* strides,
                  const int* box, bool bf16);

}  // namespace fa2
