// fa2_paged_abi.cu -- the paged-cache entry points of include/fa2.h: argument
// checks, tensor maps and launches.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa2.h"
#include "fa2_internal.h"
#include "fa2_paged.h"

namespace fa2 {
namespace {

constexpr long long kMaxStride = 1ll << 39;   // elements: 16-bit strides stay below the TMA limit of 2^40 bytes

// Pieces the work is cut into: one wave of the resident CTAs of a GB300's 152
// SMs (two per SM, one at head dim 256).  Fixed, so that neither the workspace
// nor the result depends on the device.
constexpr int paged_ctas(int d) { return d == 256 ? 152 : 304; }
// A pair's fixed cost (Q, the first products, the epilogue) in keys, and the
// shortest piece worth a CTA: 128 keys, or (many rows) the keys whose K and V
// are twice as many bytes as a partial's write and read (100 tokens over 9000
// keys, d = 128: 28.4 us, with pieces twice as long 32.1, half as long 28.5;
// 8 drafted tokens x 8 heads, 4 requests of 2000 keys: 18.8, 21.0, 19.6; 60 over
// 32000 at d = 256, few pairs of many partials, 42.7, 40.2, 55.5).
constexpr int kPagedOverhead = 128;
constexpr int kPagedMinShare = 128;
constexpr int kPagedMaxHeads = 65536;
constexpr long long kPagedMaxKeys = (1ll << 31) - 4096;   // keys of a sequence, rounded up to tiles, stay below 2^31

struct Range {
  uintptr_t at;
  size_t bytes;
};

Range range(const void* p, size_t bytes) { return Range{reinterpret_cast<uintptr_t>(p), bytes}; }
bool overlap(const Range& a, const Range& b) { return a.at < b.at + b.bytes && b.at < a.at + a.bytes; }
bool misaligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Bytes a strided tensor can touch: dims[i] with strides st[i] (elements), and
// `inner` contiguous elements.
template <int N>
Range extent(const void* p, const long long (&dims)[N], const long long (&st)[N], long long inner, int elem) {
  long long last = inner - 1;
  for (int i = 0; i < N; ++i)
    if (dims[i] > 1) last += (dims[i] - 1) * st[i];
  return range(p, (size_t)(last + 1) * (size_t)elem);
}

// Strides of dimensions larger than 1: positive multiples of 8 elements.
template <int N>
int check_strides(const long long (&dims)[N], const long long (&st)[N]) {
  for (int i = 0; i < N; ++i) {
    if (dims[i] <= 1) continue;
    if (st[i] <= 0 || st[i] >= kMaxStride) return FA2_ERR_INVALID_ARG;
    if (st[i] & 7) return FA2_ERR_MISALIGNED;
  }
  return FA2_OK;
}

// One cache tensor: (pages, heads, rows).
struct CacheView {
  long long dims[3], st[3];
  Range bytes;
};

int check_cache(const fa2_paged_cache& c, CacheView& k, CacheView& v) {
  if (c.dtype != FA2_FP16 && c.dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  if (c.num_pages < 1 || c.heads < 1 || c.page_size < 1) return FA2_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return FA2_ERR_UNSUPPORTED;
  const int ps = c.page_size;
  if (!(ps == 8 || ps == 16 || ps == 32 || ps % 64 == 0)) return FA2_ERR_UNSUPPORTED;
  if ((long long)c.num_pages * ps > INT_MAX || c.heads > kPagedMaxHeads) return FA2_ERR_UNSUPPORTED;
  if (!c.k || !c.v) return FA2_ERR_INVALID_ARG;
  if (misaligned(c.k, 16) || misaligned(c.v, 16)) return FA2_ERR_MISALIGNED;
  CacheView* view[2] = {&k, &v};
  const int64_t* st[2] = {c.k_strides, c.v_strides};
  const void* at[2] = {c.k, c.v};
  for (int i = 0; i < 2; ++i) {
    CacheView& x = *view[i];
    x.dims[0] = c.num_pages;
    x.dims[1] = c.heads;
    x.dims[2] = ps;
    for (int j = 0; j < 3; ++j) x.st[j] = (long long)st[i][j];
    const int rc = check_strides(x.dims, x.st);
    if (rc) return rc;
    x.bytes = extent(at[i], x.dims, x.st, c.head_dim, 2);
  }
  return FA2_OK;
}

struct PagedShape {
  int group, tile_tokens, box_tokens, max_q;
  int ctas, pair_ctas;
  size_t ws_o_bytes, ws_ml_bytes, ws_bytes;   // ws_bytes: all, with the pairs to merge
};

// Sizes of a paged forward call that follow from what the host knows.
int paged_shape(const fa2_paged_params& a, PagedShape& s) {
  const fa2_paged_cache& c = a.cache;
  if (a.batch < 1 || a.heads < 1 || a.total_q < 1 || a.max_seqlen_q < 1 || a.max_pages < 1) return FA2_ERR_INVALID_ARG;
  if (c.heads < 1 || c.page_size < 1) return FA2_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return FA2_ERR_UNSUPPORTED;
  if (a.heads % c.heads) return FA2_ERR_INVALID_ARG;
  s.group = a.heads / c.heads;
  if (s.group > kPagedTileRows) return FA2_ERR_UNSUPPORTED;
  if ((long long)a.max_pages * c.page_size > kPagedMaxKeys) return FA2_ERR_UNSUPPORTED;
  s.max_q = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
  const long long T = s.tile_tokens = kPagedTileRows / s.group;
  s.box_tokens = (int)(T < s.max_q ? T : s.max_q);
  // whole and partial query tiles of sequences whose rows do not overlap
  long long tiles = ((long long)a.total_q + (T - 1) * a.batch) / T;
  const long long each = (s.max_q + T - 1) / T;
  if (tiles > a.batch * each) tiles = a.batch * each;
  if (tiles > a.total_q) tiles = a.total_q;
  const long long pairs = tiles * c.heads;
  if (pairs > INT_MAX - 1024) return FA2_ERR_UNSUPPORTED;
  s.ctas = paged_ctas(c.head_dim);
  s.pair_ctas = pairs >= s.ctas ? (int)pairs : 0;
  const size_t rows = 2 * (size_t)s.ctas * (size_t)(s.group * s.box_tokens);
  s.ws_o_bytes = align256(rows * (size_t)c.head_dim * 4);
  s.ws_ml_bytes = align256(rows * 2 * 4);
  s.ws_bytes = s.ws_o_bytes + s.ws_ml_bytes + align256((size_t)s.ctas * kPagedMergeBytes);
  return FA2_OK;
}

// Map of one cache tensor: a page's 8-row groups, with pages and heads as one
// coordinate where the page stride is a whole number of head strides (as in
// [pages, heads, rows, d] and [pages, rows, heads, d], also with K and V
// interleaved); otherwise pages and heads apart, in boxes of 8 rows.
bool merged_side(const CacheView& x, PagedSide& side) {
  const long long pages = x.dims[0], heads = x.dims[1];
  long long ratio = 1;
  if (pages > 1 && heads > 1) {
    if (x.st[0] % x.st[1]) return false;
    ratio = x.st[0] / x.st[1];
  }
  const long long extent = (pages - 1) * ratio + heads;
  if (extent > INT_MAX) return false;
  side.ratio = (int)ratio;
  side.extent = (int)extent;
  return true;
}

int cache_map(CUtensorMap* m, const void* at, const CacheView& x, const PagedSide& side, int d, int box_rows,
              bool bf16) {
  const long long rows = x.dims[2], rs = x.st[2];
  if (side.ratio > 0) {
    const long long dims[5] = {64, 8, d / 64, rows / 8, side.extent};
    const long long st[4] = {rs, 64, 8 * rs, x.dims[1] > 1 ? x.st[1] : x.st[0]};
    const int box[5] = {64, 8, d / 64, box_rows / 8, 1};
    return encode_map_nd(m, at, 5, dims, st, box, bf16);
  }
  const long long dims[5] = {64, rows, d / 64, x.dims[1], x.dims[0]};
  const long long st[4] = {rs, 64, x.st[1], x.st[0]};
  const int box[5] = {64, 8, d / 64, 1, 1};
  return encode_map_nd(m, at, 5, dims, st, box, bf16);
}

int paged_forward(const fa2_paged_params& a, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const fa2_paged_cache& c = a.cache;
  CacheView kc, vc;
  int rc = check_cache(c, kc, vc);
  if (rc) return rc;
  PagedShape s;
  rc = paged_shape(a, s);
  if (rc) return rc;
  if (!std::isfinite(a.scale)) return FA2_ERR_INVALID_ARG;
  if (a.window_left < -1 || a.window_right < -1 || a.prefix_len < 0 || a.sink_len < 0) return FA2_ERR_INVALID_ARG;
  if (!a.q || !a.o || !a.lse || !a.block_table || !a.cu_seqlens_q || !a.seqlens_k || !workspace)
    return FA2_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || misaligned(a.o, 16) || misaligned(a.lse, 4) || misaligned(a.block_table, 4) ||
      misaligned(a.cu_seqlens_q, 4) || misaligned(a.seqlens_k, 4) || misaligned(workspace, 256))
    return FA2_ERR_MISALIGNED;
  if (workspace_bytes < s.ws_bytes) return FA2_ERR_INVALID_ARG;
  const long long qd[2] = {a.total_q, a.heads};
  const long long qs[2] = {(long long)a.q_strides[0], (long long)a.q_strides[1]};
  const long long os[2] = {(long long)a.o_strides[0], (long long)a.o_strides[1]};
  rc = check_strides(qd, qs);
  if (rc) return rc;
  rc = check_strides(qd, os);
  if (rc) return rc;
  const long long td[1] = {a.batch}, ts[1] = {(long long)a.table_stride};
  if (a.batch > 1 && (ts[0] < 0 || ts[0] >= kMaxStride)) return FA2_ERR_INVALID_ARG;
  const long long ld[1] = {a.heads}, ls[1] = {(long long)a.lse_stride};
  if (a.heads > 1 && (ls[0] < a.total_q || ls[0] >= kMaxStride)) return FA2_ERR_INVALID_ARG;
  const Range out[3] = {extent(a.o, qd, os, c.head_dim, 2), extent(a.lse, ld, ls, a.total_q, 4),
                        range(workspace, s.ws_bytes)};
  const Range in[6] = {extent(a.q, qd, qs, c.head_dim, 2), kc.bytes, vc.bytes,
                       extent(a.block_table, td, ts, a.max_pages, 4),
                       range(a.cu_seqlens_q, ((size_t)a.batch + 1) * 4), range(a.seqlens_k, (size_t)a.batch * 4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FA2_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlap(out[i], r)) return FA2_ERR_INVALID_ARG;
  }

  PagedLaunchArgs la;
  std::memset(&la, 0, sizeof(la));
  PagedParams& p = la.p;
  rc = paged_device_status(&p.status);
  if (rc) return rc;
  la.bf16 = c.dtype == FA2_BF16;
  // q as (d, group, heads_kv, total_q): a box is `group` heads of box_tokens tokens
  {
    const long long dims[4] = {c.head_dim, s.group, c.heads, a.total_q};
    const long long st[3] = {qs[1], qs[1] * s.group, qs[0]};
    const int box[4] = {64, s.group, 1, s.box_tokens};
    rc = encode_map_nd(&la.tm_q, a.q, 4, dims, st, box, la.bf16);
    if (rc) return rc;
  }
  // k / page_size for 0 <= k < 2^31 without a division: magic = 2^32 (2^shift - page_size) / page_size + 1, 2^shift >=
  // page_size
  while ((1ll << p.page_shift) < c.page_size) ++p.page_shift;
  p.page_magic = (unsigned)(((1ull << 32) * ((1ull << p.page_shift) - (unsigned)c.page_size)) / (unsigned)c.page_size + 1);
  p.box_rows = c.page_size < kPagedKeyTile ? c.page_size : kPagedKeyTile;
  const bool merged_k = merged_side(kc, p.k_side), merged_v = merged_side(vc, p.v_side);
  if (!merged_k || !merged_v) p.box_rows = 8;
  rc = cache_map(&la.tm_k, c.k, kc, p.k_side, c.head_dim, p.box_rows, la.bf16);
  if (rc) return rc;
  rc = cache_map(&la.tm_v, c.v, vc, p.v_side, c.head_dim, p.box_rows, la.bf16);
  if (rc) return rc;
  p.o = a.o;
  p.lse = a.lse;
  p.table = a.block_table;
  p.cu_q = a.cu_seqlens_q;
  p.lens_k = a.seqlens_k;
  p.table_stride = ts[0];
  p.o_rs = os[0];
  p.o_hs = os[1];
  p.lse_hs = ls[0];
  p.batch = a.batch;
  p.heads_kv = c.heads;
  p.group = s.group;
  p.tile_tokens = s.tile_tokens;
  p.total_q = a.total_q;
  p.max_q = s.max_q;
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.max_keys = a.max_pages * c.page_size;
  p.window_left = a.window_left;
  p.window_right = a.window_right;
  p.prefix = a.prefix_len;
  p.sinks = a.window_left >= 0 ? a.sink_len : 0;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  p.scale_log2_mag = std::fmax(std::fabs(scale_log2), FLT_MIN);
  p.qk_negate = scale_log2 < 0.f ? 1u << 13 : 0u;   // the negate-A bit of the S product's descriptor
  p.slot_rows = s.group * s.box_tokens;
  p.overhead = (kPagedOverhead + 2 * p.slot_rows + 63) / 64 * 64;
  p.ctas = s.ctas;
  p.pair_ctas = s.pair_ctas;
  p.cached_keys = (96 << 20) / (4 * c.head_dim);   // 96 of the 126 MB
  p.min_share = kPagedMinShare > 4 * p.slot_rows ? kPagedMinShare : (4 * p.slot_rows + 63) / 64 * 64;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.ws_o_bytes);
  p.merges = reinterpret_cast<PagedMerge*>(static_cast<uint8_t*>(workspace) + s.ws_o_bytes + s.ws_ml_bytes);
  // few rows (every sequence is then one query tile): the line in key tiles and 32 bits
  la.wide = p.slot_rows > kPagedTileRows / 2 ||
            (double)a.batch * c.heads * ((p.max_keys + p.overhead) / 64 + 2.0) + 1e6 > 2147483647.0;
  p.merge_cost = la.wide ? 768 : 256;
  la.band = a.window_left >= 0 || a.prefix_len > 0;
  la.stream = stream;
  int e = 0;
  switch (c.head_dim) {
    case 64: e = launch_paged_d64(la); break;
    case 128: e = launch_paged_d128(la); break;
    default: e = launch_paged_d256(la); break;
  }
  return e == 0 ? FA2_OK : FA2_ERR_CUDA;
}

int paged_append(const fa2_paged_append_params& a, cudaStream_t stream) {
  const fa2_paged_cache& c = a.cache;
  CacheView kc, vc;
  int rc = check_cache(c, kc, vc);
  if (rc) return rc;
  if (a.total < 1 || !a.k || !a.v || !a.slots) return FA2_ERR_INVALID_ARG;
  if (misaligned(a.k, 16) || misaligned(a.v, 16) || misaligned(a.slots, 4)) return FA2_ERR_MISALIGNED;
  const long long nd[2] = {a.total, c.heads};
  const long long ks[2] = {(long long)a.k_strides[0], (long long)a.k_strides[1]};
  const long long vs[2] = {(long long)a.v_strides[0], (long long)a.v_strides[1]};
  rc = check_strides(nd, ks);
  if (rc) return rc;
  rc = check_strides(nd, vs);
  if (rc) return rc;
  if (c.k == c.v) return FA2_ERR_INVALID_ARG;   // the two may interleave in one allocation, not coincide
  const Range in[3] = {extent(a.k, nd, ks, c.head_dim, 2), extent(a.v, nd, vs, c.head_dim, 2),
                       range(a.slots, (size_t)a.total * 4)};
  for (const Range& r : in)
    if (overlap(r, kc.bytes) || overlap(r, vc.bytes)) return FA2_ERR_INVALID_ARG;
  PagedAppendArgs la;
  std::memset(&la, 0, sizeof(la));
  rc = paged_device_status(&la.status);
  if (rc) return rc;
  la.k = PagedAppendSide{static_cast<const uint4*>(a.k), static_cast<uint4*>(c.k), ks[0] / 8, ks[1] / 8, kc.st[0] / 8,
                         kc.st[1] / 8, kc.st[2] / 8};
  la.v = PagedAppendSide{static_cast<const uint4*>(a.v), static_cast<uint4*>(c.v), vs[0] / 8, vs[1] / 8, vc.st[0] / 8,
                         vc.st[1] / 8, vc.st[2] / 8};
  la.slots = a.slots;
  la.total = a.total;
  la.heads = c.heads;
  la.num_slots = c.num_pages * c.page_size;
  la.page_size = c.page_size;
  la.row_chunks_log2 = c.head_dim == 64 ? 3 : c.head_dim == 128 ? 4 : 5;
  return launch_paged_append(la, stream) == 0 ? FA2_OK : FA2_ERR_CUDA;
}

int paged_plan(const fa2_paged_plan_params& a, cudaStream_t stream) {
  if (a.batch < 1 || a.max_pages < 1 || a.num_pages < 1 || a.page_size < 1 || a.total_q < 1 || a.num_free < 0)
    return FA2_ERR_INVALID_ARG;
  if (a.batch > FA2_PAGED_PLAN_MAX_BATCH) return FA2_ERR_UNSUPPORTED;
  if ((long long)a.num_pages * a.page_size > INT_MAX || (long long)a.max_pages * a.page_size > kPagedMaxKeys)
    return FA2_ERR_UNSUPPORTED;
  if (!a.free_pages && a.num_free > 0) return FA2_ERR_INVALID_ARG;
  const void* all[8] = {a.context_lens, a.query_lens, a.free_count, a.block_table,
                        a.cu_seqlens_q, a.seqlens_k, a.slots, a.free_left};
  if (misaligned(a.free_pages, 4)) return FA2_ERR_MISALIGNED;
  for (const void* p : all) {
    if (!p) return FA2_ERR_INVALID_ARG;
    if (misaligned(p, 4)) return FA2_ERR_MISALIGNED;
  }
  if (a.batch > 1 && (a.table_stride < a.max_pages || a.table_stride >= kMaxStride)) return FA2_ERR_INVALID_ARG;
  const size_t B = (size_t)a.batch;
  const long long td[1] = {a.batch}, ts[1] = {(long long)a.table_stride};
  const Range in[4] = {range(a.context_lens, B * 4), range(a.query_lens, B * 4),
                       range(a.free_pages, (size_t)a.num_free * 4), range(a.free_count, 4)};
  const Range out[5] = {extent(a.block_table, td, ts, a.max_pages, 4), range(a.cu_seqlens_q, (B + 1) * 4),
                        range(a.seqlens_k, B * 4), range(a.slots, (size_t)a.total_q * 4), range(a.free_left, 4)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FA2_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlap(out[i], r)) return FA2_ERR_INVALID_ARG;
  }
  PagedPlanArgs la;
  std::memset(&la, 0, sizeof(la));
  const int rc = paged_device_status(&la.status);
  if (rc) return rc;
  la.context_lens = a.context_lens;
  la.query_lens = a.query_lens;
  la.free_pages = a.free_pages;
  la.free_count = a.free_count;
  la.table = a.block_table;
  la.cu_q = a.cu_seqlens_q;
  la.lens_k = a.seqlens_k;
  la.slots = a.slots;
  la.free_left = a.free_left;
  la.table_stride = a.table_stride;
  la.batch = a.batch;
  la.max_pages = a.max_pages;
  la.num_pages = a.num_pages;
  la.page_size = a.page_size;
  la.total_q = a.total_q;
  la.num_free = a.num_free;
  return launch_paged_plan(la, stream) == 0 ? FA2_OK : FA2_ERR_CUDA;
}

static_assert(kPagedPlanMaxBatch == FA2_PAGED_PLAN_MAX_BATCH, "plan batch limit");

}  // namespace
}  // namespace fa2

using namespace fa2;

extern "C" size_t fa2_paged_params_size(void) { return sizeof(fa2_paged_params); }

extern "C" size_t fa2_paged_fwd_workspace_bytes(const fa2_paged_params* params) {
  if (!params) return 0;
  PagedShape s;
  if (paged_shape(*params, s)) return 0;
  return s.ws_bytes;
}

extern "C" int fa2_paged_fwd(const fa2_paged_params* params, void* workspace, size_t workspace_bytes, void* stream) {
  if (!params) return FA2_ERR_INVALID_ARG;
  return paged_forward(*params, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int fa2_paged_append(const fa2_paged_append_params* params, void* stream) {
  if (!params) return FA2_ERR_INVALID_ARG;
  return paged_append(*params, static_cast<cudaStream_t>(stream));
}

extern "C" int fa2_paged_plan(const fa2_paged_plan_params* params, void* stream) {
  if (!params) return FA2_ERR_INVALID_ARG;
  return paged_plan(*params, static_cast<cudaStream_t>(stream));
}
