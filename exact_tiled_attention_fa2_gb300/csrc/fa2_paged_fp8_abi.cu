// fa2_paged_fp8_abi.cu -- the entry points of include/fa2.h on a paged cache of
// 8-bit rows: argument checks, tensor maps and launches.
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/fa2.h"
#include "fa2_internal.h"
#include "fa2_paged_check.h"
#include "fa2_paged_fp8.h"

namespace fa2 {
namespace {

// In keys: a pair's fixed cost with up to eight rows (32 requests of 1 .. 8192 keys,
// d = 128: 55.7 us at 128, 54.4, 54.7 at 384; one of 600: 13.2, 10.8, 11.5) and with
// more (8 tokens over 16384 keys: 28.0 at 256, 22.6, 22.5 at 512; 16 requests of one
// token, 16 rows, over 1000 .. 3000 keys: 28.5, 26.5, 27.6; windows of 1023 at d =
// 256: 28.8, 28.8, 40.4), the shortest piece worth a CTA (128 and 384 within 0.2 us
// of 256, but the 600 keys 13.4 at 384) and what a merge may cost before pairs are
// left whole (the windows 41.8 us at 256, 28.8, 28.8 at 1024; the 600 keys 13.4 there).
constexpr int kFp8Overhead = 256;
constexpr int kFp8OverheadMore = 384;
constexpr int kFp8MinShare = 256;
constexpr int kFp8MergeCost = 512;

struct Fp8View {
  CacheView code[2];
  long long exp_st[2][2];
  Range bytes[4];   // codes of k and v, their exponents
};

int check_cache(const fa2_paged_cache_fp8& c, Fp8View& x) {
  if (c.num_pages < 1 || c.heads < 1 || c.page_size < 1) return FA2_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return FA2_ERR_UNSUPPORTED;
  const int ps = c.page_size;
  if (!(ps == 8 || ps == 16 || ps == 32 || ps % 64 == 0)) return FA2_ERR_UNSUPPORTED;
  if ((long long)c.num_pages * ps > INT_MAX || c.heads > kPagedMaxHeads) return FA2_ERR_UNSUPPORTED;
  const void* code[2] = {c.k, c.v};
  const void* exps[2] = {c.k_exps, c.v_exps};
  const int64_t* st[2] = {c.k_strides, c.v_strides};
  const int64_t* est[2] = {c.k_exp_strides, c.v_exp_strides};
  for (int i = 0; i < 2; ++i) {
    if (!code[i] || !exps[i]) return FA2_ERR_INVALID_ARG;
    if (misaligned(code[i], 16) || misaligned(exps[i], 8)) return FA2_ERR_MISALIGNED;
  }
  for (int i = 0; i < 2; ++i) {
    CacheView& v = x.code[i];
    v.dims[0] = c.num_pages;
    v.dims[1] = c.heads;
    v.dims[2] = ps;
    for (int j = 0; j < 3; ++j) v.st[j] = (long long)st[i][j];
    int rc = check_strides(v.dims, v.st, 16);
    if (rc) return rc;
    x.bytes[i] = v.bytes = extent(code[i], v.dims, v.st, c.head_dim, 1);
    const long long ed[2] = {c.num_pages, c.heads};
    for (int j = 0; j < 2; ++j) x.exp_st[i][j] = (long long)est[i][j];
    rc = check_strides(ed, x.exp_st[i], 8);
    if (rc) return rc;
    x.bytes[2 + i] = extent(exps[i], ed, x.exp_st[i], ps, 1);
  }
  return FA2_OK;
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

// k / page_size for 0 <= k < 2^31 without a division (see the 16-bit forward).
void page_division(int page_size, unsigned& magic, unsigned& shift) {
  shift = (unsigned)log2_of(page_size);
  magic = (unsigned)(((1ull << 32) * ((1ull << shift) - (unsigned)page_size)) / (unsigned)page_size + 1);
}

// The launch of fa2_paged_append_fp8 (write: the cache is written) or fa2_paged_read_fp8.
int fp8_rows(const fa2_paged_cache_fp8& c, void* k, void* v, const int* slots, const int64_t* k_st, const int64_t* v_st,
             int total, int dtype, bool write, cudaStream_t stream) {
  Fp8View x;
  int rc = check_cache(c, x);
  if (rc) return rc;
  if (dtype != FA2_FP16 && dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  if (total < 1 || !k || !v || !slots) return FA2_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 4)) return FA2_ERR_MISALIGNED;
  const long long nd[2] = {total, c.heads};
  const long long ks[2] = {(long long)k_st[0], (long long)k_st[1]};
  const long long vs[2] = {(long long)v_st[0], (long long)v_st[1]};
  rc = check_strides(nd, ks);
  if (rc) return rc;
  rc = check_strides(nd, vs);
  if (rc) return rc;
  // what is written may interleave in one allocation, not coincide
  if (write ? c.k == c.v || c.k_exps == c.v_exps || c.k == c.k_exps || c.k == c.v_exps || c.v == c.k_exps || c.v == c.v_exps
            : k == v)
    return FA2_ERR_INVALID_ARG;
  const Range rows[2] = {extent(k, nd, ks, c.head_dim, 2), extent(v, nd, vs, c.head_dim, 2)};
  const Range slot = range(slots, (size_t)total * 4);
  for (const Range& b : x.bytes)
    for (const Range& r : rows)
      if (overlap(r, b)) return FA2_ERR_INVALID_ARG;
  for (const Range& b : x.bytes)
    if (write && overlap(slot, b)) return FA2_ERR_INVALID_ARG;
  for (const Range& r : rows)
    if (!write && overlap(slot, r)) return FA2_ERR_INVALID_ARG;
  PagedFp8RowsArgs a;
  std::memset(&a, 0, sizeof(a));
  rc = paged_device_status(&a.status);
  if (rc) return rc;
  auto side = [&](int i, void* row, const long long* st, void* code, void* exps) {
    return PagedFp8Side{static_cast<uint4*>(row), static_cast<uint2*>(code), static_cast<uint8_t*>(exps),
                        st[0] / 8, st[1] / 8, x.code[i].st[0] / 8, x.code[i].st[1] / 8, x.code[i].st[2] / 8,
                        x.exp_st[i][0], x.exp_st[i][1]};
  };
  a.k = side(0, k, ks, c.k, c.k_exps);
  a.v = side(1, v, vs, c.v, c.v_exps);
  a.slots = slots;
  a.total = total;
  a.heads = c.heads;
  a.num_slots = c.num_pages * c.page_size;
  a.page_size = c.page_size;
  a.head_dim = c.head_dim;
  page_division(c.page_size, a.page_magic, a.page_shift);
  a.bf16 = dtype == FA2_BF16;
  return (write ? launch_paged_append_fp8(a, stream) : launch_paged_read_fp8(a, stream)) == 0 ? FA2_OK : FA2_ERR_CUDA;
}

struct Fp8Shape {
  int group, parts, tile_tokens, box_tokens, max_q, slot_rows, overhead;
  int ctas;
  size_t ws_o_bytes, ws_ml_bytes, ws_bytes;
  bool many;
};

int fp8_shape(const fa2_paged_fp8_params& a, Fp8Shape& s) {
  const fa2_paged_cache_fp8& c = a.cache;
  if (a.batch < 1 || a.heads < 1 || a.total_q < 1 || a.max_seqlen_q < 1 || a.max_pages < 1) return FA2_ERR_INVALID_ARG;
  if (c.heads < 1 || c.page_size < 1) return FA2_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return FA2_ERR_UNSUPPORTED;
  if (a.heads % c.heads) return FA2_ERR_INVALID_ARG;
  const int all = a.heads / c.heads;
  if (all > kPagedTileRows) return FA2_ERR_UNSUPPORTED;
  if ((long long)a.max_pages * c.page_size > kPagedMaxKeys) return FA2_ERR_UNSUPPORTED;
  // a K/V head's query heads in as few equal parts as fit a tile
  s.parts = 1;
  while (all % s.parts || all / s.parts > kPagedFp8Rows) ++s.parts;
  s.group = all / s.parts;
  s.max_q = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
  const long long T = s.tile_tokens = kPagedFp8Rows / s.group;
  s.box_tokens = (int)(T < s.max_q ? T : s.max_q);
  s.slot_rows = s.group * s.box_tokens;
  s.overhead = s.slot_rows > 8 ? kFp8OverheadMore : kFp8Overhead;
  // whole and partial query tiles of sequences whose rows do not overlap
  long long tiles = ((long long)a.total_q + (T - 1) * a.batch) / T;
  const long long each = (s.max_q + T - 1) / T;
  if (tiles > a.batch * each) tiles = a.batch * each;
  if (tiles > a.total_q) tiles = a.total_q;
  const long long pairs = tiles * c.heads * s.parts;
  if (pairs > INT_MAX - 1024 || (long long)c.heads * s.parts > INT_MAX) return FA2_ERR_UNSUPPORTED;
  s.many = s.max_q > T || (double)a.batch * c.heads * s.parts *
                                  (((double)a.max_pages * c.page_size + s.overhead) / 64 + 2.0) + 1e6 > 2147483647.0;
  // One wave of the resident CTAs of a GB300's 152 SMs, fixed (see paged_ctas): two
  // an SM with up to eight rows (32 requests of 1 .. 8192 keys: 70 us, with one CTA
  // and deeper rings 88, from an empty L2 cache), one with more (16 requests of 8192
  // keys, 16 rows, as then built: 80 us, with two CTAs 90; now 74)
  s.ctas = c.head_dim == 256 || s.many || s.slot_rows > 8 ? 152 : 304;
  const size_t rows = 2 * (size_t)s.ctas * (size_t)s.slot_rows;
  s.ws_o_bytes = align256(rows * (size_t)c.head_dim * 4);
  s.ws_ml_bytes = align256(rows * 2 * 4);
  s.ws_bytes = s.ws_o_bytes + s.ws_ml_bytes + align256((size_t)s.ctas * kPagedMergeBytes);
  return FA2_OK;
}

// As the 16-bit cache's: pages and heads as one coordinate where they can be.
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

// A 5-D map of bytes (64- or 128-byte swizzle, as the box's rows; as encode_map_nd).
int encode_map_u8(CUtensorMap* m, const void* base, const long long* dims, const long long* strides, const int* box) {
  static std::atomic<void*> found{nullptr};   // the driver's entry point
  void* fn = found.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return FA2_ERR_CUDA;
    found.store(fn, std::memory_order_release);
  }
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], estr[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < 5; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
  }
  for (int i = 0; i < 4; ++i) st[i] = (cuuint64_t)(dims[i + 1] > 1 ? strides[i] : dims[0]);
  const CUresult r = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
      m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), d, st, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
      box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

int cache_map(CUtensorMap* m, const void* at, const CacheView& x, const PagedSide& side, int d, int box_rows) {
  const long long rows = x.dims[2], rs = x.st[2], row = d < 128 ? d : 128;
  if (side.ratio > 0) {
    const long long dims[5] = {row, 8, d / row, rows / 8, side.extent};
    const long long st[4] = {rs, row, 8 * rs, x.dims[1] > 1 ? x.st[1] : x.st[0]};
    const int box[5] = {(int)row, 8, (int)(d / row), box_rows / 8, 1};
    return encode_map_u8(m, at, dims, st, box);
  }
  const long long dims[5] = {row, rows, d / row, x.dims[1], x.dims[0]};
  const long long st[4] = {rs, row, x.st[1], x.st[0]};
  const int box[5] = {(int)row, 8, (int)(d / row), 1, 1};
  return encode_map_u8(m, at, dims, st, box);
}

int fp8_forward(const fa2_paged_fp8_params& a, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const fa2_paged_cache_fp8& c = a.cache;
  Fp8View x;
  int rc = check_cache(c, x);
  if (rc) return rc;
  if (a.dtype != FA2_FP16 && a.dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  Fp8Shape s;
  rc = fp8_shape(a, s);
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
  const Range in[8] = {extent(a.q, qd, qs, c.head_dim, 2), x.bytes[0], x.bytes[1], x.bytes[2], x.bytes[3],
                       extent(a.block_table, td, ts, a.max_pages, 4),
                       range(a.cu_seqlens_q, ((size_t)a.batch + 1) * 4), range(a.seqlens_k, (size_t)a.batch * 4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FA2_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlap(out[i], r)) return FA2_ERR_INVALID_ARG;
  }

  PagedFp8LaunchArgs la;
  std::memset(&la, 0, sizeof(la));
  PagedFp8Params& f = la.a;
  PagedParams& p = f.p;
  rc = paged_device_status(&p.status);
  if (rc) return rc;
  page_division(c.page_size, p.page_magic, p.page_shift);
  p.box_rows = c.page_size < kPagedKeyTile ? c.page_size : kPagedKeyTile;
  const bool merged_k = merged_side(x.code[0], p.k_side), merged_v = merged_side(x.code[1], p.v_side);
  if (!merged_k || !merged_v) p.box_rows = 8;
  rc = cache_map(&la.tm_k, c.k, x.code[0], p.k_side, c.head_dim, p.box_rows);
  if (rc) return rc;
  rc = cache_map(&la.tm_v, c.v, x.code[1], p.v_side, c.head_dim, p.box_rows);
  if (rc) return rc;
  f.q = a.q;
  f.q_rs = qs[0];
  f.q_hs = qs[1];
  f.k_exps = static_cast<const uint8_t*>(c.k_exps);
  f.v_exps = static_cast<const uint8_t*>(c.v_exps);
  f.k_exp_ps = x.exp_st[0][0];
  f.k_exp_hs = x.exp_st[0][1];
  f.v_exp_ps = x.exp_st[1][0];
  f.v_exp_hs = x.exp_st[1][1];
  f.parts = s.parts;
  f.scale_log2 = a.scale * 1.4426950408889634f;
  f.bf16 = a.dtype == FA2_BF16;
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
  p.heads_kv = c.heads * s.parts;
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
  p.slot_rows = s.slot_rows;
  p.overhead = s.overhead;
  p.ctas = s.ctas;
  p.pair_ctas = 0;   // (never a CTA a pair)
  p.min_share = kFp8MinShare;
  p.merge_cost = kFp8MergeCost;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.ws_o_bytes);
  p.merges = reinterpret_cast<PagedMerge*>(static_cast<uint8_t*>(workspace) + s.ws_o_bytes + s.ws_ml_bytes);
  la.many = s.many;
  la.stream = stream;
  int e = 0;
  switch (c.head_dim) {
    case 64: e = launch_paged_fp8_d64(la); break;
    case 128: e = launch_paged_fp8_d128(la); break;
    default: e = launch_paged_fp8_d256(la); break;
  }
  return e == 0 ? FA2_OK : FA2_ERR_CUDA;
}

}  // namespace
}  // namespace fa2

using namespace fa2;

extern "C" int fa2_paged_append_fp8(const fa2_paged_append_fp8_params* a, void* stream) {
  if (!a) return FA2_ERR_INVALID_ARG;
  return fp8_rows(a->cache, const_cast<void*>(a->k), const_cast<void*>(a->v), a->slots, a->k_strides, a->v_strides, a->total,
                  a->dtype, true, static_cast<cudaStream_t>(stream));
}

extern "C" int fa2_paged_read_fp8(const fa2_paged_read_fp8_params* a, void* stream) {
  if (!a) return FA2_ERR_INVALID_ARG;
  return fp8_rows(a->cache, a->k, a->v, a->slots, a->k_strides, a->v_strides, a->total, a->dtype, false,
                  static_cast<cudaStream_t>(stream));
}

extern "C" size_t fa2_paged_fp8_params_size(void) { return sizeof(fa2_paged_fp8_params); }

extern "C" size_t fa2_paged_fwd_fp8_workspace_bytes(const fa2_paged_fp8_params* params) {
  if (!params) return 0;
  Fp8Shape s;
  if (fp8_shape(*params, s)) return 0;
  return s.ws_bytes;
}

extern "C" int fa2_paged_fwd_fp8(const fa2_paged_fp8_params* params, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!params) return FA2_ERR_INVALID_ARG;
  return fp8_forward(*params, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
