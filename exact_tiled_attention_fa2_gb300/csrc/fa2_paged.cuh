// fa2_paged.cuh -- attention of each sequence's new query tokens over a paged
// key/value cache with grouped query heads.
//
// S = scale Q K^T, O = softmax(S) V, L = ln sum exp S per query row, with the
// general forward's masks (KeyMask); key j of K/V head h of sequence b is row
// j % page_size of page table[b][j / page_size].
//
// One query tile is 128 / group tokens of one K/V head with all `group` query
// heads that share it, so a tile's K and V are read once for the whole group:
// a decoding step's tile has `group` rows and is bound by reading K and V
// (4 d bytes a key), a prompt chunk's has up to 128 and is bound by the tensor
// cores.  Row r of the tile is token r / group, query head h * group +
// r % group, the order in which a TMA box (64 columns x group x tokens) lands.
//
// Schedule.  The lengths are on the device, so the CTAs lay the batch's work
// out themselves: every (query tile, K/V head) pair is a span of keys, the
// spans of all pairs make one line, and each of the p.ctas CTAs (two per SM,
// one at d = 256) takes an equal piece of it, whatever the lengths are.  A
// piece is a run of fragments: the end of one pair, whole pairs, the start of
// another.  Whole pairs write O and L; the others leave fp32 partials (m, l,
// O~) in the CTA's two slots, which a second kernel, launched as a programmatic
// dependent, merges.  Where cutting gains less than it costs (whole_pairs), all
// pairs, or a batch's full waves of them, run one per CTA instead.
//
// One CTA, 192 threads (224 with query tiles of few rows), as the
// double-buffered forward kernel (fa2_fwd_dbuf.cuh: tensor-memory layout, two S
// buffers, rings of K and V stages, one softmax thread per row), with the
// rings' and barriers' phases counted across its fragments: while the softmax
// warps finish a fragment, the TMA warp already loads the next one's K, V and Q
// and the MMA thread issues its first S products.
//
// A 64-key tile lands as [8-row group][64-column block][8 rows][128 bytes]
// (128-byte swizzle), so that rows of any page size follow each other with one
// stride: one 5-D box per page and tile (pages of 8 .. 32 rows: 8 .. 2 boxes, of
// 64 k rows: one), issued by one lane of the TMA warp per page, which reads
// its page from the block table four tiles ahead.  Pages none of the tile's
// rows see are not loaded, and key tiles between a prefix and the band are not
// visited.  V rows no row of the tile sees (the last page's tail, keys before
// a window) may hold anything: they are zeroed in shared memory before the
// product, since 0 x NaN would reach the sums.
#pragma once

#include <climits>

#include "fa2_fwd_dbuf.cuh"
#include "fa2_paged.h"

namespace fa2 {

// Barriers (8 bytes each).  Phases count key tiles g (K, V, S, P, O) or
// fragments f of the CTA (the others).  One completion tells all who wait for
// it: S(g) the softmax warps (scores there) and the TMA warp (K stage free),
// PV(g) the TMA warp (V stage free) and the softmax warps (O~ may be rescaled
// or read); none of them can fall a whole round of stages behind.
enum : int {
  PG_Q = 0,        // + f & 1: the fragment's description and Q are in shared memory
  PG_QEMPTY = 2,   // + f & 1: the fragment's last S product is done with Q
  PG_P = 4,        // + buffer (four softmax warps)
  PG_ODONE = 6,    // + f & 1: the softmax warps are done with O~ and the description
  PG_EXIT = 8,
  PG_S = 9,        // + K stage: S(g) complete
  PG_O = 13,       // + V stage: PV(g) complete
  PG_KFULL = 17,   // + stage
  PG_VFULL = 21,   // + stage
  PG_PLAN = 25,    // + f & 3: the fragment's description is there (planner -> TMA warp)
  PG_FREE = 29,    // + f & 3: its slot is free (softmax warps -> planner)
  PG_BARS = 33,
};

// Everything the softmax warps and the MMA thread need of a fragment: written
// by the TMA warp, in a ring of four.
struct PagedFrag {
  const int* table;   // the sequence's block-table row
  int n;           // key tiles (0: the pair has no visible key; -1: no more fragments)
  int j0;          // first of them, as a visited index of the pair
  int row;         // first token's row of q / o / lse
  int q0;          // first token within its sequence
  int rows;        // live rows: group x tokens
  int h;           // K/V head
  int slot;        // partial slot, or -1: write O and L
  int split;       // every bf16 P is split (else the masked tiles')
  TileMask tm;     // key tiles every row sees, by index from j0
  KeyMask km;      // with the last row's pre_end
  int npre, skip;  // visited index j is key tile j + (j >= npre ? skip : 0)
  int lo, end;     // the band's keys (the prefix's: km.pre_end)
  __device__ __forceinline__ int tile(int j) const { return j + (j >= npre ? skip : 0); }
};

// WIDE: query tiles of more than 64 rows (p.slot_rows).
template <int D_, bool WIDE_>
struct PagedConfig {
  static constexpr int D = D_;
  static constexpr bool WIDE = WIDE_;
  static constexpr int BR = kPagedTileRows;
  static constexpr int BC = kPagedKeyTile;
  static constexpr int KSTAGES = D == 64 ? 4 : 2;
  static constexpr int VSTAGES = D == 64 ? 4 : 2;
  // Few rows: a warp of its own walks the fragments (many short ones).  Many
  // rows: the TMA warp does, between loads.
  static constexpr bool PLANNER = !WIDE;
  static constexpr int THREADS = PLANNER ? 224 : 192;
  static constexpr int MMA_WARP = 4;
  static constexpr int TMA_WARP = 5;
  static constexpr int PLAN_WARP = 6;
  static constexpr int BLOCKS = D / 64;                 // 64-column blocks of a row
  static constexpr uint32_t GROUP_BYTES = BLOCKS * 1024;   // 8 key rows
  static constexpr uint32_t Q_BYTES = BR * D * 2;
  static constexpr uint32_t KV_BYTES = BC * D * 2;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + Q_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + KSTAGES * KV_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_V + VSTAGES * KV_BYTES;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (PG_BARS + 1) / 2 * 16;   // TMEM address, abort flag
  static constexpr uint32_t OFF_FRAG = OFF_MISC + 16;
  static constexpr uint32_t OFF_SCAN = OFF_FRAG + 512;
  static constexpr uint32_t SMEM_BYTES = OFF_SCAN + 320 + 1024;
  static constexpr uint32_t TMEM_S = 0;   // + 64 * buffer
  static constexpr uint32_t TMEM_O = 128;
  static constexpr uint32_t TMEM_COLS = D == 256 ? 512 : 256;
  static constexpr int CTAS_PER_SM = D == 256 ? 1 : 2;
  static_assert(4 * sizeof(PagedFrag) <= 512, "fragment descriptions");
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 233472, "shared memory per SM");
};

// ---------------------------------------------------------------- the line of work

// The key tiles a query tile visits (PagedFrag::tile), and its band's keys.
struct TileWalk {
  int npre, skip, n;
  int lo, end;
};

__device__ __forceinline__ TileWalk tile_walk(const KeyMask& km, int first, int last) {
  TileWalk w;
  w.lo = km.row_lo(first);
  w.end = km.row_hi(last) + 1;
  const int tp = (km.pre_end + kPagedKeyTile - 1) / kPagedKeyTile;
  const int t0 = w.lo / kPagedKeyTile, t1 = (w.end + kPagedKeyTile - 1) / kPagedKeyTile;
  if (w.end <= w.lo) {   // no band keys
    w.lo = w.end = 0;
    w.npre = tp;
    w.skip = 0;
    w.n = tp;
  } else if (t0 <= tp) {   // one run of tiles, from 0 under a prefix
    w.npre = 0;
    w.skip = tp > 0 ? 0 : t0;
    w.n = max(tp, t1) - w.skip;
  } else {
    w.npre = tp;
    w.skip = t0 - tp;
    w.n = tp + t1 - t0;
  }
  return w;
}

// The end of the keys [0, end) that row `row` sees beside its band: the prefix
// and, as far as the band's right edge, the sinks.  It does not fall from row to
// row, so what some row of a tile sees ends with its last row's, what all see
// with its first row's.
__device__ __forceinline__ int prefix_end(const PagedParams& p, const KeyMask& km, int row) {
  const int prefix = min(p.prefix, km.n_k);
  return p.sinks > 0 ? max(prefix, min(p.sinks, km.row_hi(row) + 1)) : prefix;
}

// The mask whose pre_end is that of row `row`.
__device__ __forceinline__ KeyMask paged_mask(const PagedParams& p, int n_q, int n_k, int row) {
  KeyMask km;
  km.n_k = n_k;
  km.off = n_k - n_q;
  km.wl = p.window_left;
  km.wr = p.window_right;
  km.pre_end = prefix_end(p, km, row);
  return km;
}

// Positions on the line: keys, in 64 bits; with tiles of few rows (WIDE false,
// and every sequence one query tile) key tiles, in 32 bits, which the host has
// made sure of.
template <bool WIDE>
struct LineOf {
  using T = long long;
  static constexpr int KEYS = 1;   // of a unit
};
template <>
struct LineOf<false> {
  using T = int;
  static constexpr int KEYS = kPagedKeyTile;
};

// a / b for 0 <= a, 0 < b: a 32-bit division where both fit.
__device__ __forceinline__ long long line_div(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}
__device__ __forceinline__ int line_div(int a, int b) { return (int)((unsigned)a / (unsigned)b); }

// One sequence's part of the line: `tiles` query tiles x heads_kv pairs, in
// order of the tiles, heads fastest.
struct PagedSeq {
  int row0, n_q, n_k;
  int tiles;
  int keys;      // a pair's span in keys, or -1: a causal chunk, whose spans
                 // grow by tile_tokens from tile to tile and end at N_k
  template <bool WIDE>
  __device__ __forceinline__ int width(const PagedParams& p, int t) const {
    if constexpr (WIDE)
      return p.overhead + (keys >= 0 ? keys : n_k - n_q + min((t + 1) * p.tile_tokens, n_q));
    else
      return (p.overhead + keys) / kPagedKeyTile;
  }
  // spans of the tiles before t (one head's)
  __device__ __forceinline__ long long before(const PagedParams& p, int t) const {
    return keys >= 0 ? (long long)t * (p.overhead + keys)
                     : (long long)t * (p.overhead + n_k - n_q) + (long long)p.tile_tokens * t * (t + 1) / 2;
  }
  // and of the first t tiles, all heads
  template <bool WIDE>
  __device__ __forceinline__ typename LineOf<WIDE>::T span(const PagedParams& p, int t) const {
    if (t == 0) return 0;
    if constexpr (WIDE)
      return (before(p, t - 1) + width<true>(p, t - 1)) * p.heads_kv;
    else
      return width<false>(p, 0) * p.heads_kv;
  }
};

// The sequence of query rows [a, b) and k keys; no tiles (and the bad-offsets
// bit, if `report`) when these are out of range.
template <bool WIDE>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int a, int b, int k, bool report) {
  PagedSeq s;
  s.row0 = a;
  s.n_q = b - a;
  s.n_k = k;
  s.tiles = 0;
  s.keys = 0;
  if (!(0 <= a && a <= b && b <= p.total_q && b - a <= p.max_q && 0 <= k && k <= p.max_keys)) {
    if (report) atomicOr(p.status, kStatusBadSeqlens);
    return s;
  }
  if (s.n_q == 0) return s;
  const KeyMask km = paged_mask(p, s.n_q, s.n_k, s.n_q - 1);
  s.tiles = 1;
  int nv;   // most key tiles one of the query tiles visits
  if constexpr (WIDE) {
    s.tiles = (s.n_q + p.tile_tokens - 1) / p.tile_tokens;
    if (s.tiles > 1 && p.window_left < 0 && p.window_right == 0 && km.off + p.tile_tokens >= max(km.pre_end, 1)) {
      s.keys = -1;
      return s;
    }
    if (s.tiles > 1 && p.window_left >= 0) {
      const long long band = (long long)p.window_left + (p.window_right < 0 ? s.n_k : p.window_right) + p.tile_tokens;
      const long long all = (s.n_k + kPagedKeyTile - 1) / kPagedKeyTile;
      const long long n = (km.pre_end + kPagedKeyTile - 1) / kPagedKeyTile + band / kPagedKeyTile + 2;
      nv = (int)(n < all ? n : all);
    } else {   // without a left window the last tile visits the most
      nv = tile_walk(km, (s.tiles - 1) * p.tile_tokens, s.n_q - 1).n;
    }
  } else {
    nv = tile_walk(km, 0, s.n_q - 1).n;
  }
  s.keys = max(nv, 1) * kPagedKeyTile;
  return s;
}

template <bool WIDE>
static __device__ __noinline__ PagedSeq read_seq(const PagedParams& p, int i, bool report) {
  return paged_seq<WIDE>(p, p.cu_q[i], p.cu_q[i + 1], p.lens_k[i], report);
}

// What a CTA works on.
template <bool WIDE>
struct PagedPlace {
  typename LineOf<WIDE>::T at;      // the sequence's start on the line
  typename LineOf<WIDE>::T share;   // a piece; 0: this CTA has one pair, whole
  typename LineOf<WIDE>::T total;   // the line's length
  PagedSeq s;        // the sequence that holds the piece's start (the pair)
  int seq;           // its index, or -1: nothing to do
  int piece;         // of the line
  int rank;          // one pair: its index in its sequence
  bool line;         // the line is cut at this CTA's piece, or ends before it (one pair: false)
};

template <bool WIDE>
struct PagedScan {
  typename LineOf<WIDE>::T warp_sum[3][8];
  int warp_longest[8];
  // the first pairs run whole, `whole` of them; the line holds the rest: of
  // sequence cut_seq the first cut_tiles query tiles, and the sequences after it
  int whole, cut_seq, cut_tiles;
  typename LineOf<WIDE>::T shift;   // positions of the sequences after it lie this much lower
  PagedPlace<WIDE> place;
};

// How many pairs, in order (sequences, their query tiles from the last, heads
// fastest), run whole, one per CTA, before the rest goes on the line: all,
// where cutting pairs gains less than it costs to merge them; none; or the
// full waves of a batch of long pairs, whose CTAs then walk the same keys
// together (on the line they would not, and K and V past the L2 cache would be
// read again for each: chunk of 2048 over 62048 keys, 1878 us all on the line,
// 1618 us so; of 2048 over 16048 keys, which stay in L2, 389 and 430 us).
// `spans`: the line's length were all on it; `chunk_keys`: keys of the
// sequences of several query tiles, all K/V heads.
template <bool WIDE>
__device__ __forceinline__ int whole_pairs(const PagedParams& p, typename LineOf<WIDE>::T spans,
                                           typename LineOf<WIDE>::T chunk_keys, typename LineOf<WIDE>::T pairs,
                                           int longest) {
  using Line = typename LineOf<WIDE>::T;
  const Line cost = p.merge_cost / LineOf<WIDE>::KEYS, mean_load = line_div(spans, (Line)p.ctas);
  if (pairs == 0) return 0;
  if (longest > max(mean_load, (Line)(p.min_share / LineOf<WIDE>::KEYS)) + cost) {
    // one of the pairs alone outlasts an even share
  } else if (pairs <= p.ctas) {
    return (int)pairs;
  } else if (WIDE && pairs <= p.pair_ctas) {
    // The last wave's `rest` pairs, taking the spans to fall evenly from the
    // longest to the shortest: they end `w` after the full waves, in place of
    // their spans' even share
    const float P = (float)pairs, S = (float)p.ctas, mean = (float)spans / P;
    const float low = fmaxf(2.f * mean - (float)longest, 0.f);
    const int full = (int)(pairs / p.ctas) * p.ctas;
    const float w = (float)longest - ((float)longest - low) * ((float)full / P);
    if (full == pairs || w - 0.5f * (w + low) * ((float)(pairs - full) / S) <= (float)cost) return (int)pairs;
  }
  if (WIDE && pairs >= p.ctas && pairs <= p.pair_ctas && 2 * (Line)longest * pairs <= 3 * spans &&
      chunk_keys > p.cached_keys)
    return (int)(pairs / p.ctas) * p.ctas;
  return 0;
}

// What follows for CTA `block` from the pairs that run whole and the line's rest.
template <bool WIDE>
__device__ __forceinline__ void place_piece(PagedPlace<WIDE>& r, int block, int whole, typename LineOf<WIDE>::T all_pairs,
                                            typename LineOf<WIDE>::T share, typename LineOf<WIDE>::T rest) {
  r.share = block < whole ? 0 : share;
  r.total = rest;
  r.piece = block - whole;
  r.line = block >= whole;
  if (whole == all_pairs) {   // no line: the first CTAs say so to the merge
    r.piece = block;
    r.line = true;
  }
}

// Finds what CTA `block` works on, query tiles of few rows and at most 32
// sequences: one a lane of the calling warp.
__device__ __forceinline__ PagedPlace<false> find_place_small(const PagedParams& p, int block, bool report) {
  constexpr int KEYS = LineOf<false>::KEYS;
  const int lane = (int)threadIdx.x & 31;
  int span = 0, pairs = 0, longest = 0;
  PagedSeq s;
  s.tiles = s.keys = s.n_q = s.n_k = s.row0 = 0;
  if (lane < p.batch) {
    s = paged_seq<false>(p, p.cu_q[lane], p.cu_q[lane + 1], p.lens_k[lane], report);
    span = s.span<false>(p, s.tiles);
    pairs = s.tiles * p.heads_kv;
    if (s.tiles > 0) longest = s.width<false>(p, 0);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  int a = span, b = pairs;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int va = __shfl_up_sync(0xffffffffu, a, o), vb = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += va;
      b += vb;
    }
  }
  const int total = __shfl_sync(0xffffffffu, a, 31), all_pairs = __shfl_sync(0xffffffffu, b, 31);
  const int whole = whole_pairs<false>(p, total, 0, all_pairs, longest);   // all or none
  const int rest = whole == all_pairs ? 0 : total;
  const int share = max(line_div(rest + p.ctas - 1, p.ctas), p.min_share / KEYS);
  const bool one = block < whole;
  const int pos = one ? block : (block - whole) * share;
  const int size = one ? pairs : span, mine = (one ? b : a) - size;
  const unsigned holds = __ballot_sync(0xffffffffu, (one || pos < rest) && pos >= mine && pos < mine + size);
  PagedPlace<false> r;
  r.seq = __ffs(holds) - 1;   // -1: none
  const int src = max(r.seq, 0);
  r.at = __shfl_sync(0xffffffffu, mine, src);
  r.s.row0 = __shfl_sync(0xffffffffu, s.row0, src);
  r.s.n_q = __shfl_sync(0xffffffffu, s.n_q, src);
  r.s.n_k = __shfl_sync(0xffffffffu, s.n_k, src);
  r.s.tiles = __shfl_sync(0xffffffffu, s.tiles, src);
  r.s.keys = __shfl_sync(0xffffffffu, s.keys, src);
  r.rank = one ? pos - r.at : 0;
  place_piece<false>(r, block, whole, all_pairs, share, rest);
  return r;
}

// The same of any number of sequences: every thread sums a run of them; every
// thread returns the same.
template <int THREADS, bool WIDE>
__device__ __forceinline__ PagedPlace<WIDE> find_place(const PagedParams& p, int block, PagedScan<WIDE>* sh,
                                                       bool report) {
  using Line = typename LineOf<WIDE>::T;
  constexpr int KEYS = LineOf<WIDE>::KEYS;
  constexpr int NW = THREADS / 32;
  const int tid = (int)threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (p.batch + THREADS - 1) / THREADS;
  const int i0 = min(tid * per, p.batch), i1 = min(i0 + per, p.batch);
  // chunks: keys of the sequences of several query tiles, all K/V heads
  Line span = 0, pairs = 0, chunks = 0;
  int longest = 0;   // pair
  PagedSeq s;
  s.tiles = s.keys = s.n_q = s.n_k = s.row0 = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    s = read_seq<WIDE>(p, i, report);
    const Line x = s.span<WIDE>(p, s.tiles);
    span += x;
    pairs += (Line)s.tiles * p.heads_kv;
    if (s.tiles > 0) longest = max(longest, s.width<WIDE>(p, s.tiles - 1));
    if (WIDE && s.tiles > 1) chunks += (Line)s.n_k * p.heads_kv;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  Line a = span, b = pairs, c = chunks;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Line va = __shfl_up_sync(0xffffffffu, a, o), vb = __shfl_up_sync(0xffffffffu, b, o);
    const Line vc = WIDE ? __shfl_up_sync(0xffffffffu, c, o) : 0;
    if (lane >= o) {
      a += va;
      b += vb;
      c += vc;
    }
  }
  if (lane == 31) {
    sh->warp_sum[0][w] = a;
    sh->warp_sum[1][w] = b;
    sh->warp_sum[2][w] = c;
    sh->warp_longest[w] = longest;
  }
  if (tid == 0) sh->place.seq = -1;
  __syncthreads();
  a -= span;
  b -= pairs;
  Line total = 0, all_pairs = 0, all_chunks = 0;
#pragma unroll 1
  for (int j = 0; j < NW; ++j) {
    if (j == w) {
      a += total;
      b += all_pairs;
    }
    total += sh->warp_sum[0][j];
    all_pairs += sh->warp_sum[1][j];
    all_chunks += sh->warp_sum[2][j];
    longest = max(longest, sh->warp_longest[j]);
  }
  int whole = whole_pairs<WIDE>(p, total, all_chunks, all_pairs, longest);
  int cut_seq = -1, cut_tiles = 0;
  Line shift = 0;
  if (WIDE && whole > 0 && whole < all_pairs) {   // part of the pairs: cut at a query tile's first head
    if (whole >= b && whole < b + pairs) {
      Line x = a, n = b;
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        if (per > 1) s = read_seq<WIDE>(p, i, false);
        const Line sx = s.span<WIDE>(p, s.tiles), sn = (Line)s.tiles * p.heads_kv;
        if (whole < n + sn) {
          const int tiles = (int)(whole - n) / p.heads_kv;   // from the last
          sh->whole = (int)n + tiles * p.heads_kv;
          sh->cut_seq = i;
          sh->cut_tiles = s.tiles - tiles;
          sh->shift = x + sx - s.span<WIDE>(p, s.tiles - tiles);
          break;
        }
        x += sx;
        n += sn;
      }
    }
    __syncthreads();
    whole = sh->whole;
    cut_seq = sh->cut_seq;
    cut_tiles = sh->cut_tiles;
    shift = sh->shift;
  }
  const Line rest = whole == all_pairs ? 0 : total - shift;   // the line's length
  Line share = line_div(rest + p.ctas - 1, (Line)p.ctas);
  if (share < p.min_share / KEYS) share = p.min_share / KEYS;
  const bool one = block < whole;
  const Line pos = one ? block : (block - whole) * share;
  const Line mine = one ? b : a - shift, size = one ? pairs : span;
  if ((one || pos < rest) && pos >= mine && pos < mine + size) {
    Line x = mine;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      if (per > 1) s = read_seq<WIDE>(p, i, false);
      const Line step = one ? (Line)s.tiles * p.heads_kv : s.span<WIDE>(p, s.tiles);
      if (pos < x + step) {
        if (WIDE && !one && i == cut_seq) {   // ends where it did, and starts the line
          x += step - s.span<WIDE>(p, cut_tiles);
          s.tiles = cut_tiles;
        }
        sh->place.at = x;
        sh->place.s = s;
        sh->place.seq = i;
        sh->place.rank = one ? (int)(pos - x) : 0;
        break;
      }
      x += step;
    }
  }
  __syncthreads();
  PagedPlace<WIDE> r = sh->place;
  place_piece<WIDE>(r, block, whole, all_pairs, share, rest);
  return r;
}

// The pair of sequence s that holds offset y of the sequence's span: query
// tile, head, and the pair's start within the span.  (Many rows: by a whole
// warp, the tile searched 32 ways at a time.)
template <bool WIDE>
__device__ __forceinline__ typename LineOf<WIDE>::T pair_at(const PagedParams& p, const PagedSeq& s,
                                                            typename LineOf<WIDE>::T y, int& tile, int& h) {
  tile = 0;
  typename LineOf<WIDE>::T base = 0;
  if constexpr (WIDE) {
    int lo = 0, hi = s.tiles;
#pragma unroll 1
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, mid = lo + ((int)threadIdx.x & 31) * step;
      const unsigned below = __ballot_sync(0xffffffffu, mid < hi && s.before(p, mid) * p.heads_kv <= y);
      lo += (31 - __clz(below)) * step;
      hi = min(hi, lo + step);
    }
    tile = lo;
    base = s.before(p, lo) * p.heads_kv;
  }
  const int w = s.width<WIDE>(p, tile);
  h = (int)line_div(y - base, (typename LineOf<WIDE>::T)w);
  return base + (typename LineOf<WIDE>::T)h * w;
}

// First visited key tile at or after offset y of a pair's span, of n.
__device__ __forceinline__ int span_tile(const PagedParams& p, long long y, int n) {
  const long long k = y - p.overhead;
  const long long j = k <= 0 ? 0 : (k + kPagedKeyTile - 1) / kPagedKeyTile;
  return (int)(j < n ? j : n);
}
__device__ __forceinline__ int span_tile(const PagedParams& p, int y, int n) {
  return max(0, min(y - p.overhead / kPagedKeyTile, n));
}

// A pair whose partials are to be merged: left by the CTA at whose start the
// pair is cut for the first time.
struct PagedMerge {
  int count;      // partials, of pieces c0, c0 + 1 ..; -1: nothing to merge here
  int c0;
  int from_start; // the first of them holds the pair's start (the odd one of its piece's two slots)
  int row, rows;  // first row of q / o / lse; live rows
  int h;          // K/V head
  int pad[2];
};
static_assert(sizeof(PagedMerge) == kPagedMergeBytes, "merge description");

// Walks the fragments of one CTA's piece; every lane of the TMA warp in step.
// What the pairs of one query tile share is worked out once, and the next
// sequence's lengths are read a sequence ahead.
template <bool BAND, bool WIDE>
struct FragWalk {
  using Line = typename LineOf<WIDE>::T;
  PagedSeq s;
  PagedFrag base;     // the current query tile's facts, for all of its key tiles
  int tiles_n;        // its key tiles
  int w;              // its pairs' span
  const int* table;   // the sequence's block-table row
  Line x, begin, end;   // the pair's start on the line; the piece
  int cta, seq, tile, h;
  int next_a, next_b, next_k;   // sequence seq + 1
  bool more, one;     // one: a single pair, whole
  PagedMerge merge;   // the pair cut by the piece's start

  __device__ __forceinline__ void read_ahead(const PagedParams& p) {
    if (seq + 1 < p.batch) {
      next_a = p.cu_q[seq + 1];
      next_b = p.cu_q[seq + 2];
      next_k = p.lens_k[seq + 1];
    }
  }

  __device__ void start_tile(const PagedParams& p) {
    const int q0 = tile * p.tile_tokens, last = min(q0 + p.tile_tokens, s.n_q) - 1;
    base.km = paged_mask(p, s.n_q, s.n_k, last);
    const TileWalk walk = tile_walk(base.km, q0, last);
    tiles_n = walk.n;
    w = s.template width<WIDE>(p, tile);
    base.row = s.row0 + q0;
    base.q0 = q0;
    base.rows = (last + 1 - q0) * p.group;
    base.split = tiles_n <= 3;   // few keys: rounding shows most
    base.npre = walk.npre;
    base.skip = walk.skip;
    base.lo = walk.lo;
    base.end = walk.end;
    KeyMask all = base.km;   // what all rows see
    if constexpr (BAND) all.pre_end = prefix_end(p, all, q0);
    base.tm = tile_mask<BAND>(all, q0, last, kPagedKeyTile);
    if (walk.npre == 0) base.tm.pre -= walk.skip;
    base.tm.lo -= walk.skip;
    base.tm.hi -= walk.skip;
  }

  __device__ __forceinline__ void start(const PagedParams& p, const PagedPlace<WIDE>& pl) {
    const int piece = pl.piece;
    cta = piece;
    seq = pl.seq;
    s = pl.s;
    more = true;
    one = pl.share == 0;
    merge.count = -1;
    table = p.table + (long long)seq * p.table_stride;
    begin = piece * pl.share;   // one: 0
    end = min(begin + pl.share, pl.total);
    if (one) {   // the query tiles from the last (the most keys) to the first
      h = pl.rank % p.heads_kv;
      tile = s.tiles - 1 - pl.rank / p.heads_kv;
      x = 0;
    } else {
      x = pl.at + pair_at<WIDE>(p, s, begin - pl.at, tile, h);
      read_ahead(p);
    }
    start_tile(p);
    if (one) end = w;
    if (begin > x && x >= begin - pl.share) {
      // pieces with key tiles of the pair: the first whose end lies past the
      // pair's overhead, the last that starts before its last tile's end
      constexpr int KEYS = LineOf<WIDE>::KEYS;
      const Line keys = x + p.overhead / KEYS;
      const int c0 = (int)line_div(keys, pl.share);
      const int c1 = (int)line_div(min(keys + (Line)(tiles_n - 1) * (kPagedKeyTile / KEYS), x + w - 1), pl.share);
      merge.count = tiles_n > 0 ? c1 - c0 + 1 : 0;
      merge.c0 = c0;
      merge.from_start = c0 == piece - 1;
      merge.row = base.row;
      merge.rows = base.rows;
      merge.h = h;
    }
  }
};

// The next fragment, to shared memory; false when the piece is done.
template <bool BAND, bool WIDE>
__device__ __forceinline__ bool next_fragment(FragWalk<BAND, WIDE>& k, const PagedParams& p, PagedFrag* dst, int lane) {
  while (k.more) {
    const bool from_start = k.begin <= k.x, to_end = k.end - k.x >= k.w, whole = from_start && to_end;
    const int j0 = from_start ? 0 : span_tile(p, k.begin - k.x, k.tiles_n);
    const int n = (to_end ? k.tiles_n : span_tile(p, k.end - k.x, k.tiles_n)) - j0;
    const bool some = n > 0 || whole;   // else: nothing of this pair falls here (its merge sees the same)
    if (some && lane == 0) {
      *dst = k.base;
      dst->table = k.table;
      dst->h = k.h;
      dst->j0 = j0;
      dst->n = n;
      dst->slot = whole ? -1 : 2 * k.cta + (from_start ? 1 : 0);
      dst->tm = k.base.tm.from(j0);
    }
    // on to the next pair
    k.x += k.w;
    if (k.one || k.x >= k.end) {
      k.more = false;
    } else if (++k.h == p.heads_kv) {
      k.h = 0;
      if (!WIDE || ++k.tile == k.s.tiles) {
        k.tile = 0;
        do {
          if (++k.seq >= p.batch) {
            k.more = false;
            break;
          }
          k.table += p.table_stride;
          k.s = paged_seq<WIDE>(p, k.next_a, k.next_b, k.next_k, false);
          k.read_ahead(p);
        } while (k.s.tiles == 0);
      }
      if (k.more) k.start_tile(p);
    }
    if (some) {
      __syncwarp();
      return true;
    }
  }
  return false;
}

// The same out of line, for the TMA warp between its loads (inlined there, a
// prompt chunk of 2048 over 16384 keys takes 449 us in place of 428).
template <bool BAND, bool WIDE>
static __device__ __noinline__ bool next_fragment_far(FragWalk<BAND, WIDE>& k, const PagedParams& p, PagedFrag* dst,
                                                      int lane) {
  return next_fragment(k, p, dst, lane);
}

// ---------------------------------------------------------------- the warps' roles

// Waits as wait_or_abort.  A kernel of few rows runs little of its code often,
// and what each of the many waits carries along is fetched from L2 again and
// again (256 requests of 1..1000 keys, d = 128: 28 % of the instruction cache's
// requests missed with them inline), so all but a wait's first look is out of
// line.  With many rows the MMA thread's waits are inline (a call costs more:
// prompt chunk of 2048 over 16384 keys 469 against 426 us).
static __device__ __noinline__ bool paged_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                    uint32_t* status, uint32_t site) {
  return wait_or_abort(bar, parity, abort_flag, status, site);
}
template <bool WIDE>
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                           uint32_t site) {
  if constexpr (WIDE)
    return wait_or_abort(bar, parity, abort_flag, status, site);
  else
    return mbar_try_wait(bar, parity) || paged_wait_slow(bar, parity, abort_flag, status, site);
}
// A whole warp whose lanes look together: a barrier already passed costs one
// look and one vote.
static __device__ __noinline__ bool paged_warp_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                         uint32_t* status, uint32_t site) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((it & 31u) == 0) {
      bool stop = *abort_flag != 0;
      if (!stop && global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(status, kStatusTimeout | (1u << (8 + site)));
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}
__device__ __forceinline__ bool paged_warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                uint32_t* status, uint32_t site) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         paged_warp_wait_slow(bar, parity, abort_flag, status, site);
}
static __device__ __noinline__ void paged_drain(uint32_t bar, uint32_t parity, uint32_t* status) {
  wait_drain(bar, parity, status);
}

template <class C>
struct PagedCtx {
  uint32_t bar0, sQ, sK, sV, tmem;
  volatile int* abort_flag;
  uint32_t* status;
  PagedFrag* frags;   // four
  __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
  // The TMA or planner warp: its lanes look together, then lane 0 waits for all.
  // The TMA warp's time per tile is part of the tile loop's period (2048 tokens
  // over 10048 keys in pages of 16, d = 128: 247 us, 274 with lane 0 alone).
  __device__ __forceinline__ bool warp_wait(int i, int phase, uint32_t site, int lane) const {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), (uint32_t)phase & 1))) return true;
    bool ok = true;
    if (lane == 0) ok = paged_wait_slow(bar(i), (uint32_t)phase & 1, abort_flag, status, site);
    return __all_sync(0xffffffffu, ok);
  }
};

// 5-D tiled load (see tma_load_4d).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

// The planner warp (few rows): walks the piece's fragments, up to four ahead of
// the softmax.
template <class C, bool BAND>
__device__ __forceinline__ void pg_plan(const PagedCtx<C>& t, const PagedParams& p, const PagedPlace<C::WIDE>& place, int lane) {
  FragWalk<BAND, C::WIDE> walk;
  walk.start(p, place);
  bool have = true;
#pragma unroll 1
  for (int nf = 0; have; ++nf) {
    if (nf >= 4 && !t.warp_wait(PG_FREE + (nf & 3), (nf >> 2) - 1, kSiteProducerEmpty, lane)) break;
    PagedFrag* f = t.frags + (nf & 3);
    have = next_fragment(walk, p, f, lane);
    if (lane == 0) {
      if (!have) f->n = -1;
      mbar_arrive(t.bar(PG_PLAN + (nf & 3)));
      if (nf == 0 && place.line && place.piece < p.ctas) p.merges[place.piece] = walk.merge;
    }
  }
}

// The TMA warp: publishes the piece's fragments (with Q; many rows: walks them too) and loads
// their key tiles, K_0 K_1 V_0 K_2 V_1 .. (a K stage frees at S(j), just before
// PV(j - 1) frees a V stage).  The boxes of four tiles are worked out at once,
// lane 8 q + b holding box b (rows b * box_rows ..) of tile q, and their
// block-table entries read four tiles ahead (the next fragment's first four
// while this one is loaded): with two stages, the time from a free stage to its
// next load is part of the tile loop's period, and between the two stand only a
// wait and the issue.
template <class C, bool BAND>
__device__ __forceinline__ void pg_load(const PagedCtx<C>& t, const PagedParams& p, const CUtensorMap* tm_q,
                                        const CUtensorMap* tm_k, const CUtensorMap* tm_v, const PagedPlace<C::WIDE>& place,
                                        int lane) {
  FragWalk<BAND, C::WIDE> walk;
  if constexpr (!C::PLANNER) {
    walk.start(p, place);
    if (lane == 0 && place.line && place.piece < p.ctas) p.merges[place.piece] = walk.merge;
  }
  // Q loads of at most 64 rows leave room for the next fragment's in the other
  // half of the rows (the products then read 64 rows of whatever follows, which
  // reach no live row).
  constexpr bool two_q = !C::WIDE;
  const int my_tile = lane >> 3, my_box = lane & 7;
  const bool has_box = my_box < C::BC / p.box_rows;
  int walked = 0, published = 0;   // fragments
  bool ok = true, bad = false;
  // Four tiles' boxes: this lane's page and first row within it (-1: no box,
  // or no row of the query tile sees a key of it).
  struct Ahead {
    int page, row;
  };
  auto fetch = [&](const PagedFrag* f, int j4) -> Ahead {
    Ahead x;
    const int k0 = f->tile(f->j0 + j4 + my_tile) * C::BC + my_box * p.box_rows;   // the box's keys [k0, k0 + box_rows)
    const int at = (int)((__umulhi((unsigned)k0, p.page_magic) + (unsigned)k0) >> p.page_shift);   // k0 / page_size
    const bool need = j4 + my_tile < f->n && has_box &&
                      (k0 < f->km.pre_end || (k0 < f->end && k0 + p.box_rows > f->lo));
    x.page = need ? f->table[at] : 0;
    x.row = need ? k0 - at * p.page_size : -1;
    return x;
  };
  Ahead next4;    // the fragment's next four tiles
  Ahead first4;   // the next fragment's first four
  // The next fragment into its slot (whose last user, four before, is done:
  // publishing the one before waited for a later one).
  auto look_ahead = [&]() {
    PagedFrag* f = t.frags + (walked & 3);
    if constexpr (C::PLANNER) {
      ok = t.warp_wait(PG_PLAN + (walked & 3), walked >> 2, kSiteProducerEmpty, lane);
      if (!ok || f->n < 0) return;
    } else {
      if (!next_fragment_far(walk, p, f, lane)) return;
    }
    first4 = fetch(f, 0);
    ++walked;
  };
  // The next fragment's description (and Q), or the end of them, to the other
  // warps, once the last users of its barriers and of Q are done.
  auto publish = [&]() {
    const int nf = published, before = two_q ? nf - 2 : nf - 1;   // `before` used this Q
    ok = (before < 0 || t.warp_wait(PG_QEMPTY + (before & 1), before >> 1, kSiteProducerEmpty, lane)) &&
         (nf < 2 || t.warp_wait(PG_ODONE + (nf & 1), (nf - 2) >> 1, kSiteProducerEmpty, lane));
    if (!ok) return;
    if (lane == 0) {
      PagedFrag* f = t.frags + (nf & 3);
      if (!C::PLANNER && nf == walked) f->n = -1;
      const uint32_t bar = t.bar(PG_Q + (nf & 1));
      if (f->n > 0) {
        const uint32_t sQ = t.sQ + (two_q && (nf & 1) ? C::BR / 2 * 128u : 0u);
        mbar_arrive_expect_tx(bar, (uint32_t)C::BLOCKS * (uint32_t)p.slot_rows * 128u);
#pragma unroll 1
        for (int kb = 0; kb < C::BLOCKS; ++kb)
          tma_load_4d(sQ + kb * (C::BR * 128), tm_q, kb * 64, 0, f->h, f->row, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    ++published;
    __syncwarp();
  };
  // Coordinates of this lane's box in one tensor: merged (page, head), or head
  // and page apart; an out-of-range page is read as zeros from outside the map.
  struct At {
    int c1, c3, c4;
  };
  auto place_box = [&](const Ahead& x, const PagedSide& side, int h) -> At {
    const bool off = x.page < 0 || x.page >= p.num_pages;
    At c;
    if (side.ratio > 0) {
      c.c1 = 0;
      c.c3 = x.row >> 3;
      c.c4 = off ? side.extent : x.page * side.ratio + h;
    } else {
      c.c1 = x.row;
      c.c3 = h;
      c.c4 = off ? p.num_pages : x.page;
    }
    if (x.row >= 0 && off) bad = true;
    return c;
  };
  const uint32_t box_bytes = (uint32_t)p.box_rows * (uint32_t)(C::D * 2);
  // Tile q of the four whose lanes with a box are `lanes`.  (The boxes may land
  // before lane 0 has announced their bytes: its arrival is what lets the
  // barrier complete.  Keeping the lanes in step is faster with many rows, 240
  // against 250 us for 2048 tokens over 10048 keys, and slower with few, 120
  // against 102 for 256 requests of 1..1000 keys.)
  auto issue = [&](const At& c, unsigned lanes, int q, const CUtensorMap* tm, uint32_t s_tile, uint32_t bar) {
    const unsigned mine = lanes & (255u << (8 * q));
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(mine) * box_bytes);
    if constexpr (C::WIDE) __syncwarp();
    if ((mine >> lane) & 1u) tma_load_5d(s_tile + (uint32_t)my_box * box_bytes, tm, 0, c.c1, 0, c.c3, c.c4, bar);
    if constexpr (C::WIDE) __syncwarp();
  };
  int g = 0, gv = 0;            // key tiles loaded
  int nf = -1, j = 0, n = 0;    // the fragment, the tile to load next, its tiles
  At ck, cv, cv_last;           // the four tiles' boxes; V's of the tile before
  unsigned lanes = 0, lanes_last = 0;
  int v_left = 0;               // a V tile to load: 1 + its index of four
  auto load_v = [&]() {
    if (v_left == 0) return;
    const int s = gv % C::VSTAGES;
    if (gv >= C::VSTAGES) ok = t.warp_wait(PG_O + s, gv / C::VSTAGES - 1, kSiteProducerEmpty, lane);
    if (!ok) return;
    issue(cv_last, lanes_last, v_left - 1, tm_v, t.sV + s * C::KV_BYTES, t.bar(PG_VFULL + s));
    v_left = 0;
    ++gv;
  };
#pragma unroll 1
  while (true) {
    // the next tile, of this fragment or of the next with keys
    if (++j >= n) {
      // a fragment's last V goes before anything of the next: what publish waits for may need it
      load_v();
      if (!ok) break;
      j = 0;
#pragma unroll 1
      do {
        ++nf;
        if (nf == walked) look_ahead();
        if (!ok) break;
        n = nf < walked ? t.frags[nf & 3].n : -1;
        if (published == nf && n <= 0) publish();   // without keys, or the end
      } while (ok && n == 0);
      if (!ok || n < 0) break;
      if (C::WIDE && g == 0 && published == nf) {   // the first Q, the longest load, before the first K
        publish();
        if (!ok) break;
      }
      next4 = first4;
    }
    if ((j & 3) == 0) {
      const PagedFrag* f = t.frags + (nf & 3);
      const Ahead now = next4;
      next4 = fetch(f, j + 4);
      ck = place_box(now, p.k_side, f->h);
      cv = place_box(now, p.v_side, f->h);
      lanes = __ballot_sync(0xffffffffu, now.row >= 0);
    }
    const int s = g % C::KSTAGES;
    if (g >= C::KSTAGES) ok = t.warp_wait(PG_S + s, g / C::KSTAGES - 1, kSiteProducerEmpty, lane);
    if (!ok) break;
    issue(ck, lanes, j & 3, tm_k, t.sK + s * C::KV_BYTES, t.bar(PG_KFULL + s));
    ++g;
    load_v();
    if (!ok) break;
    cv_last = cv;
    lanes_last = lanes;
    v_left = 1 + (j & 3);
    if (j > C::VSTAGES + 1) continue;   // what follows is due by then
    if (j > 0 && j == min(n, 3) - 1 && walked == nf + 1) look_ahead();
    if (!ok) break;
    // this fragment at its first tile; the next one, with room for its Q, once V_j with j = VSTAGES has waited
    // for PV(0), which followed the epilogue of the fragment before
    if (published == nf || (two_q && j == C::VSTAGES + 1 && published == nf + 1 && walked > published)) publish();
    if (!ok) break;
  }
  if (bad) atomicOr(p.status, kStatusBadPages);
  // own copies in flight land before the CTA may exit
  if (lane == 0) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
      if (published > i) paged_drain(t.bar(PG_Q + i), (uint32_t)((published - 1 - i) / 2) & 1, t.status);
#pragma unroll 1
    for (int s = 0; s < C::KSTAGES; ++s) {
      if (g > s) paged_drain(t.bar(PG_KFULL + s), (uint32_t)((g - 1 - s) / C::KSTAGES) & 1, t.status);
      if (gv > s) paged_drain(t.bar(PG_VFULL + s), (uint32_t)((gv - 1 - s) / C::VSTAGES) & 1, t.status);
    }
  }
}

// The MMA thread: per fragment S(0), S(1), PV(0), S(2), PV(1) .. (PV(j): O~ +=
// P(j) V_j), as db_mma; with few rows, in a loop with one place in the code for
// each product.  O~ of the fragment before must have been read (PG_ODONE) before PV(0); the S products
// run ahead of that.  P of keys 32 c .. of a tile lies in the columns its
// scores had, low parts (split) 16 columns on.
template <class C, bool BF16>
__device__ __forceinline__ void pg_mma(const PagedCtx<C>& t, const PagedParams& p) {
  const uint32_t idesc_qk = make_idesc_f16(C::BR, C::BC, BF16, false, false) | p.qk_negate;
  constexpr uint32_t idesc_pv = make_idesc_f16(C::BR, C::D, BF16, false, true);
  const uint64_t dq0 = make_sdesc_sw128(t.sQ, 16, 1024);
  const uint64_t dk0 = make_sdesc_sw128(t.sK, 16, C::GROUP_BYTES);
  const uint64_t dv0 = make_sdesc_sw128(t.sV, 1024, C::GROUP_BYTES);
  constexpr bool two_q = !C::WIDE;
  auto wait = [&](int bar, int phase, uint32_t site) -> bool {
    return paged_wait<C::WIDE>(t.bar(bar), (uint32_t)phase & 1, t.abort_flag, t.status, site);
  };
  bool ok = true;
  int g0 = 0;   // key tiles of the fragments before
#pragma unroll 1
  for (int nf = 0; ok; ++nf) {
    if (!wait(PG_Q + (nf & 1), nf >> 1, kSiteMmaQ)) break;
    const PagedFrag* f = t.frags + (nf & 3);
    const int n = f->n;
    if (n < 0) break;
    if (n == 0) {
      mbar_arrive(t.bar(PG_QEMPTY + (nf & 1)));
      continue;
    }
    const TileMask tm = f->tm;
    const bool always = f->split != 0;
    const uint64_t a0 = dq0 + (two_q && (nf & 1) ? (uint64_t)((C::BR / 2 * 128) >> 4) : 0ull);
    auto issue_s = [&](int i) -> bool {
      const int g = g0 + i, sk = g % C::KSTAGES;
      if (!wait(PG_KFULL + sk, g / C::KSTAGES, kSiteMmaK)) return false;
      tc_fence_after();
      const uint64_t b0 = dk0 + (uint64_t)((sk * C::KV_BYTES) >> 4);
      const uint32_t tS = t.tmem + C::TMEM_S + 64 * (g & 1);
#pragma unroll
      for (int k = 0; k < C::D / 16; ++k)
        umma_ss(tS, a0 + (uint64_t)(((k >> 2) * (C::BR * 128) + (k & 3) * 32) >> 4),
                b0 + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc_qk, k > 0 ? 1u : 0u);
      umma_commit(t.bar(PG_S + sk));
      if (i + 1 == n) umma_commit(t.bar(PG_QEMPTY + (nf & 1)));
      return true;
    };
    auto issue_pv = [&](int j) -> bool {
      const int g = g0 + j, sv = g % C::VSTAGES;
      if (j == 0 && nf > 0 && !wait(PG_ODONE + ((nf - 1) & 1), (nf - 1) >> 1, kSiteMmaO)) return false;
      if (!wait(PG_P + (g & 1), g >> 1, kSiteMmaP) || !wait(PG_VFULL + sv, g / C::VSTAGES, kSiteMmaV)) return false;
      tc_fence_after();
      const uint64_t b0 = dv0 + (uint64_t)((sv * C::KV_BYTES) >> 4);
      const uint32_t tS = t.tmem + C::TMEM_S + 64 * (g & 1);
      const uint32_t tO = t.tmem + C::TMEM_O;
      const bool split = BF16 && (always || !tm.full(j));
      auto product = [&](bool both) {
#pragma unroll
        for (int k = 0; k < C::BC / 16; ++k) {
          const uint64_t bk = b0 + (uint64_t)((k * 2 * C::GROUP_BYTES) >> 4);
          const uint32_t pk = tS + (k >> 1) * 32 + (k & 1) * 8;
          umma_ts(tO, pk, bk, idesc_pv, (j > 0 || k > 0) ? 1u : 0u);
          if (both) umma_ts(tO, pk + 16, bk, idesc_pv, 1u);
        }
      };
      if (split)
        product(true);
      else
        product(false);
      umma_commit(t.bar(PG_O + sv));
      return true;
    };
    if constexpr (C::WIDE) {
#pragma unroll 1
      for (int i = 0; i < min(n, 2) && ok; ++i) ok = issue_s(i);
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) ok = issue_pv(j) && (j + 2 >= n || issue_s(j + 2));
    } else {
#pragma unroll 1
      for (int i = 0; i <= n && ok; ++i) ok = (i == n || issue_s(i)) && (i == 0 || issue_pv(i - 1));
    }
    g0 += n;
  }
  umma_commit(t.bar(PG_EXIT));
  paged_drain(t.bar(PG_EXIT), 0, t.status);
}

// Zeroes the rows of V tile `kt` (shared memory) whose keys no row of the
// query tile sees; 128 threads, thread `tid`.
template <class C>
__device__ __forceinline__ void zero_hidden_rows(uint32_t sV, int kt, const PagedFrag* f, int tid) {
  const int lo = f->lo, end = f->end, pre = f->km.pre_end;
  for (int c = tid; c < C::BC * (C::D / 8); c += 128) {
    // 16-byte chunk c % 8 of row (c / 8) % 8, column block, 8-row group
    const int key = kt * C::BC + c / (64 * C::BLOCKS) * 8 + (c / 8) % 8;
    if (key < pre || (key >= lo && key < end)) continue;
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sV + (uint32_t)c * 16u), "r"(0u) : "memory");
  }
}

// P = 2^(s * scale - m) of 32 keys into 16 columns of 16-bit pairs, its low part
// P - P_hi (SPLIT) into the 16 after them: the columns their scores had.
template <bool BF16, bool SPLIT>
__device__ __forceinline__ void paged_p_run(const uint32_t* sr, uint32_t tP, float2 scale2, float2 neg_m2, float2& sum0,
                                            float2& sum1) {
  uint32_t ph[16];
  uint32_t pl[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), scale2, neg_m2);
    x.x = ex2_approx(x.x);
    x.y = ex2_approx(x.y);
    if (c & 1)
      sum1 = __fadd2_rn(sum1, x);
    else
      sum0 = __fadd2_rn(sum0, x);
    ph[c] = pack2<BF16>(x.x, x.y);
    if constexpr (SPLIT) {
      const float2 h = unpack2<BF16>(ph[c]);
      pl[c] = pack2<BF16>(x.x - h.x, x.y - h.y);
    }
  }
  tmem_st_32x32b_x16(tP, ph);
  if constexpr (SPLIT) tmem_st_32x32b_x16(tP + 16, pl);
}

// Output row r of a tile: the token's row, the query head's columns.
__device__ __forceinline__ uint8_t* paged_o_row(const PagedParams& p, int row, int head) {
  return reinterpret_cast<uint8_t*>(p.o) + 2 * ((long long)row * p.o_rs + (long long)head * p.o_hs);
}

template <class C, bool BF16, bool BAND>
__device__ __forceinline__ void pg_softmax(const PagedCtx<C>& t, const PagedParams& p, int warp, int lane) {
  const int quad = warp & 3;
  const int r = quad * 32 + lane;
  const int tok = r / p.group;
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  const uint32_t tO = t.tmem + lane_off + C::TMEM_O;
  const float sl2 = p.scale_log2_mag;
  auto wait = [&](int bar, int phase, uint32_t site) -> bool {
    // (2048 tokens over 10048 keys: d = 64 198 us with the looks together, 201
    // apart, d = 256 497 and 515; but d = 128, many rows, 253 and 241)
    if constexpr (C::WIDE && C::D == 128)
      return __all_sync(0xffffffffu, wait_or_abort(t.bar(bar), (uint32_t)phase & 1, t.abort_flag, t.status, site));
    else
      return paged_warp_wait(t.bar(bar), (uint32_t)phase & 1, t.abort_flag, t.status, site);
  };
  int g = 0;   // key tiles
  for (int nf = 0;; ++nf) {
    if (!wait(PG_Q + (nf & 1), nf >> 1, kSiteMmaQ)) return;
    const PagedFrag* f = t.frags + (nf & 3);
    const int n = f->n;
    if (n < 0) return;
    const int rows = f->rows;
    const bool live = r < rows;
    const bool warp_live = quad * 32 < rows;
    const int head = f->h * p.group + (r - tok * p.group);
    const TileMask tmask = f->tm;
    const bool always = f->split != 0;
    float m_run = -INFINITY;
    float l_run = 0.f;
    for (int j = 0; j < n; ++j, ++g) {
      const uint32_t tS = t.tmem + lane_off + C::TMEM_S + 64 * (g & 1);
      if (!wait(PG_S + g % C::KSTAGES, g / C::KSTAGES, kSiteSoftmaxS)) return;
      tc_fence_after();
      const bool masked = !tmask.full(j);
      if (warp_live) {
        const int k0 = f->tile(f->j0 + j) * C::BC, tok_row = f->q0 + tok;
        const bool split = BF16 && (always || masked);
        // The tile's 64 scores: in registers (a warp of live rows, where the
        // softmax is what bounds the loop), or read from tensor memory twice in
        // runs of 32, half the code (few rows: the loop waits for the keys, and
        // code costs more than the second read)
        uint32_t sr[C::WIDE ? C::BC : 32];
        auto row_mask = [&]() {
          KeyMask km = f->km;
          if constexpr (BAND) km.pre_end = prefix_end(p, km, tok_row);
          return km;
        };
        auto read = [&](int c) {
          tmem_ld_32x32b_x32(tS + c, sr + (C::WIDE ? c : 0));
          tmem_ld_wait_x32(sr + (C::WIDE ? c : 0));
          if (masked) mask_scores<32, BAND>(sr + (C::WIDE ? c : 0), row_mask(), tok_row, k0 + c);
        };
        float m_tile = -INFINITY;
        auto top = [&](int c) {
          const uint32_t* x = sr + (C::WIDE ? c : 0);
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            mx0 = fmax3(mx0, __uint_as_float(x[i + 0]), __uint_as_float(x[i + 1]));
            mx1 = fmax3(mx1, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
            mx2 = fmax3(mx2, __uint_as_float(x[i + 4]), __uint_as_float(x[i + 5]));
            mx3 = fmax3(mx3, __uint_as_float(x[i + 6]), __uint_as_float(x[i + 7]));
          }
          m_tile = fmaxf(m_tile, fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)));
        };
        if constexpr (C::WIDE) {
          tmem_ld_32x32b_x32(tS, sr);
          tmem_ld_32x32b_x32(tS + 32, sr + 32);
          tmem_ld_wait_x32(sr);
          tmem_ld_wait_x32(sr + 32);
          if (masked) mask_scores<C::BC, BAND>(sr, row_mask(), tok_row, k0);
          top(0);
          top(32);
        } else {
#pragma unroll 1
          for (int c = 0; c < C::BC; c += 32) {
            read(c);
            top(c);
          }
        }
        m_tile *= sl2;
        const bool raise = live && m_tile > m_run + kRescaleLog2;
        const float m_new = raise ? m_tile : m_run;
        const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
        const float alpha = raise ? ex2_approx(m_run - m_use) : 1.f;
        const float2 scale2 = make_float2(sl2, sl2);
        const float2 neg_m2 = make_float2(-m_use, -m_use);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        if constexpr (C::WIDE) {
          if (split) {
            paged_p_run<BF16, true>(sr, tS, scale2, neg_m2, sum0, sum1);
            paged_p_run<BF16, true>(sr + 32, tS + 32, scale2, neg_m2, sum0, sum1);
          } else {
            paged_p_run<BF16, false>(sr, tS, scale2, neg_m2, sum0, sum1);
            paged_p_run<BF16, false>(sr + 32, tS + 32, scale2, neg_m2, sum0, sum1);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < C::BC; c += 32) {
            read(c);
            if (split)
              paged_p_run<BF16, true>(sr, tS + c, scale2, neg_m2, sum0, sum1);
            else
              paged_p_run<BF16, false>(sr, tS + c, scale2, neg_m2, sum0, sum1);
          }
        }
        const float2 sum2 = __fadd2_rn(sum0, sum1);
        l_run = l_run * alpha + (sum2.x + sum2.y);
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
          // S(g) was issued before PV(g-1): wait for that product before rescaling
          if (!wait(PG_O + (g - 1) % C::VSTAGES, (g - 1) / C::VSTAGES, kSiteSoftmaxO)) return;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < C::D; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + c, o);
            tmem_ld_wait_x32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32x32b_x32(tO + c, o);
          }
        }
        tmem_st_wait();
        m_run = m_new;
      }
      if (masked) {
        const int kt = f->tile(f->j0 + j);
        if (!((kt + 1) * C::BC <= f->km.pre_end || (kt * C::BC >= f->lo && (kt + 1) * C::BC <= f->end))) {
          // some key of the tile is hidden from every row: its V row may be anything
          const int sv = g % C::VSTAGES;
          if (!wait(PG_VFULL + sv, g / C::VSTAGES, kSiteMmaV)) return;
          zero_hidden_rows<C>(t.sV + sv * C::KV_BYTES, kt, f, r);
          fence_proxy_async_smem();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(t.bar(PG_P + (g & 1)));
    }
    if (n > 0) {
      if (!wait(PG_O + (g - 1) % C::VSTAGES, (g - 1) / C::VSTAGES, kSiteEpilogueO)) return;
      tc_fence_after();
    }
    const int slot_at = f->slot;
    const int row = f->row + tok;
    if (warp_live && slot_at >= 0) {
      // four columns of a row are 16 bytes, the rows of four columns follow
      // each other: a warp's store is one contiguous run (row-major, its 32
      // rows would be 32 lines)
      float4* dst = reinterpret_cast<float4*>(p.ws_o) + (size_t)slot_at * (size_t)(C::D / 4) * (size_t)p.slot_rows + r;
#pragma unroll 1
      for (int c = 0; c < C::D; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tO + c, o);
        tmem_ld_wait_x32(o);
        if (live) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(c / 4 + i) * p.slot_rows] =
                make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                            __uint_as_float(o[4 * i + 3]));
        }
      }
      if (live)
        *reinterpret_cast<float2*>(p.ws_ml + ((size_t)slot_at * (size_t)p.slot_rows + r) * 2) =
            make_float2(m_run, l_run);
    } else if (warp_live) {
      const bool empty = l_run == 0.f;   // sees no key; a NaN sum is no such row's
      const float inv_l = empty ? 0.f : 1.f / l_run;
      uint8_t* o_row = paged_o_row(p, row, head);
#pragma unroll 1
      for (int c = 0; c < C::D; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tO + c, o);   // n = 0: not used
        tmem_ld_wait_x32(o);
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(o_row + c * 2);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = empty ? 0u : pack2<BF16>(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
      if (live)
        p.lse[(long long)head * p.lse_hs + row] = empty ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(t.bar(PG_ODONE + (nf & 1)));
      if (C::PLANNER) mbar_arrive(t.bar(PG_FREE + (nf & 3)));
    }
  }
}

// SMALL: few rows and at most 32 sequences (find_place_small: 1 request of 600
// keys 11.1 us, 11.8 with the general search; 8 x 5 drafted tokens 16.8, 17.8.
// Its own kernel, since the code of both in one costs batches of hundreds: 500
// requests of 1..300 keys 105 us, 115).
template <int D, bool BF16, bool BAND, bool WIDE, bool SMALL>
__global__ void __launch_bounds__(PagedConfig<D, WIDE>::THREADS, PagedConfig<D, WIDE>::CTAS_PER_SM)
    fa2_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using C = PagedConfig<D, WIDE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  PagedScan<WIDE>* scan = reinterpret_cast<PagedScan<WIDE>*>(smem + C::OFF_SCAN);
  static_assert(sizeof(PagedScan<WIDE>) <= 320 && C::OFF_SCAN % 8 == 0, "scan area");
  const int warp = (int)(threadIdx.x >> 5);
  const int lane = (int)(threadIdx.x & 31);
  grid_launch_dependents();   // the merge may be scheduled once every CTA has started; it waits for the partials

  PagedCtx<C> t;
  t.bar0 = sbase + C::OFF_BAR;
  t.sQ = sbase + C::OFF_Q;
  t.sK = sbase + C::OFF_K;
  t.sV = sbase + C::OFF_V;
  t.abort_flag = abort_flag;
  t.status = p.status;
  t.frags = reinterpret_cast<PagedFrag*>(smem + C::OFF_FRAG);
  if (warp == C::TMA_WARP && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < PG_BARS; ++i)
      mbar_init(t.bar(i), (i >= PG_P && i < PG_EXIT) || i >= PG_FREE ? 4 : 1);   // four softmax warps, or one arrival
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // What precedes this kernel is complete: from here on it touches memory, and
  // takes tensor memory (held while waiting, it could be what a kernel before
  // this one waits for).
  grid_dependency_wait();
  // Tensor memory before the schedule: an SM's second CTA starts only when the
  // first has let go of the allocation permit (measured: 3.6 us into the kernel
  // with the allocation behind the schedule, half of the CTAs).
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  PagedPlace<WIDE> place;
  if constexpr (SMALL) {
    if (warp == C::PLAN_WARP) {
      place = find_place_small(p, (int)blockIdx.x, blockIdx.x == 0);
      if (lane == 0) scan->place = place;
    }
    __syncthreads();
    place = scan->place;
  } else {
    place = find_place<C::THREADS, WIDE>(p, (int)blockIdx.x, scan, blockIdx.x == 0);   // with its barriers
  }
  tc_fence_after();
  t.tmem = *tmem_slot;

  if (place.seq < 0) {   // nothing for this CTA
    if (threadIdx.x == 0 && place.line && place.piece < p.ctas) p.merges[place.piece].count = -1;
  } else if (warp == C::TMA_WARP) {
    pg_load<C, BAND>(t, p, &tm_q, &tm_k, &tm_v, place, lane);
  } else if (warp == C::MMA_WARP) {
    if (lane == 0) pg_mma<C, BF16>(t, p);
    __syncwarp();
  } else if (C::PLANNER && warp == C::PLAN_WARP) {
    pg_plan<C, BAND>(t, p, place, lane);
  } else {
    pg_softmax<C, BF16, BAND>(t, p, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(t.tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- the merge

constexpr int kPagedMergeThreads = 256;
constexpr int kPagedMergeRows = 32;   // rows of a block

// Block (m, y): rows 32 y .. of the pair that the start of piece m + 1 cuts
// first.  Each warp takes every eighth run of four columns; its lanes are the
// rows, or (fewer than 17 rows) rows x partials, each with its own running
// maximum, whose sums are then joined by shuffles in a fixed order.  The rows
// go out through shared memory, whole.
template <int D, bool BF16>
__global__ void __launch_bounds__(kPagedMergeThreads) fa2_paged_merge_kernel(const __grid_constant__ PagedParams p) {
  constexpr int NW = kPagedMergeThreads / 32;
  constexpr int E = D / 4 / NW;   // column runs of a warp
  __shared__ uint2 stage[kPagedMergeRows][D / 4];
  const int r0 = (int)blockIdx.y * kPagedMergeRows;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  grid_dependency_wait();   // the partials and descriptions are complete and visible
  grid_launch_dependents();
  const PagedMerge mg = p.merges[blockIdx.x + 1];
  if (mg.count < 0 || r0 >= mg.rows) return;
  const int here = min(mg.rows - r0, kPagedMergeRows);
  const int width_log2 = here <= 1 ? 0 : 32 - __clz(here - 1);   // lanes of rows
  const int r = lane & ((1 << width_log2) - 1), sub = lane >> width_log2, subs = 32 >> width_log2;
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + r0 + r;
  const float4* part = reinterpret_cast<const float4*>(p.ws_o) + (size_t)warp * p.slot_rows + r0 + r;
  float m = -INFINITY, l = 0.f;
  float4 acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  // two partials at a time: the reads of both are in flight together
  constexpr int U = E <= 4 ? 2 : 1;
#pragma unroll 1
  for (int k0 = r < here ? sub : mg.count; k0 < mg.count; k0 += U * subs) {
    float2 s[U];
    float4 v[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * subs;
      s[u] = make_float2(-INFINITY, 0.f);
      if (k < mg.count) {
        const size_t slot = (size_t)(2 * (mg.c0 + k) + (k == 0 ? mg.from_start : 0)) * (size_t)p.slot_rows;
        s[u] = ml[slot];
        const float4* src = part + slot * (D / 4);
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = src[(size_t)(e * NW) * p.slot_rows];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s[u].y == 0.f) continue;   // shows the row nothing (a NaN sum stays)
      const float top = fmaxf(m, s[u].x);
      const float f0 = ex2_approx(m - top), f = ex2_approx(s[u].x - top);   // f0: 0 before the first
      m = top;
      l = l * f0 + s[u].y * f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[e].x = fmaf(f, v[u][e].x, acc[e].x * f0);
        acc[e].y = fmaf(f, v[u][e].y, acc[e].y * f0);
        acc[e].z = fmaf(f, v[u][e].z, acc[e].z * f0);
        acc[e].w = fmaf(f, v[u][e].w, acc[e].w * f0);
      }
    }
  }
  float M = m;
#pragma unroll 1
  for (int o = 1 << width_log2; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float f = m == -INFINITY ? 0.f : ex2_approx(m - M);
  float L = l * f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float4(acc[e].x * f, acc[e].y * f, acc[e].z * f, acc[e].w * f);
#pragma unroll 1
  for (int o = 1 << width_log2; o < 32; o <<= 1) {
    L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      acc[e].x += __shfl_xor_sync(0xffffffffu, acc[e].x, o);
      acc[e].y += __shfl_xor_sync(0xffffffffu, acc[e].y, o);
      acc[e].z += __shfl_xor_sync(0xffffffffu, acc[e].z, o);
      acc[e].w += __shfl_xor_sync(0xffffffffu, acc[e].w, o);
    }
  }
  const bool empty = L == 0.f;
  const float inv_l = empty ? 0.f : 1.f / L;
  if (sub == 0 && r < here) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      stage[r][warp + e * NW] = empty ? make_uint2(0u, 0u)
                                      : make_uint2(pack2<BF16>(acc[e].x * inv_l, acc[e].y * inv_l),
                                                   pack2<BF16>(acc[e].z * inv_l, acc[e].w * inv_l));
    if (warp == 0) {
      const int at = r0 + r, tok = at / p.group;
      p.lse[(long long)(mg.h * p.group + at - tok * p.group) * p.lse_hs + mg.row + tok] =
          empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < here * (D / 8); i += kPagedMergeThreads) {
    const int at = r0 + i / (D / 8), c = i % (D / 8), tok = at / p.group;
    reinterpret_cast<uint4*>(paged_o_row(p, mg.row + tok, mg.h * p.group + at - tok * p.group))[c] =
        reinterpret_cast<const uint4*>(stage[at - r0])[c];
  }
}

template <int D, bool BF16, bool BAND, bool WIDE, bool SMALL>
int launch_paged_kernels(const PagedLaunchArgs& a) {
  using C = PagedConfig<D, WIDE>;
  auto kern = fa2_paged_kernel<D, BF16, BAND, WIDE, SMALL>;
  static std::atomic<unsigned long long> configured{0};
  const int e = once_per_device(configured, [&]() -> int {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_BYTES);
    if (r != cudaSuccess) return (int)r;
    cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    return (int)cudaFuncSetAttribute(fa2_paged_merge_kernel<D, BF16>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  if (e != 0) return e;
  // whole waves (few rows: all of the batch is on the line, or at most `ctas` pairs)
  const int waves = WIDE ? (a.p.pair_ctas + a.p.ctas - 1) / a.p.ctas : 1;
  const int grid = a.p.ctas * (waves > 1 ? waves : 1);
  const int r = launch_dependent(kern, dim3((unsigned)grid), C::THREADS, C::SMEM_BYTES, a.stream, a.tm_q, a.tm_k, a.tm_v,
                                 a.p);
  if (r != 0) return r;
  const dim3 blocks((unsigned)(a.p.ctas - 1), (unsigned)((a.p.slot_rows + kPagedMergeRows - 1) / kPagedMergeRows));
  return launch_dependent(fa2_paged_merge_kernel<D, BF16>, blocks, kPagedMergeThreads, 0, a.stream, a.p);
}

template <int D, bool BF16, bool BAND>
int launch_paged_rows(const PagedLaunchArgs& a) {
  if (a.wide) return launch_paged_kernels<D, BF16, BAND, true, false>(a);
  return a.p.batch <= 32 ? launch_paged_kernels<D, BF16, BAND, false, true>(a)
                         : launch_paged_kernels<D, BF16, BAND, false, false>(a);
}

template <int D>
int launch_paged(const PagedLaunchArgs& a) {
  if (a.bf16) return a.band ? launch_paged_rows<D, true, true>(a) : launch_paged_rows<D, true, false>(a);
  return a.band ? launch_paged_rows<D, false, true>(a) : launch_paged_rows<D, false, false>(a);
}

}  // namespace fa2
