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
// The tile loop is the double-buffered forward kernel's (fa2_fwd_dbuf.cuh: its
// MMA role, barriers, tensor-memory layout and two-CTA size classes).  What
// differs: a 64-key tile arrives as one box per page (pages of 8 .. 32 rows)
// or as one box (pages of 64 k rows); the TMA warp's lanes each read their
// box's page from the block table three tiles ahead and issue their own box,
// so the table's latency stays off the pipeline.  Pages none of the tile's
// rows see are not loaded, and key tiles between a prefix and the band are not
// visited.  V rows no row of the tile sees (the last page's tail, keys before
// a window) may hold anything: they are zeroed in shared memory before the
// product, since 0 x NaN would reach the sums.
//
// Key splits: the lengths are on the device, so every CTA sums the batch's
// work (the visited key tiles of all query tiles), derives the split size that
// cuts it into about target_units equal units, and finds its own unit by a
// prefix sum over the sequences.  A tile cut into several units leaves fp32
// partials (m, l, O~) that a second kernel, launched as a programmatic
// dependent, merges; other tiles write O and L directly.
#pragma once

#include <cstring>

#include "fa2_fwd_dbuf.cuh"
#include "fa2_paged.h"

namespace fa2 {

template <int D_>
struct PagedConfig : DbufConfig<D_> {
  using Base = DbufConfig<D_>;
  static constexpr bool TMA_GATES_P = false;
  static constexpr uint32_t MISC_BYTES = 512;   // TMEM address, abort flag, unit; scan scratch
  static constexpr uint32_t SMEM_BYTES = Base::OFF_MISC + MISC_BYTES + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
  static_assert(Base::CTAS_PER_SM * (SMEM_BYTES + 1024) <= 233472, "shared memory per SM");
};

// One sequence's part in the schedule.
struct PagedSeq {
  int row0, n_q, n_k;
  int tiles;   // query tiles
  int nv;      // most key tiles one of them visits
};

// The key tiles a query tile visits: visited index j is key tile j + (j >=
// npre ? skip : 0).  lo / end: the band's keys; pre_end (KeyMask): the prefix.
struct TileWalk {
  int npre, skip, n;
  int lo, end;
  __device__ __forceinline__ int tile(int j) const { return j + (j >= npre ? skip : 0); }
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

__device__ __forceinline__ KeyMask paged_mask(const PagedParams& p, int n_q, int n_k) {
  KeyMask km;
  km.n_k = n_k;
  km.off = n_k - n_q;
  km.wl = p.window_left;
  km.wr = p.window_right;
  km.pre_end = min(p.prefix, n_k);
  return km;
}

// Sequence i; no tiles (and the bad-offsets bit, if `report`) when its row
// offsets or its length are out of range.
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int i, bool report) {
  PagedSeq s;
  const int a = __ldg(p.cu_q + i), b = __ldg(p.cu_q + i + 1), k = __ldg(p.lens_k + i);
  s.row0 = a;
  s.n_q = b - a;
  s.n_k = k;
  s.tiles = 0;
  s.nv = 0;
  if (!(0 <= a && a <= b && b <= p.total_q && b - a <= p.max_q && 0 <= k &&
        (long long)k <= (long long)p.max_pages * p.page_size)) {
    if (report) atomicOr(p.status, kStatusBadSeqlens);
    return s;
  }
  if (s.n_q == 0) return s;
  s.tiles = (s.n_q + p.tile_tokens - 1) / p.tile_tokens;
  const KeyMask km = paged_mask(p, s.n_q, s.n_k);
  if (p.window_left < 0 || s.tiles == 1) {
    // without a left window the last tile visits the most
    s.nv = tile_walk(km, (s.tiles - 1) * p.tile_tokens, s.n_q - 1).n;
  } else {
    const long long band = (long long)p.window_left + (p.window_right < 0 ? s.n_k : p.window_right) + p.tile_tokens;
    const long long all = (s.n_k + kPagedKeyTile - 1) / kPagedKeyTile;
    const long long n = (km.pre_end + kPagedKeyTile - 1) / kPagedKeyTile + band / kPagedKeyTile + 2;
    s.nv = (int)(n < all ? n : all);
  }
  return s;
}

// What a CTA works on: a query tile of one K/V head of one sequence, and the
// split size that its units follow.
struct PagedUnit {
  int seq, row0, n_q, n_k;
  int h, tile;
  int split;        // this unit's chunk
  int splits;       // chunks the sequence's tiles are cut into at most
  int chunk;        // the split size C in key tiles
  int slot0;        // first partial slot of the sequence (splits > 1)
};

// Chunks a tile of n visited key tiles is cut into, given the split size.
__device__ __forceinline__ int tile_splits(int n, int chunk) { return n > chunk ? (n + chunk - 1) / chunk : 1; }

// Slot of a tile's chunk `s`: the sequence's units in launch order.
__device__ __forceinline__ int unit_slot(const PagedUnit& u, int tiles, int heads, int s) {
  return u.slot0 + ((tiles - 1 - u.tile) * u.splits + s) * heads + u.h;
}

struct PagedScan {
  long long warp_a[8], warp_b[8];
  PagedUnit unit;
  int found;
};

template <int THREADS>
__device__ __forceinline__ long long block_sum(long long x, long long* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  long long sum = 0;
#pragma unroll
  for (int j = 0; j < THREADS / 32; ++j) sum += scratch[j];
  return sum;
}

// Places `index` in the batch: unit `index` (MERGE = false) or split (query
// tile, K/V head) pair `index` (MERGE = true).  Every thread takes a run of
// sequences and returns the same answer; false if there is no such unit.
// Inside a sequence units run over K/V heads fastest, then chunks, then query
// tiles from the last (under a causal mask the one with the most keys), so
// the CTAs resident at a time walk the same keys.
template <int THREADS, bool MERGE>
__device__ __forceinline__ bool find_unit(const PagedParams& p, long long index, PagedScan* sh, PagedUnit& out) {
  const int tid = (int)threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (p.batch + THREADS - 1) / THREADS;
  const int i0 = min(tid * per, p.batch), i1 = min(i0 + per, p.batch);
  const bool report = !MERGE && blockIdx.x == 0;
  PagedSeq s;
  s.tiles = s.nv = 0;
  long long work = 0;
  for (int i = i0; i < i1; ++i) {
    s = paged_seq(p, i, report);
    work += (long long)s.tiles * s.nv;
  }
  if (tid == 0) sh->found = 0;
  work = block_sum<THREADS>(work, sh->warp_a) * p.heads_kv;
  const long long want = (work + p.target_units - 1) / p.target_units;
  const int chunk = (int)(want > p.min_chunk ? (want < INT_MAX ? want : INT_MAX) : p.min_chunk);
  // units (or split pairs) and slots before this thread's sequences
  long long n = 0, slots = 0;
  for (int i = i0; i < i1; ++i) {
    if (per > 1) s = paged_seq(p, i, false);
    const long long pairs = (long long)s.tiles * p.heads_kv;
    const int splits = tile_splits(s.nv, chunk);
    n += MERGE ? (splits > 1 ? pairs : 0) : pairs * splits;
    if (splits > 1) slots += pairs * splits;
  }
  long long in = n, is = slots;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, in, o), b = __shfl_up_sync(0xffffffffu, is, o);
    if (lane >= o) {
      in += a;
      is += b;
    }
  }
  __syncthreads();   // block_sum's reads of warp_a
  if (lane == 31) {
    sh->warp_a[w] = in;
    sh->warp_b[w] = is;
  }
  __syncthreads();
  long long at = in - n, slot = is - slots;
  for (int j = 0; j < w; ++j) {
    at += sh->warp_a[j];
    slot += sh->warp_b[j];
  }
  if (index >= at && index < at + n) {
    for (int i = i0; i < i1; ++i) {
      if (per > 1) s = paged_seq(p, i, false);
      const long long pairs = (long long)s.tiles * p.heads_kv;
      const int splits = tile_splits(s.nv, chunk);
      const long long mine = MERGE ? (splits > 1 ? pairs : 0) : pairs * splits;
      if (index < at + mine) {
        const int r = (int)(index - at);
        PagedUnit u;
        u.seq = i;
        u.row0 = s.row0;
        u.n_q = s.n_q;
        u.n_k = s.n_k;
        u.h = r % p.heads_kv;
        const int rest = r / p.heads_kv;
        u.split = MERGE ? 0 : rest % splits;
        u.tile = s.tiles - 1 - (MERGE ? rest : rest / splits);
        u.splits = splits;
        u.chunk = chunk;
        u.slot0 = (int)slot;
        // more slots than the workspace: only offsets that overlap lead here
        if (splits > 1 && slot + pairs * splits > p.max_slots) {
          if (!MERGE) atomicOr(p.status, kStatusBadSeqlens);
        } else {
          sh->unit = u;
          sh->found = 1;
        }
        break;
      }
      at += mine;
      if (splits > 1) slot += pairs * splits;
    }
  }
  __syncthreads();
  out = sh->unit;
  return sh->found != 0;
}

// A unit's place in its tile, beside DbufCtx (whose q0 / kv0 are not used).
struct PagedTile {
  int seq, h, row0;
  int q0;            // first token of the tile
  int rows;          // live rows: group x tokens
  int j0;            // first visited index of the unit
  TileWalk walk;
  int slot;          // partial slot, or -1: write O and L
};

// The TMA warp.  Lane l holds box l of a key tile: rows of page l % sub of the
// tile's `sub` pages, columns 64 (l / sub) ..
template <class C>
__device__ __forceinline__ void pg_producer(const DbufCtx& t, const PagedTile& u, const PagedParams& p,
                                            const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                            const CUtensorMap* tm_v, int lane) {
  const int ps = p.page_size;
  const int box_rows = min(ps, C::BC);
  const int sub = C::BC / box_rows;                 // pages per key tile, or 1
  const int tpp = ps > C::BC ? ps / C::BC : 1;      // key tiles per page, or 1
  const int my_sub = lane % sub, my_kb = lane / sub;
  const bool has_box = my_kb < C::D / 64;
  const int* row = p.table + (long long)u.seq * p.table_stride;
  bool bad = false;
  // Page of this lane's box of visited tile j: -1 when no row of the query
  // tile sees a key of it; an out-of-range page is reported and read as zeros
  // (num_pages lies outside the map).
  auto fetch = [&](int j) -> int {
    if (j >= t.nkv || !has_box) return -1;
    const int kt = u.walk.tile(u.j0 + j);
    const int k0 = kt * C::BC + my_sub * box_rows, k1 = k0 + box_rows;   // the box's keys
    if (!(k0 < t.km.pre_end || (k0 < u.walk.end && k1 > u.walk.lo))) return -1;
    const int page = __ldg(row + (sub > 1 ? kt * sub + my_sub : kt / tpp));
    if (page < 0 || page >= p.num_pages) {
      bad = true;
      return p.num_pages;
    }
    return page;
  };
  auto load = [&](uint32_t s_tile, uint32_t bar, const CUtensorMap* tm, int page, int j) {
    const unsigned boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * (uint32_t)box_rows * 128u);
    __syncwarp();
    if (page >= 0) {
      const int kt = u.walk.tile(u.j0 + j);
      tma_load_4d(s_tile + (uint32_t)my_kb * (C::BC * 128) + (uint32_t)(my_sub * box_rows) * 128u, tm, my_kb * 64,
                  tpp > 1 ? (kt % tpp) * C::BC : 0, u.h, page, bar);
    }
    __syncwarp();
  };
  int pg0 = fetch(0), pg1 = fetch(1), pg2 = fetch(2), pg3 = fetch(3);
  if (lane == 0) {
    mbar_arrive_expect_tx(t.bar(DB_Q), (uint32_t)(C::D / 64) * (uint32_t)p.slot_rows * 128u);
    for (int kb = 0; kb < C::D / 64; ++kb)
      tma_load_4d(t.sQ + kb * (C::BR * 128), tm_q, kb * 64, 0, u.h, u.row0 + u.q0, t.bar(DB_Q));
  }
  __syncwarp();
  // K_j is needed two products before V_j, and a K stage frees at S(j), before
  // PV(j) frees V's: K_0 V_0 K_1 V_1 K_2 (K_3 V_2) (K_4 V_3) ..
  load(t.sK, t.bar(DB_KFULL), tm_k, pg0, 0);
  load(t.sV, t.bar(DB_VFULL), tm_v, pg0, 0);
  int jk = 1, jv = 1;
  if (t.nkv > 1) {
    load(t.sK + C::KV_BYTES, t.bar(DB_KFULL + 1), tm_k, pg1, 1);
    load(t.sV + C::KV_BYTES, t.bar(DB_VFULL + 1), tm_v, pg1, 1);
    jk = jv = 2;
  }
  int prev = pg1;   // pages of tile j - 1
  pg0 = pg2;
  pg1 = pg3;
  pg2 = fetch(4);
  auto wait = [&](int bar, int phase) -> bool {
    bool ok = true;
    if (lane == 0)
      ok = wait_or_abort(t.bar(bar), (uint32_t)phase & 1, t.abort_flag, t.status, kSiteProducerEmpty);
    return __all_sync(0xffffffffu, ok);
  };
  for (int j = 2; j <= t.nkv; ++j) {   // pg0: pages of tile j
    const int ahead = fetch(j + 3);
    if (j < t.nkv) {
      const int s = j % C::KSTAGES, n = j / C::KSTAGES;
      if (!wait(DB_KEMPTY + s, n - 1)) break;
      load(t.sK + s * C::KV_BYTES, t.bar(DB_KFULL + s), tm_k, pg0, j);
      jk = j + 1;
    }
    if (j > 2) {
      const int jj = j - 1, s = jj % C::VSTAGES, n = jj / C::VSTAGES;
      if (!wait(DB_VEMPTY + s, n - 1)) break;
      load(t.sV + s * C::KV_BYTES, t.bar(DB_VFULL + s), tm_v, prev, jj);
      jv = jj + 1;
    }
    prev = pg0;
    pg0 = pg1;
    pg1 = pg2;
    pg2 = ahead;
  }
  if (bad) atomicOr(p.status, kStatusBadPages);
  // own copies in flight land before the CTA may exit
  if (lane == 0) {
    wait_drain(t.bar(DB_Q), 0, t.status);
    for (int s = 0; s < C::KSTAGES; ++s)
      if (jk > s) wait_drain(t.bar(DB_KFULL + s), (uint32_t)((jk - 1 - s) / C::KSTAGES) & 1, t.status);
    for (int s = 0; s < C::VSTAGES; ++s)
      if (jv > s) wait_drain(t.bar(DB_VFULL + s), (uint32_t)((jv - 1 - s) / C::VSTAGES) & 1, t.status);
  }
}

// Zeroes the rows of V tile `kt` (shared memory, 64 rows x D, 64-column blocks)
// whose keys no row of the query tile sees; 128 threads, thread `tid`.
template <class C>
__device__ __forceinline__ void zero_hidden_rows(uint32_t sV, int kt, const TileWalk& w, int pre_end, int tid) {
  for (int c = tid; c < C::BC * (C::D / 8); c += 128) {
    const int r = (c / 8) % C::BC, kb = c / (8 * C::BC);   // 16-byte chunk c % 8 of row r, column block kb
    const int key = kt * C::BC + r;
    if (key < pre_end || (key >= w.lo && key < w.end)) continue;
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sV + (uint32_t)kb * (C::BC * 128) +
                                                                   (uint32_t)r * 128u + (uint32_t)(c % 8) * 16u),
                 "r"(0u)
                 : "memory");
  }
}

// Output row r of a tile: the token's row, the query head's columns.
__device__ __forceinline__ uint8_t* paged_o_row(const PagedParams& p, int row, int head) {
  return reinterpret_cast<uint8_t*>(p.o) + 2 * ((long long)row * p.o_rs + (long long)head * p.o_hs);
}

template <class C, bool BF16, bool BAND>
__device__ __forceinline__ void pg_softmax(const DbufCtx& t, const PagedTile& u, const PagedParams& p, int warp,
                                           int lane) {
  const int quad = warp & 3;
  const int r = quad * 32 + lane;
  const bool live = r < u.rows;
  const bool warp_live = quad * 32 < u.rows;
  const int tok = r / p.group;
  const int row = u.q0 + tok;                        // token of the sequence
  const int head = u.h * p.group + (r - tok * p.group);
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  const uint32_t tO = t.tmem + lane_off + C::TMEM_O;
  const float sl2 = p.scale_log2_mag;
  const TileMask tmask = t.tm;
  const bool few_keys = t.few_keys;
  float m_run = -INFINITY;
  float l_run = 0.f;
  bool ok = true;
  if constexpr (C::Q_IN_TMEM) {
    // row r of Q_i into TMEM lane r, as in fa2_fwd_dbuf.cuh; rows past the
    // loaded box hold whatever was there, and reach only their own lanes
    ok = wait_or_abort(t.bar(DB_Q), 0, t.abort_flag, t.status, kSiteMmaQ);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      if (warp_live) {
#pragma unroll 1
        for (int kb = 0; kb < C::D / 64; ++kb) {
          const uint32_t src = t.sQ + kb * (C::BR * 128) + r * 128;
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = lds128(src + ((c ^ (r & 7)) << 4));
            w[4 * c] = x.x;
            w[4 * c + 1] = x.y;
            w[4 * c + 2] = x.z;
            w[4 * c + 3] = x.w;
          }
          tmem_st_32x32b_x32(t.tmem + lane_off + C::TMEM_Q + kb * 32, w);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(t.bar(DB_QT));
    }
  }
  for (int j = 0; ok && j < t.nkv; ++j) {
    const uint32_t tS = t.tmem + lane_off + C::TMEM_S + 64 * (j & 1);
    ok = wait_or_abort(t.bar(DB_S + (j & 1)), (uint32_t)(j >> 1) & 1, t.abort_flag, t.status, kSiteSoftmaxS);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    tc_fence_after();
    const bool masked = !tmask.full(j);
    const int kt = u.walk.tile(u.j0 + j);
    if (warp_live) {
      uint32_t sr[C::BC];
#pragma unroll
      for (int c = 0; c < C::BC; c += 32) tmem_ld_32x32b_x32(tS + c, sr + c);
#pragma unroll
      for (int c = 0; c < C::BC; c += 32) tmem_ld_wait_x32(sr + c);
      if (masked) mask_scores<C::BC, BAND>(sr, t.km, row, kt * C::BC);
      float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < C::BC; c += 8) {
        mx0 = fmax3(mx0, __uint_as_float(sr[c + 0]), __uint_as_float(sr[c + 1]));
        mx1 = fmax3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
        mx2 = fmax3(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
        mx3 = fmax3(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
      }
      const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
      const bool raise = live && m_tile > m_run + kRescaleLog2;
      const float m_new = raise ? m_tile : m_run;
      const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
      const float alpha = raise ? ex2_approx(m_run - m_use) : 1.f;
      const float2 scale2 = make_float2(sl2, sl2);
      const float2 neg_m2 = make_float2(-m_use, -m_use);
      float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
      if (split_tile<BF16>(masked, few_keys)) {
#pragma unroll
        for (int ch = 0; ch < C::BC / 32; ++ch)
          softmax_p_chunk<C, BF16, true>(sr, ch, tS, scale2, neg_m2, sum0, sum1);
      } else {
#pragma unroll
        for (int ch = 0; ch < C::BC / 32; ++ch)
          softmax_p_chunk<C, BF16, false>(sr, ch, tS, scale2, neg_m2, sum0, sum1);
      }
      const float2 sum2 = __fadd2_rn(sum0, sum1);
      l_run = l_run * alpha + (sum2.x + sum2.y);
      if (j > 0 && __any_sync(0xffffffffu, raise)) {
        // S(j) was issued before PV(j-1): wait for that product before rescaling
        bool ok2 = wait_or_abort(t.bar(DB_O), (uint32_t)(j - 1) & 1, t.abort_flag, t.status, kSiteSoftmaxO);
        ok2 = __all_sync(0xffffffffu, ok2);
        if (!ok2) {
          ok = false;
          break;
        }
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
    if (masked && !((kt + 1) * C::BC <= t.km.pre_end ||
                    (kt * C::BC >= u.walk.lo && (kt + 1) * C::BC <= u.walk.end))) {
      // some key of the tile is hidden from every row: its V row may be anything
      const int sv = j % C::VSTAGES;
      ok = wait_or_abort(t.bar(DB_VFULL + sv), (uint32_t)(j / C::VSTAGES) & 1, t.abort_flag, t.status, kSiteMmaV);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      zero_hidden_rows<C>(t.sV + sv * C::KV_BYTES, kt, u.walk, t.km.pre_end, r);
      fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(t.bar(DB_P + (j & 1)));
  }
  if (ok) {
    ok = wait_or_abort(t.bar(DB_OLAST), 0, t.abort_flag, t.status, kSiteEpilogueO);
    ok = __all_sync(0xffffffffu, ok);
  }
  if (!ok || !warp_live) return;
  tc_fence_after();
  if (u.slot >= 0) {
    const size_t slot = (size_t)u.slot * (size_t)p.slot_rows + (size_t)r;
    float4* dst = reinterpret_cast<float4*>(p.ws_o + slot * C::D);
#pragma unroll 1
    for (int c = 0; c < C::D; c += 32) {
      uint32_t o[32];
      tmem_ld_32x32b_x32(tO + c, o);
      tmem_ld_wait_x32(o);
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[c / 4 + i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                       __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
      }
    }
    if (live) *reinterpret_cast<float2*>(p.ws_ml + slot * 2) = make_float2(m_run, l_run);
    return;
  }
  const bool empty = !(l_run > 0.f);
  const float inv_l = empty ? 0.f : 1.f / l_run;
  uint8_t* o_row = paged_o_row(p, u.row0 + row, head);
#pragma unroll 1
  for (int c = 0; c < C::D; c += 32) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(tO + c, o);
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
    p.lse[(long long)head * p.lse_hs + u.row0 + row] =
        empty ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
}

// A unit without a key: O = 0 and L = -inf (whole tiles only: a split tile's
// chunks all have keys).
template <class C>
__device__ __forceinline__ void pg_store_empty(const PagedTile& u, const PagedParams& p, int tid) {
  constexpr int CH = C::D / 8;
  for (int i = tid; i < u.rows * CH; i += C::THREADS) {
    const int r = i / CH, tok = r / p.group;
    uint8_t* o_row = paged_o_row(p, u.row0 + u.q0 + tok, u.h * p.group + r - tok * p.group);
    reinterpret_cast<uint4*>(o_row)[i % CH] = make_uint4(0u, 0u, 0u, 0u);
  }
  for (int r = tid; r < u.rows; r += C::THREADS) {
    const int tok = r / p.group;
    p.lse[(long long)(u.h * p.group + r - tok * p.group) * p.lse_hs + u.row0 + u.q0 + tok] = -INFINITY;
  }
}

template <int D, bool BF16, bool BAND>
__global__ void __launch_bounds__(192, PagedConfig<D>::CTAS_PER_SM)
    fa2_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using C = PagedConfig<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  PagedScan* scan = reinterpret_cast<PagedScan*>(smem + C::OFF_MISC + 16);
  static_assert(16 + sizeof(PagedScan) <= C::MISC_BYTES, "shared-memory misc area");
  static_assert(C::OFF_MISC % 8 == 0, "scan alignment");
  const int warp = (int)(threadIdx.x >> 5);
  const int lane = (int)(threadIdx.x & 31);
  grid_launch_dependents();   // the merge may be scheduled once every unit has started; it waits for the partials

  // The whole CTA leaves together, before any barrier or TMEM set-up, when it
  // has no unit.
  PagedUnit un;
  if (!find_unit<C::THREADS, false>(p, (long long)blockIdx.x, scan, un)) return;
  DbufCtx t;
  PagedTile u;
  u.seq = un.seq;
  u.h = un.h;
  u.row0 = un.row0;
  u.q0 = un.tile * p.tile_tokens;
  const int last = min(u.q0 + p.tile_tokens, un.n_q) - 1;
  u.rows = (last + 1 - u.q0) * p.group;
  t.km = paged_mask(p, un.n_q, un.n_k);
  u.walk = tile_walk(t.km, u.q0, last);
  const int splits = tile_splits(u.walk.n, un.chunk);   // this tile's; at most the sequence's
  if (un.split >= splits) return;
  // equal chunks: the tile's n key tiles over its splits, none of them empty
  // (splits - 1 chunks of at most C tiles hold fewer than n)
  const int size = (u.walk.n + splits - 1) / splits;
  u.j0 = un.split * size;
  t.nkv = min(size, u.walk.n - u.j0);
  u.slot = -1;
  if (splits > 1) {
    const int tiles = (un.n_q + p.tile_tokens - 1) / p.tile_tokens;
    u.slot = unit_slot(un, tiles, p.heads_kv, un.split);
  }
  if (t.nkv == 0) {   // no row of the tile sees a key (a split tile's chunks all have some)
    pg_store_empty<C>(u, p, (int)threadIdx.x);
    return;
  }
  t.bar0 = sbase + C::OFF_BAR;
  t.sQ = sbase + C::OFF_Q;
  t.sK = sbase + C::OFF_K;
  t.sV = sbase + C::OFF_V;
  t.abort_flag = abort_flag;
  t.status = p.status;
  // key tiles every row sees, by visited index of this unit
  TileMask tm = tile_mask<BAND>(t.km, u.q0, last, C::BC);
  if (u.walk.npre == 0) tm.pre -= u.walk.skip;
  tm.lo -= u.walk.skip;
  tm.hi -= u.walk.skip;
  t.tm = tm.from(u.j0);
  t.few_keys = t.km.n_k <= 2 * C::BC;

  if (warp == C::TMA_WARP && lane == 0) {
    mbar_init(t.bar(DB_Q), 1);
    for (int s = 0; s < C::KSTAGES; ++s) {
      mbar_init(t.bar(DB_KFULL + s), 1);
      mbar_init(t.bar(DB_KEMPTY + s), 1);
    }
    for (int s = 0; s < C::VSTAGES; ++s) {
      mbar_init(t.bar(DB_VFULL + s), 1);
      mbar_init(t.bar(DB_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(t.bar(DB_S + s), 1);
      mbar_init(t.bar(DB_P + s), 4);
    }
    mbar_init(t.bar(DB_O), 1);
    mbar_init(t.bar(DB_OLAST), 1);
    mbar_init(t.bar(DB_EXIT), 1);
    mbar_init(t.bar(DB_QT), 4);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  t.tmem = *tmem_slot;

  if (warp == C::TMA_WARP) {
    pg_producer<C>(t, u, p, &tm_q, &tm_k, &tm_v, lane);
  } else if (warp == C::MMA_WARP) {
    KernelParams kp;
    kp.qk_negate = p.qk_negate;
    if (lane == 0) db_mma<C, BF16>(t, kp);
    __syncwarp();
  } else {
    pg_softmax<C, BF16, BAND>(t, u, p, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(t.tmem, C::TMEM_COLS);
  }
}

constexpr int kPagedMergeThreads = 128;
constexpr int kPagedMergeRows = 16;   // rows a block merges, four a warp

// One block per split (query tile, K/V head) and 16 of its rows: a warp per
// row, a lane per D / 32 columns, the chunks' states added in chunk order with
// the online softmax's rescaling.  The place of the block in the batch is
// found before the wait for the partials.
template <int D, bool BF16>
__global__ void __launch_bounds__(kPagedMergeThreads) fa2_paged_merge_kernel(const PagedParams p) {
  __shared__ PagedScan scan;
  PagedUnit u;
  const bool any = find_unit<kPagedMergeThreads, true>(p, (long long)blockIdx.x, &scan, u);
  grid_dependency_wait();   // the partials are complete and visible
  if (!any) return;
  const int q0 = u.tile * p.tile_tokens;
  const int last = min(q0 + p.tile_tokens, u.n_q) - 1;
  const int rows = (last + 1 - q0) * p.group;
  const KeyMask km = paged_mask(p, u.n_q, u.n_k);
  const int splits = tile_splits(tile_walk(km, q0, last).n, u.chunk);
  if (splits <= 1) return;   // its one unit has written O and L
  const int tiles = (u.n_q + p.tile_tokens - 1) / p.tile_tokens;
  const int slot0 = unit_slot(u, tiles, p.heads_kv, 0);
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  constexpr int E = D / 32;   // columns of a lane
  const int r1 = min(((int)blockIdx.y + 1) * kPagedMergeRows, rows);
  for (int r = (int)blockIdx.y * kPagedMergeRows + warp; r < r1; r += kPagedMergeThreads / 32) {
    float M = -INFINITY;
    for (int s = lane; s < splits; s += 32)
      M = fmaxf(M, p.ws_ml[((size_t)(slot0 + s * p.heads_kv) * p.slot_rows + r) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const size_t slot = (size_t)(slot0 + s * p.heads_kv) * p.slot_rows + r;
      const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + slot * 2);
      if (ml.x == -INFINITY) continue;   // a chunk that shows the row nothing: O~ is not read
      const float f = ex2_approx(ml.x - M);
      L = fmaf(f, ml.y, L);
      const float* src = p.ws_o + slot * D + lane * E;
      if constexpr (E == 2) {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(f, x.x, acc[0]);
        acc[1] = fmaf(f, x.y, acc[1]);
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(src + e);
          acc[e] = fmaf(f, x.x, acc[e]);
          acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
          acc[e + 2] = fmaf(f, x.z, acc[e + 2]);
          acc[e + 3] = fmaf(f, x.w, acc[e + 3]);
        }
      }
    }
    const bool empty = !(L > 0.f);
    const float inv_l = empty ? 0.f : 1.f / L;
    const int tok = r / p.group, head = u.h * p.group + r - tok * p.group;
    uint32_t* dst = reinterpret_cast<uint32_t*>(paged_o_row(p, u.row0 + q0 + tok, head)) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = empty ? 0u : pack2<BF16>(acc[e] * inv_l, acc[e + 1] * inv_l);
    if (lane == 0)
      p.lse[(long long)head * p.lse_hs + u.row0 + q0 + tok] =
          empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

template <int D, bool BF16, bool BAND>
int launch_paged_kernels(const PagedLaunchArgs& a) {
  using C = PagedConfig<D>;
  auto kern = fa2_paged_kernel<D, BF16, BAND>;
  static std::atomic<unsigned long long> configured{0};
  const int e = once_per_device(configured, [&]() -> int {
    return (int)cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_BYTES);
  });
  if (e != 0) return e;
  kern<<<(unsigned)a.grid, C::THREADS, C::SMEM_BYTES, a.stream>>>(a.tm_q, a.tm_k, a.tm_v, a.p);
  const cudaError_t r = cudaGetLastError();
  if (r != cudaSuccess) return (int)r;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.merge_tiles, (unsigned)((a.p.slot_rows + kPagedMergeRows - 1) / kPagedMergeRows));
  cfg.blockDim = dim3(kPagedMergeThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, fa2_paged_merge_kernel<D, BF16>, a.p);
}

template <int D>
int launch_paged(const PagedLaunchArgs& a) {
  if (a.band) return a.bf16 ? launch_paged_kernels<D, true, true>(a) : launch_paged_kernels<D, false, true>(a);
  return a.bf16 ? launch_paged_kernels<D, true, false>(a) : launch_paged_kernels<D, false, false>(a);
}

}  // namespace fa2
