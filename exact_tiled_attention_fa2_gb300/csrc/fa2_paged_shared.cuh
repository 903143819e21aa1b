// fa2_paged_shared.cuh -- paged attention of sequences that share the first pages
// of their prompts: the roles of fa2_paged.cuh over two lines of work, and a merge.
//
// A softmax over two sets of keys is joined from each set's (m, l, O~): m = max
// m_i, l = sum l_i 2^(m_i - m), O = sum O~_i 2^(m_i - m) / l.  So the keys that
// the sequences of a group share are attended once, with the group's query rows
// as one sequence's (128 rows of any of its requests a tile), and the rest by
// each sequence for itself.  Both passes leave fp32 partials of every pair; a
// row's lie in one pair of the group and one of its sequence, which differ in
// how many tokens they hold, so the merge takes row by row.
//
// Both passes are one launch: every CTA sums both lines, the wave of CTAs is
// divided between them by their lengths, and each takes a piece of one.  The query
// tiles of a group read the same keys, so each tile's line starts with a piece:
// the tiles are then cut at the same keys, and the CTAs side by side read them
// together, from the L2 cache all but the first.
#pragma once

#include "fa2_paged.cuh"

namespace fa2 {

constexpr int kSharedMergeThreads = 256;
constexpr int kSharedMergeRows = 32;

// Where one pass's partials of a row are: slots first + 2 k (k = 0: + odd), row
// `row` of each.
struct SharedRow {
  int count, first, odd, row;
};

// Row `row` of pair `id` of the pass p.
__device__ __forceinline__ SharedRow shared_row(const PagedParams& p, int id, int row) {
  const PagedPair pair = p.pairs[id];
  SharedRow x;
  x.count = x.first = x.odd = 0;   // (a pass that gave up left no word: nothing outside the workspace is read)
  x.row = row;
  if (pair.count == -1) {
    x.count = 1;
    x.first = 2 * p.ctas + id;
  } else if (pair.count > 0 && pair.c0 >= 0 && pair.count <= p.ctas && pair.c0 <= p.ctas - pair.count) {
    x.count = pair.count;
    x.first = 2 * pair.c0;
    x.odd = pair.from_start != 0;
  }
  return x;
}

// Up to 32 groups: the line of shared keys with every query tile's stretch starting
// at a piece.  Each warp finds the same, lane g for group g.
template <bool WIDE>
struct GroupLine {
  using Line = typename LineOf<WIDE>::T;
  PagedSeq s;          // the lane's group
  int first;           // its first sequence
  Line stretch;        // of one of its query tiles, all K/V heads
  long long total;     // all stretches, in keys
  int tiles;           // of all groups
};

template <bool WIDE>
__device__ __forceinline__ GroupLine<WIDE> group_line(const PagedParams& p, bool report) {
  const int lane = (int)threadIdx.x & 31;
  GroupLine<WIDE> g;
  g.s.tiles = g.s.keys = g.s.n_q = g.s.n_k = g.s.row0 = 0;
  g.stretch = 0;
  g.first = 0;
  if (lane < p.batch) {
    g.first = p.cu_groups[lane];
    g.s = read_seq<WIDE, 1>(p, lane, report);
    if (g.s.tiles > 0) g.stretch = (typename LineOf<WIDE>::T)g.s.template width<WIDE>(p, 0) * p.heads_kv;
  }
  g.total = (long long)g.stretch * g.s.tiles * LineOf<WIDE>::KEYS;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) g.total += __shfl_xor_sync(0xffffffffu, g.total, o);
  g.tiles = __reduce_add_sync(0xffffffffu, g.s.tiles);
  return g;
}

// The shortest piece that gives at most `ctas` pieces, at least p.tiles of them;
// `pieces`: of one of the lane's tiles, `all`: of all.  From an even share up, to
// the next length at which some group's tiles take a piece less.
template <bool WIDE>
__device__ __forceinline__ typename LineOf<WIDE>::T group_share(const PagedParams& p, const GroupLine<WIDE>& g, int ctas,
                                                                int& pieces, int& all) {
  using Line = typename LineOf<WIDE>::T;
  Line share = max((Line)(p.min_share / LineOf<WIDE>::KEYS), (Line)((g.total / LineOf<WIDE>::KEYS + ctas - 1) / ctas));
#pragma unroll 1
  for (int step = 0;; ++step) {
    pieces = (int)line_div(g.stretch + share - 1, share);
    all = __reduce_add_sync(0xffffffffu, pieces * g.s.tiles);
    if (all <= ctas) return share;
    Line next = pieces > 1 ? line_div(g.stretch + pieces - 2, (Line)(pieces - 1)) : LineOf<WIDE>::MOST;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) next = min(next, __shfl_xor_sync(0xffffffffu, next, o));
    share = max(next, step < 24 ? share + 1 : share + share / 4);   // (many groups: a bounded search)
  }
}

// CTA `block`'s piece of that line: pieces of the tiles side by side.
template <bool WIDE>
__device__ __forceinline__ PagedPlace<WIDE> group_place(const PagedParams& p, const GroupLine<WIDE>& g, int block,
                                                        typename LineOf<WIDE>::T share, int pieces) {
  using Line = typename LineOf<WIDE>::T;
  const int lane = (int)threadIdx.x & 31, mine = pieces * g.s.tiles;
  int end = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  const unsigned holds = __ballot_sync(0xffffffffu, block >= end - mine && block < end);
  PagedPlace<WIDE> r;
  r.seq = __ffs(holds) - 1;   // -1: none
  const int src = max(r.seq, 0), start = __shfl_sync(0xffffffffu, end - mine, src);
  r.s.row0 = __shfl_sync(0xffffffffu, g.s.row0, src);
  r.s.n_q = __shfl_sync(0xffffffffu, g.s.n_q, src);
  r.s.n_k = __shfl_sync(0xffffffffu, g.s.n_k, src);
  r.s.tiles = __shfl_sync(0xffffffffu, g.s.tiles, src);
  r.s.keys = __shfl_sync(0xffffffffu, g.s.keys, src);
  const int of_tile = __shfl_sync(0xffffffffu, pieces, src);
  const Line stretch = __shfl_sync(0xffffffffu, g.stretch, src);
  const int at = block - start, tiles = max(r.s.tiles, 1), piece = at / tiles;
  r.tile = at - piece * tiles;
  r.piece = start + r.tile * of_tile + piece;
  r.at = (Line)(start + r.tile * of_tile) * share;
  r.share = share;
  r.total = r.at + stretch;
  r.rank = 0;
  r.skip = __shfl_sync(0xffffffffu, g.first, src);
  r.line = true;
  return r;
}

// CTAs of `ctas` that take the shared keys, whole units and `limit` at most: `group`
// and `own` are the lines' lengths in keys.  Rounded down, for a short line of the
// sequences' own suffers more from a unit less (two requests behind 20000 shared
// keys: 39.8 us, rounded to the nearest 51.4).
__device__ __forceinline__ int shared_ctas(const PagedParams& pa, long long group, long long own, int ctas, int limit,
                                           int unit) {
  if (group == 0) return 0;
  const float a = (float)group * pa.share_weight, b = (float)own;
  const int n = max((int)((float)(ctas / unit) * a / (a + b)), 1) * unit;
  const long long most = (group + pa.min_share - 1) / pa.min_share;   // pieces there are
  return max(1, min(min(n, limit), (int)(most < limit ? most : limit)));
}

template <class C, bool BF16, int PASS>
__device__ __forceinline__ void shared_roles(const PagedCtx<C>& t, const PagedParams& p, const CUtensorMap* tm_q,
                                             const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                             const PagedPlace<C::WIDE>& place, int warp, int lane) {
  if (place.seq < 0) return;   // nothing for this CTA
  if (warp == C::TMA_WARP) {
    pg_load<C, false, PASS>(t, p, tm_q, tm_k, tm_v, place, lane);
  } else if (warp == C::MMA_WARP) {
    if (lane == 0) pg_mma<C, BF16>(t, p);
    __syncwarp();
  } else if (warp == C::PLAN_WARP) {
    if constexpr (C::PLANNER) pg_plan<C, false, PASS>(t, p, place, lane);
  } else {
    pg_softmax<C, BF16, false>(t, p, warp, lane);
  }
}

// WA, WB: many rows (PagedConfig) in the pass over the shared keys, over the
// sequences' own.  Where two CTAs fit an SM they are the two halves of one block
// here, each a CTA of fa2_paged_kernel with its own shared and tensor memory, and
// blocks come in clusters of two, the SMs of a TPC; all of these are of the same
// pass: the code of both does not fit the instruction caches that they share (128
// requests behind 32000 shared keys: the shared pass ends at 97 us on TPCs of that
// pass alone, at 150 beside an SM of the other, at 164 on an SM with both).
template <int D, bool WA, bool WB>
struct SharedConfig {
  using A = PagedConfig<D, WA>;
  using B = PagedConfig<D, WB>;
  static constexpr int HALVES = B::CTAS_PER_SM;
  static constexpr int CLUSTER = 2;
  static constexpr int UNIT = HALVES * CLUSTER;   // CTAs of one pass together
  static constexpr int HALF_THREADS = A::THREADS > B::THREADS ? A::THREADS : B::THREADS;
  static constexpr int THREADS = HALVES * HALF_THREADS;
  static constexpr uint32_t HALF_BYTES = (B::SMEM_BYTES - 1024 + 1023) / 1024 * 1024;
  static constexpr uint32_t SMEM_BYTES = HALVES * HALF_BYTES + 1024;
  static_assert(A::OFF_BAR == B::OFF_BAR && A::OFF_SCAN == B::OFF_SCAN && A::SMEM_BYTES == B::SMEM_BYTES &&
                    A::TMEM_COLS == B::TMEM_COLS && A::CTAS_PER_SM == B::CTAS_PER_SM,
                "one layout");
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

template <int D, bool BF16, bool WA, bool WB>
__global__ void __launch_bounds__(SharedConfig<D, WA, WB>::THREADS, 1)
    fa2_paged_shared_kernel(const __grid_constant__ CUtensorMap tm_qa, const __grid_constant__ CUtensorMap tm_qb,
                            const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ PagedParams pa, const __grid_constant__ PagedParams pb) {
  using S = SharedConfig<D, WA, WB>;
  using A = typename S::A;
  using B = typename S::B;
  extern __shared__ uint8_t smem_raw[];
  const int half = S::HALVES == 1 ? 0 : (int)threadIdx.x / S::HALF_THREADS;
  const int tid = (int)threadIdx.x - half * S::HALF_THREADS;
  // a softmax warp is the one that can reach its quarter of tensor memory's lanes
  const int warp = (tid >> 5) < 4 ? (int)(threadIdx.x >> 5) & 3 : tid >> 5, lane = tid & 31;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* block_smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* smem = block_smem + half * S::HALF_BYTES;
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(block_smem + B::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + B::OFF_MISC + 4);
  if (warp == B::TMA_WARP && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < PG_BARS; ++i)   // as fa2_paged_kernel
      mbar_init(sbase + B::OFF_BAR + 8u * (uint32_t)i, (i >= PG_P && i < PG_EXIT) || i >= PG_FREE ? 4 : 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_qa);
    tma_prefetch_desc(&tm_qb);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_dependency_wait();   // what precedes this kernel is complete
  grid_launch_dependents();   // so the merge may read lengths and groups; for the partials it waits
  if (half == 0 && warp == B::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), S::HALVES * B::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  // the line of shared keys: by query tile, or (more than 32 groups, or more query tiles than CTAs) as it falls
  const bool first = blockIdx.x == 0 && half == 0;
  constexpr int SCAN_THREADS = S::HALF_THREADS - 32;
  const int ctas = (int)gridDim.x * S::HALVES, limit = ctas - S::UNIT;   // the rest for the other pass
  // (each half's last warp looks at the groups while the others sum the sequences)
  PagedScan<WA>* scan_a = reinterpret_cast<PagedScan<WA>*>(smem + A::OFF_SCAN);
  PagedScan<WB>* scan_b = reinterpret_cast<PagedScan<WB>*>(smem + B::OFF_SCAN);
  GroupLine<WA>* found = reinterpret_cast<GroupLine<WA>*>(smem);   // of each lane; Q is not there yet
  static_assert(32 * sizeof(GroupLine<WA>) <= B::Q_BYTES, "room for the groups");
  const LineScan<WB> own_scan = line_scan<SCAN_THREADS, WB, 2>(pb, tid, scan_b, first, [&] {
    if (pa.batch <= 32) found[lane] = group_line<WA>(pa, first);
  });
  GroupLine<WA> groups;
  groups.tiles = 0;
  groups.total = 0;
  if (pa.batch <= 32) groups = found[lane];
  const bool by_tile = groups.tiles > 0 && groups.tiles <= limit;
  const bool as_it_falls = pa.batch > 32 || groups.tiles > limit;
  LineScan<WA> group_scan;
  fence_proxy_async_smem();
  __syncthreads();   // read by all before Q lands there
  if (as_it_falls) {
    group_scan = line_scan<SCAN_THREADS, WA, 1>(pa, tid, scan_a, first && pa.batch > 32, [] {});
    groups.total = (long long)group_scan.total * LineOf<WA>::KEYS;
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot + (uint32_t)half * B::TMEM_COLS;
  int group_ctas = shared_ctas(pa, groups.total, (long long)own_scan.total * LineOf<WB>::KEYS, ctas, limit, S::UNIT), pieces = 0;
  typename LineOf<WA>::T share = 0;
  if (by_tile) share = group_share<WA>(pa, groups, max(group_ctas, groups.tiles), pieces, group_ctas);
  const int group_blocks = (group_ctas + S::UNIT - 1) / S::UNIT * S::CLUSTER;
  auto context = [&](auto& t, const PagedParams& p) {
    t.bar0 = sbase + B::OFF_BAR;
    t.sQ = sbase + B::OFF_Q;
    t.sK = sbase + B::OFF_K;
    t.sV = sbase + B::OFF_V;
    t.tmem = tmem;
    t.abort_flag = abort_flag;
    t.status = p.status;
    t.frags = reinterpret_cast<PagedFrag*>(smem + B::OFF_FRAG);
  };
  if ((int)blockIdx.x < group_blocks) {
    PagedCtx<A> t;
    context(t, pa);
    const int at = (int)blockIdx.x * S::HALVES + half;
    PagedPlace<WA> place;
    if (by_tile) {
      place = group_place<WA>(pa, groups, at, share, pieces);
    } else {
      place = line_place<WA, 1>(pa, group_scan, at, group_ctas, scan_a);
      place.tile = -1;
      if (at >= group_ctas) place.seq = -1;
    }
    shared_roles<A, BF16, 1>(t, pa, &tm_qa, &tm_k, &tm_v, place, warp, lane);
  } else {
    PagedCtx<B> t;
    context(t, pb);
    const int at = ((int)blockIdx.x - group_blocks) * S::HALVES + half;
    if (as_it_falls) {   // (the other line's scan was there)
      __syncthreads();
      if (tid == 0) scan_b->place.seq = -1;
      __syncthreads();
    }
    const PagedPlace<WB> place = line_place<WB, 2>(pb, own_scan, at, ctas - group_blocks * S::HALVES, scan_b);
    shared_roles<B, BF16, 2>(t, pb, &tm_qb, &tm_k, &tm_v, place, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (half == 0 && warp == B::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, S::HALVES * B::TMEM_COLS);
  }
}

// Block (b, y): of sequence b's rows, those of one K/V head after those of another,
// chunk y of `chunk`, and on by the grid.  The first warp finds where the rows'
// partials are, a row a lane (every warp for itself: 820 instructions a warp, most
// of a merge's 15 us).  The lanes of a warp are then rows x partials, its columns
// every eighth run of four, as in fa2_paged_merge_kernel.  (With two partials of a
// lane in flight 64 requests behind 8200 keys take 60.1 us in place of 57.1, chunks
// at d = 256 103 in place of 82.)
template <int D, bool BF16>
__global__ void __launch_bounds__(kSharedMergeThreads, D == 256 ? 3 : 4)
    fa2_paged_shared_merge_kernel(const __grid_constant__ PagedParams shared, const __grid_constant__ PagedParams own,
                                  int chunk) {
  constexpr int NW = kSharedMergeThreads / 32;
  constexpr int E = D / 4 / NW;   // column runs of a warp
  __shared__ uint2 stage[kSharedMergeRows][D / 4];
  __shared__ SharedRow rows[2][kSharedMergeRows];   // of the sequence's own keys, of the shared ones
  __shared__ long long o_at[kSharedMergeRows], lse_at[kSharedMergeRows];
  __shared__ OwnRead seq_of;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int seq = (int)blockIdx.x, group = own.group, T = own.tile_tokens;
  // lengths and groups, while the passes still run: what wrote them is complete when
  // this kernel is let in
  if (threadIdx.x == 0) {
    OwnRead q = own_read(own, seq);
    const PagedSeq s = paged_seq<true>(own, q.s.a, q.s.b, q.s.k, false);
    if (s.tiles == 0) q.s.b = q.s.a;   // idle, or out of range
    seq_of = q;
  }
  __syncthreads();
  const int row0 = seq_of.s.a, each = (seq_of.s.b - row0) * group, rows_all = each * own.heads_kv;   // each: of a K/V head
  grid_dependency_wait();   // both passes are complete and visible
  grid_launch_dependents();
  for (int r0 = (int)blockIdx.y * chunk; r0 < rows_all; r0 += (int)gridDim.y * chunk) {
    const int here = min(rows_all - r0, chunk);
    if (warp == 0 && lane < here) {
      const int h = (r0 + lane) / each, at = r0 + lane - h * each, tok = at / group, in_group = at - tok * group, tile = tok / T;
      rows[0][lane] = shared_row(own, (row0 / T + seq + tile) * own.heads_kv + h, (tok - tile * T) * group + in_group);
      SharedRow x;
      x.count = x.first = x.odd = x.row = 0;
      if (seq_of.keys > 0) {
        const int g_tok = row0 + tok - seq_of.group_row, g_tile = g_tok / T;
        x = shared_row(shared, (seq_of.group_row / T + seq_of.group + g_tile) * own.heads_kv + h,
                       (g_tok - g_tile * T) * group + in_group);
      }
      rows[1][lane] = x;
      const long long head = h * group + in_group;
      o_at[lane] = (long long)(row0 + tok) * own.o_rs + head * own.o_hs;
      lse_at[lane] = head * own.lse_hs + row0 + tok;
    }
    __syncthreads();
    const int width_log2 = here <= 1 ? 0 : 32 - __clz(here - 1);   // lanes of rows
    const int r = lane & ((1 << width_log2) - 1), sub = lane >> width_log2, subs = 32 >> width_log2;
    const SharedRow mine = rows[0][min(r, here - 1)], theirs = rows[1][min(r, here - 1)];
    const int parts = mine.count + theirs.count;
    float m = -INFINITY, l = 0.f;
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k = r < here ? sub : parts; k < parts; k += subs) {
      const bool is_mine = k < mine.count;
      const SharedRow& x = is_mine ? mine : theirs;
      const PagedParams& p = is_mine ? own : shared;
      const int n = is_mine ? k : k - mine.count;
      const size_t slot = (size_t)(x.first + 2 * n + (n == 0 ? x.odd : 0)) * (size_t)p.slot_rows;
      const float2 st = reinterpret_cast<const float2*>(p.ws_ml)[slot + x.row];
      const float4* src = reinterpret_cast<const float4*>(p.ws_o) + slot * (D / 4) + (size_t)(warp * p.slot_rows + x.row);
      float4 v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = src[(size_t)(e * NW) * p.slot_rows];
      if (st.y == 0.f) continue;   // shows the row nothing (a NaN sum stays)
      const float top = fmaxf(m, st.x);
      const float f0 = ex2_approx(m - top), f = ex2_approx(st.x - top);   // f0: 0 before the first
      m = top;
      l = l * f0 + st.y * f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[e].x = fmaf(f, v[e].x, acc[e].x * f0);
        acc[e].y = fmaf(f, v[e].y, acc[e].y * f0);
        acc[e].z = fmaf(f, v[e].z, acc[e].z * f0);
        acc[e].w = fmaf(f, v[e].w, acc[e].w * f0);
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
      if (warp == 0) own.lse[lse_at[r]] = empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();
    for (int w = (int)threadIdx.x; w < here * (D / 8); w += kSharedMergeThreads) {
      const int row = w / (D / 8), c = w % (D / 8);
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(own.o) + o_at[row])[c] = reinterpret_cast<const uint4*>(stage[row])[c];
    }
    __syncthreads();
  }
}

template <int D, bool BF16, bool WA, bool WB>
int launch_paged_shared_kernels(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  using S = SharedConfig<D, WA, WB>;
  auto kern = fa2_paged_shared_kernel<D, BF16, WA, WB>;
  static std::atomic<unsigned long long> configured{0};
  const int e = once_per_device(configured, [&]() -> int {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM_BYTES);
    if (r != cudaSuccess) return (int)r;
    cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    return (int)cudaFuncSetAttribute(fa2_paged_shared_merge_kernel<D, BF16>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     100);
  });
  if (e != 0) return e;
  const PagedParams& p = own.p;
  const int r = launch_dependent_clusters(kern, S::CLUSTER, dim3((unsigned)(p.ctas / S::HALVES)), S::THREADS, S::SMEM_BYTES,
                                          own.stream, shared.tm_q, own.tm_q, own.tm_k, own.tm_v, shared.p, p);
  if (r != 0) return r;
  // few rows a block while the blocks fit the GPU at once (four an SM): 2048 rows
  // 58.0 us the call at 4, 59.4 at 8, 70.7 at 32; 4096 rows 110, 106, 119; 7000 rows
  // of d = 256 96, 86, 81
  const long long all = (long long)p.total_q * p.group * p.heads_kv;
  const int chunk = all <= 600 * 4 ? 4 : all <= 600 * 8 ? 8 : kSharedMergeRows;
  const long long most = ((long long)p.max_q * p.group * p.heads_kv + chunk - 1) / chunk;
  const dim3 blocks((unsigned)p.batch, (unsigned)(most < 256 ? most : 256));
  return launch_chained(fa2_paged_shared_merge_kernel<D, BF16>, blocks, kSharedMergeThreads, 0, own.stream, shared.p, p, chunk);
}

template <int D, bool BF16>
int launch_paged_shared_rows(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  if (own.wide) return launch_paged_shared_kernels<D, BF16, true, true>(shared, own);
  return shared.wide ? launch_paged_shared_kernels<D, BF16, true, false>(shared, own)
                     : launch_paged_shared_kernels<D, BF16, false, false>(shared, own);
}

template <int D>
int launch_paged_shared(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  return own.bf16 ? launch_paged_shared_rows<D, true>(shared, own) : launch_paged_shared_rows<D, false>(shared, own);
}

}  // namespace fa2
