// fa2_paged_shared.cuh -- paged attention of sequences that share the first pages
// of their prompts: fa2_paged_kernel twice, then one merge.
//
// A softmax over two sets of keys is joined from each set's (m, l, O~): m = max
// m_i, l = sum l_i 2^(m_i - m), O = sum O~_i 2^(m_i - m) / l.  So the keys that
// the sequences of a group share are attended once, with the group's query rows
// as one sequence's (128 rows of any of its requests a tile), and the rest by
// each sequence for itself.  Both passes leave fp32 partials of every pair; a
// row's lie in one pair of the group and one of its sequence, which differ in
// how many tokens they hold, so the merge takes row by row.
#pragma once

#include "fa2_paged.cuh"

namespace fa2 {

constexpr int kSharedMergeThreads = 256;
constexpr int kSharedMergeRows = 32;

// Where one pass's partials of a row are: partial k, column run c is at
// at + (slot(k) * runs + c) * slot_rows float4s.
struct SharedRow {
  const float4* o;
  const float2* ml;
  int slot_rows, count, first_slot, odd_first;   // slots first_slot + 2 k (k = 0: + odd_first)
  __device__ __forceinline__ size_t slot(int k) const {
    return (size_t)(first_slot + 2 * k + (k == 0 ? odd_first : 0)) * (size_t)slot_rows;
  }
};

// Row r of pair `id` of the pass p.
__device__ __forceinline__ SharedRow shared_row(const PagedParams& p, int id, int r) {
  SharedRow x;
  x.o = reinterpret_cast<const float4*>(p.ws_o) + r;
  x.ml = reinterpret_cast<const float2*>(p.ws_ml) + r;
  x.slot_rows = p.slot_rows;
  const PagedPair pair = p.pairs[id];
  x.count = 0;   // (a pass that gave up left no word: nothing outside the workspace is read)
  x.first_slot = x.odd_first = 0;
  if (pair.count == -1) {
    x.count = 1;
    x.first_slot = 2 * p.ctas + id;
  } else if (pair.count > 0 && pair.c0 >= 0 && pair.count <= p.ctas && pair.c0 <= p.ctas - pair.count) {
    x.count = pair.count;
    x.first_slot = 2 * pair.c0;
    x.odd_first = pair.from_start != 0;
  }
  return x;
}

// Block (b, y): of sequence b, chunk y of 32 rows of a K/V head, and on by the grid.  The lanes of a
// warp are rows x partials, its columns every eighth run of four, as in
// fa2_paged_merge_kernel.
template <int D, bool BF16>
__global__ void __launch_bounds__(kSharedMergeThreads)
    fa2_paged_shared_merge_kernel(const __grid_constant__ PagedParams shared, const __grid_constant__ PagedParams own) {
  constexpr int NW = kSharedMergeThreads / 32;
  constexpr int E = D / 4 / NW;   // column runs of a warp
  __shared__ uint2 stage[kSharedMergeRows][D / 4];
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int seq = (int)blockIdx.x, group = own.group, T = own.tile_tokens;
  grid_dependency_wait();   // both passes are complete and visible
  grid_launch_dependents();
  const SeqRead q = seq_read<true>(own, seq);
  const PagedSeq s = paged_seq<true>(own, q.a, q.b, q.k, false);
  if (s.tiles == 0) return;   // idle, or out of range
  int first, end, keys = 0, g_row = 0;
  const int g = group_of(own, seq, first, end);
  if (g >= 0) keys = group_keys(own, first, end, own.shared_lens[g]);
  if (keys > 0) g_row = own.cu_q[first];
  const int rows_all = s.n_q * group, chunks = (rows_all + kSharedMergeRows - 1) / kSharedMergeRows;
  for (int i = (int)blockIdx.y; i < chunks * own.heads_kv; i += (int)gridDim.y) {
    const int h = i % own.heads_kv, r0 = i / own.heads_kv * kSharedMergeRows;
    const int here = min(rows_all - r0, kSharedMergeRows);
    const int width_log2 = here <= 1 ? 0 : 32 - __clz(here - 1);   // lanes of rows
    const int r = lane & ((1 << width_log2) - 1), sub = lane >> width_log2, subs = 32 >> width_log2;
    const int at = r0 + min(r, here - 1), tok = at / group, in_group = at - tok * group;
    const int tile = tok / T;
    const SharedRow mine = shared_row(own, (s.row0 / T + seq + tile) * own.heads_kv + h, (tok - tile * T) * group + in_group);
    SharedRow theirs = mine;
    theirs.count = 0;
    if (keys > 0) {
      const int g_tok = s.row0 + tok - g_row, g_tile = g_tok / T;
      theirs = shared_row(shared, (g_row / T + g + g_tile) * own.heads_kv + h, (g_tok - g_tile * T) * group + in_group);
    }
    const int parts = mine.count + theirs.count;
    float m = -INFINITY, l = 0.f;
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = E <= 4 ? 2 : 1;   // partials whose reads are in flight together
#pragma unroll 1
    for (int k0 = r < here ? sub : parts; k0 < parts; k0 += U * subs) {
      float2 st[U];
      float4 v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * subs;
        st[u] = make_float2(-INFINITY, 0.f);
        if (k < parts) {
          const bool is_mine = k < mine.count;
          const SharedRow& x = is_mine ? mine : theirs;
          const size_t slot = x.slot(is_mine ? k : k - mine.count);
          st[u] = x.ml[slot];
          const float4* src = x.o + slot * (D / 4) + (size_t)warp * x.slot_rows;
#pragma unroll
          for (int e = 0; e < E; ++e) v[u][e] = src[(size_t)(e * NW) * x.slot_rows];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (st[u].y == 0.f) continue;   // shows the row nothing (a NaN sum stays)
        const float top = fmaxf(m, st[u].x);
        const float f0 = ex2_approx(m - top), f = ex2_approx(st[u].x - top);   // f0: 0 before the first
        m = top;
        l = l * f0 + st[u].y * f;
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
      if (warp == 0)
        own.lse[(long long)(h * group + in_group) * own.lse_hs + s.row0 + tok] =
            empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();
    for (int w = (int)threadIdx.x; w < here * (D / 8); w += kSharedMergeThreads) {
      const int row = w / (D / 8), c = w % (D / 8), t = (r0 + row) / group;
      reinterpret_cast<uint4*>(paged_o_row(own, s.row0 + t, h * group + r0 + row - t * group))[c] =
          reinterpret_cast<const uint4*>(stage[row])[c];
    }
    __syncthreads();
  }
}

template <int D, bool BF16>
int launch_paged_shared_pass(const PagedLaunchArgs& a) {
  if (a.wide) return launch_paged_kernel<D, BF16, false, true, false, true>(a);
  return a.p.batch <= 32 ? launch_paged_kernel<D, BF16, false, false, true, true>(a)
                         : launch_paged_kernel<D, BF16, false, false, false, true>(a);
}

template <int D, bool BF16>
int launch_paged_shared_all(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  static std::atomic<unsigned long long> configured{0};
  const int e = once_per_device(configured, [&]() -> int {
    return (int)cudaFuncSetAttribute(fa2_paged_shared_merge_kernel<D, BF16>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     100);
  });
  if (e != 0) return e;
  int r = launch_paged_shared_pass<D, BF16>(shared);
  if (r == 0) r = launch_paged_shared_pass<D, BF16>(own);
  if (r != 0) return r;
  const PagedParams& p = own.p;
  const long long chunks = ((long long)p.max_q * p.group + kSharedMergeRows - 1) / kSharedMergeRows;
  const long long most = chunks * p.heads_kv;
  const dim3 blocks((unsigned)p.batch, (unsigned)(most < 256 ? most : 256));
  return launch_chained(fa2_paged_shared_merge_kernel<D, BF16>, blocks, kSharedMergeThreads, 0, own.stream, shared.p, p);
}

template <int D>
int launch_paged_shared(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  return own.bf16 ? launch_paged_shared_all<D, true>(shared, own) : launch_paged_shared_all<D, false>(shared, own);
}

}  // namespace fa2
