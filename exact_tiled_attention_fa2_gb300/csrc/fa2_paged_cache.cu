// fa2_paged_cache.cu -- the kernels that fill a paged key/value cache: one
// step's block tables and slot map from its request lengths, and new
// key/value rows written to their slots.
#include "fa2_paged.h"

#include <atomic>

#include "fa2_internal.h"
#include "sm103_ptx.cuh"

namespace fa2 {
namespace {

constexpr int kPlanThreads = 1024;   // of a block, at most

// Inclusive prefix sums of (a, b) over a warp's lanes.
__device__ __forceinline__ void warp_scan2(long long& a, long long& b, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long va = __shfl_up_sync(0xffffffffu, a, o), vb = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += va;
      b += vb;
    }
  }
}

// Exclusive prefix sums of (a, b) over the block's threads and their totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& total_a, long long& total_b,
                                            long long* scratch) {
  const int lane = (int)threadIdx.x & 31, w = (int)threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
  long long ia = a, ib = b;
  warp_scan2(ia, ib, lane);
  if (lane == 31) {
    scratch[2 * w] = ia;
    scratch[2 * w + 1] = ib;
  }
  __syncthreads();
  // the warps' sums, scanned by every warp
  long long wa = lane < warps ? scratch[2 * lane] : 0, wb = lane < warps ? scratch[2 * lane + 1] : 0;
  warp_scan2(wa, wb, lane);
  total_a = __shfl_sync(0xffffffffu, wa, 31);
  total_b = __shfl_sync(0xffffffffu, wb, 31);
  const long long before_a = __shfl_sync(0xffffffffu, wa, max(w - 1, 0));
  const long long before_b = __shfl_sync(0xffffffffu, wb, max(w - 1, 0));
  a = (w > 0 ? before_a : 0) + ia - a;
  b = (w > 0 ? before_b : 0) + ib - b;
}

// Last index i in [0, n) with x[i] <= v (x non-decreasing, x[0] <= v).
__device__ __forceinline__ int last_at_most(const int* x, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (x[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Every block sums all requests' new tokens and new pages (8 bytes a request,
// from L2 after the first block), so the blocks need nothing from each other:
// then each writes its part of the tokens' slots and of the new pages' table
// entries, finding an item's request by bisection in shared memory.  A slot
// in a new page comes from the free list itself, not from the table entry
// another block may still be writing.  Bound by latency (three reads that depend
// on each other, a scan, the bisection): 8 requests 2.9 us, 2048 with 103000
// tokens 6.5 us, 16000 decoding ones 12.9 us (48.7 with each thread reading its
// own run of requests).
__global__ void __launch_bounds__(kPlanThreads) fa2_paged_plan_kernel(const PagedPlanArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  extern __shared__ int sums[];             // [batch] first token, [batch] first new page
  __shared__ long long scratch[2 * kPlanThreads / 32];
  int* tok = sums;
  int* pag = sums + a.batch;
  const int tid = (int)threadIdx.x, threads = (int)blockDim.x;
  const unsigned ps = (unsigned)a.page_size;
  const int count = *a.free_count;
  // read side by side, summed in runs of an odd length (no two lanes of a warp
  // then meet in a bank)
  bool bad = false;
#pragma unroll 4
  for (int i = tid; i < a.batch; i += threads) {
    const long long c = a.context_lens[i], n = a.query_lens[i];
    const bool out = c < 0 || n < 0 || c + n > (long long)a.max_pages * ps;
    bad |= out;
    tok[i] = out ? 0 : (int)n;
    pag[i] = out ? 0 : (int)(((unsigned)(c + n) + ps - 1) / ps - ((unsigned)c + ps - 1) / ps);
  }
  const bool bad_any = __syncthreads_or(bad) != 0;
  const int per = (a.batch + threads - 1) / threads | 1;
  const int i0 = min(tid * per, a.batch), i1 = min(i0 + per, a.batch);
  long long n_tok = 0, n_pag = 0;
  for (int i = i0; i < i1; ++i) {
    n_tok += tok[i];
    n_pag += pag[i];
  }
  long long at_tok = n_tok, at_pag = n_pag, all_tok, all_pag;
  block_scan2(at_tok, at_pag, all_tok, all_pag, scratch);
  if (bad_any || all_tok > a.total_q || count < 0 || count > a.num_free || all_pag > count) {
    // refused: an empty step, the table and the free list as they were
    for (long long i = (long long)blockIdx.x * threads + tid; i < max(a.total_q, a.batch + 1);
         i += (int)gridDim.x * threads) {
      if (i < a.total_q) a.slots[i] = -1;
      if (i <= a.batch) a.cu_q[i] = 0;
      if (i < a.batch) a.lens_k[i] = 0;
    }
    if (blockIdx.x == 0 && tid == 0) {
      *a.free_left = count;
      atomicOr(a.status, kStatusBadPages);
    }
    return;
  }
  for (int i = i0; i < i1; ++i) {
    const int n = tok[i], w = pag[i];
    tok[i] = (int)at_tok;
    pag[i] = (int)at_pag;
    at_tok += n;
    at_pag += w;
  }
  __syncthreads();
  const int stride = (int)gridDim.x * threads, first = (int)blockIdx.x * threads + tid;
  for (int i = first; i < a.batch; i += stride) {
    a.cu_q[i] = tok[i];
    a.lens_k[i] = a.context_lens[i] + a.query_lens[i];
  }
  if (first == 0) {
    a.cu_q[a.batch] = (int)all_tok;
    *a.free_left = count - (int)all_pag;
  }
  bool bad_page = false;
  for (long long tl = first; tl < a.total_q; tl += stride) {
    const int t = (int)tl;
    int slot = -1;
    if (t < (int)all_tok) {
      const int b = last_at_most(tok, a.batch, t);
      const unsigned c = (unsigned)a.context_lens[b], pos = c + (unsigned)(t - tok[b]);
      const unsigned held = (c + ps - 1) / ps, page_at = pos / ps;
      const int page = page_at < held ? a.table[(long long)b * a.table_stride + page_at]
                                      : a.free_pages[count - 1 - (pag[b] + (int)(page_at - held))];
      if (page >= 0 && page < a.num_pages)
        slot = page * (int)ps + (int)(pos - page_at * ps);
      else
        bad_page = true;
    }
    a.slots[t] = slot;
  }
  for (long long nl = first; nl < all_pag; nl += stride) {
    const int n = (int)nl;
    const int b = last_at_most(pag, a.batch, n);
    const unsigned held = ((unsigned)a.context_lens[b] + ps - 1) / ps;
    const int page = a.free_pages[count - 1 - n];
    if (page < 0 || page >= a.num_pages) bad_page = true;
    a.table[(long long)b * a.table_stride + held + (unsigned)(n - pag[b])] = page;
  }
  if (bad_page) atomicOr(a.status, kStatusBadPages);
}

// Threads x walk the 16-byte chunks of a token's heads (a head's row is
// contiguous on both sides), threads y and the blocks the tokens: one each, its
// rows read beside its slot.  Bound by HBM: 32768 tokens of 8 heads x 128, 268
// MB in 41.1 us (6.53 TB/s).  The rows stay in the L2 as far as it holds them, for
// the forward that reads them (with loads and stores that pass it by, that call
// alone 42.5 us, and with the forward of prompts of 128 tokens 419 us, 416 so).
__global__ void __launch_bounds__(256) fa2_paged_append_kernel(const PagedAppendArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int items = a.heads << a.row_chunks_log2;
  const int mask = (1 << a.row_chunks_log2) - 1;
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.total) return;
  const int slot = a.slots[t];
  for (int i = (int)threadIdx.x; i < items; i += (int)blockDim.x) {
    const long long h = i >> a.row_chunks_log2;
    const int c = i & mask;
    const uint4 *ks = a.k.src + t * a.k.src_rs + h * a.k.src_hs + c, *vs = a.v.src + t * a.v.src_rs + h * a.v.src_hs + c;
    const uint4 x = *ks, y = *vs;
    if (slot < 0 || slot >= a.num_slots) continue;
    const long long page = slot / a.page_size, at = slot % a.page_size;
    uint4* kd = a.k.dst + page * a.k.dst_ps + at * a.k.dst_rs + h * a.k.dst_hs + c;
    uint4* vd = a.v.dst + page * a.v.dst_ps + at * a.v.dst_rs + h * a.v.dst_hs + c;
    *kd = x;
    *vd = y;
  }
  if (slot >= a.num_slots && threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
}

}  // namespace

int launch_paged_plan(const PagedPlanArgs& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  const int e = once_per_device(configured, [&]() -> int {
    return (int)cudaFuncSetAttribute(fa2_paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     2 * kPagedPlanMaxBatch * (int)sizeof(int));
  });
  if (e != 0) return e;
  // few requests: small blocks, whose scan is short
  const int threads = a.batch <= 256 ? 256 : kPlanThreads;
  long long blocks = ((long long)a.total_q + threads - 1) / threads;
  if (blocks > 152 * kPlanThreads / threads) blocks = 152 * kPlanThreads / threads;
  const size_t smem = 2 * (size_t)a.batch * sizeof(int);
  return launch_dependent(fa2_paged_plan_kernel, dim3((unsigned)blocks), threads, smem, stream, a);
}

int launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  const int items = a.heads << a.row_chunks_log2;
  int x = 8;
  while (x < 256 && x < items) x *= 2;
  const int tokens = 256 / x;   // of a block
  const unsigned blocks = (unsigned)(((long long)a.total + tokens - 1) / tokens);
  return launch_dependent(fa2_paged_append_kernel, dim3(blocks), dim3(x, tokens), 0, stream, a);
}

}  // namespace fa2
