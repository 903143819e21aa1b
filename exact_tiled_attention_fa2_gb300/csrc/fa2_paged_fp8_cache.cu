// fa2_paged_fp8_cache.cu -- the kernels that fill and read a paged key/value
// cache of 8-bit rows: rows of 16 bits quantised to their slots, and back.
//
// A row x (one token of one head) becomes codes c_i = e4m3(x_i * 2^-e) and the
// byte e + 127, with e the smallest integer that has max |x_i| <= 448 * 2^e.
// With max |x| = f * 2^n, f in [1, 2): 448 = 1.75 * 2^8, so e = n - 8, plus one
// if f > 1.75: read off the bits of the maximum as fp32.  x * 2^-e is exact in
// fp32, so each value is rounded once, to its code; code * 2^e has four
// significant bits and is exact in bf16, and in fp16 within e's limits there.
//
// Both kernels move 16 values of K and of V a thread and head, as pieces of 8 half
// a row apart, so that every access of a warp is made of whole runs; a head's row
// is d / 16 = 4, 8 or 16 neighbouring lanes, which find its maximum by shuffles.
// Reading is bound by HBM: 32768 rows of 8 heads x 128, 202 MB in 29 to 31 us (6.7
// TB/s; two heads a thread, so that enough loads are in flight; one, 32 us;
// neighbouring pieces a thread, whose stores half-fill their sectors, 41).  Writing
// is bound by HBM and its instructions together: the same rows in 33 us (44 with
// indexes computed at run time and every value clamped).
#include "fa2_paged_fp8.h"

#include <cuda_fp8.h>

#include "fa2_common.cuh"

namespace fa2 {
namespace {

constexpr int kRowThreads = 256;

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

// The row's exponent from its largest |value| (0: a row of zeros).
template <bool BF16>
__device__ __forceinline__ int row_exponent(float top) {
  const unsigned bits = __float_as_uint(top);
  int e = (int)(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = BF16 ? max(-60, min(e, 60)) : max(-15, min(e, 8));
  return top == 0.f ? 0 : e;
}

// The largest |value| of a word's two and of `top`'s, packed (a NaN is passed over).
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t top, uint32_t w) {
  const uint32_t m = w & 0x7fff7fffu;
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&top), *reinterpret_cast<const __nv_bfloat162*>(&m));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&top), *reinterpret_cast<const __half2*>(&m));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// A word's two values within 240 times the last power of two (a NaN stays).
template <bool BF16>
__device__ __forceinline__ uint32_t clamp2(uint32_t w) {
  if constexpr (BF16) {
    const __nv_bfloat162 hi = __float2bfloat162_rn(240.f * 1152921504606846976.f);   // 240 * 2^60
    const __nv_bfloat162 r = __hmax2_nan(__hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), hi), __hneg2(hi));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 hi = __float2half2_rn(61440.f);   // 240 * 2^8
    const __half2 r = __hmax2_nan(__hmin2_nan(*reinterpret_cast<const __half2*>(&w), hi), __hneg2(hi));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// A thread's 16 values of a row, 8 in each half.
struct Row16 {
  uint4 w[2];
};
struct Codes16 {
  uint2 c[2];
};

// Their codes; the row is shared by LANES lanes.  e: its exponent.
template <int LANES, bool BF16>
__device__ __forceinline__ Codes16 quantise16(const Row16& x, unsigned mask, int& e) {
  uint32_t w[8] = {x.w[0].x, x.w[0].y, x.w[0].z, x.w[0].w, x.w[1].x, x.w[1].y, x.w[1].z, x.w[1].w};
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top2 = max_abs2<BF16>(top2, w[i]);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) top2 = max_abs2<BF16>(top2, __shfl_xor_sync(mask, top2, o));
  const float2 tops = unpack2<BF16>(top2);
  const float top = fmaxf(tops.x, tops.y);
  e = row_exponent<BF16>(top);
  // x 2^-e is at most 448 unless e is at its end: there codes end at 240, past
  // which fp16 has no value for 2^8 code
  if (top > (BF16 ? 240.f * 1152921504606846976.f : 61440.f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = clamp2<BF16>(w[i]);
  }
  const float f = exp2_int(-e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(unpack2<BF16>(w[2 * i]), make_float2(f, f));
    const float2 z = __fmul2_rn(unpack2<BF16>(w[2 * i + 1]), make_float2(f, f));
    c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3) << 16;
  }
  return Codes16{{make_uint2(c[0], c[1]), make_uint2(c[2], c[3])}};
}

template <bool BF16>
__device__ __forceinline__ uint4 values8(const uint2& codes, float f) {
  const uint32_t c[2] = {codes.x, codes.y};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 y = __fmul2_rn(__half22float2(__half2(h)), make_float2(f, f));
    out[i] = pack2<BF16>(y.x, y.y);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Page and row of a slot.
struct SlotAt {
  long long page, row;
};
__device__ __forceinline__ SlotAt slot_at(const PagedFp8RowsArgs& a, int slot) {
  const int page = (int)((__umulhi((unsigned)slot, a.page_magic) + (unsigned)slot) >> a.page_shift);   // slot / page_size
  return SlotAt{page, slot - page * a.page_size};
}

// Threads x walk the pieces of a token's heads, threads y and the blocks the
// tokens.  (mask: the lanes that share the thread's row, whole rows at any item.)
// SM_BLOCKS: blocks an SM holds, which sets the registers: six with K's loads before
// V's, or three with all in flight together (8 heads x 128, three and six: 2047 rows
// 2.9 and 3.7 us, 4096 4.6 both, 6000 7.9 and 7.1, 32768 37.7 and 33.0).
template <int LANES, bool BF16, int SM_BLOCKS>
__global__ void __launch_bounds__(kRowThreads, SM_BLOCKS) fa2_paged_append_fp8_kernel(const PagedFp8RowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int items = a.heads * LANES;
  const int lane = (int)((threadIdx.y * blockDim.x + threadIdx.x) & 31);
  const unsigned mask = (unsigned)((1ull << LANES) - 1) << (lane & ~(LANES - 1));
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.total) return;
  const int slot = a.slots[t];
  const uint4 *kr = a.k.rows + t * a.k.row_rs, *vr = a.v.rows + t * a.v.row_rs;
  const bool skip = slot < 0 || slot >= a.num_slots;
  const SlotAt s = slot_at(a, skip ? 0 : slot);
  uint2 *kc = a.k.codes + s.page * a.k.code_ps + s.row * a.k.code_rs, *vc = a.v.codes + s.page * a.v.code_ps + s.row * a.v.code_rs;
  uint8_t *ke = a.k.exps + s.page * a.k.exp_ps + s.row, *ve = a.v.exps + s.page * a.v.exp_ps + s.row;
  for (int i = (int)threadIdx.x; i < items; i += (int)blockDim.x) {
    const int h = i / LANES, c = i % LANES;
    const uint4 *ks = kr + (h * a.k.row_hs + c), *vs = vr + (h * a.v.row_hs + c);
    const Row16 x = {{ks[0], ks[LANES]}}, y = {{vs[0], vs[LANES]}};
    if (skip) continue;
    int kx, vx;
    const Codes16 k = quantise16<LANES, BF16>(x, mask, kx), v = quantise16<LANES, BF16>(y, mask, vx);
    uint2 *kd = kc + (h * a.k.code_hs + c), *vd = vc + (h * a.v.code_hs + c);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      kd[j * LANES] = k.c[j];
      vd[j * LANES] = v.c[j];
    }
    if (c == 0) {
      ke[h * a.k.exp_hs] = (uint8_t)(kx + 127);
      ve[h * a.v.exp_hs] = (uint8_t)(vx + 127);
    }
  }
  if (slot >= a.num_slots && threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
}

template <int LANES, bool BF16>
__global__ void __launch_bounds__(kRowThreads, 4) fa2_paged_read_fp8_kernel(const PagedFp8RowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int items = a.heads * LANES, step = (int)blockDim.x;
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.total) return;
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) {
    if (slot >= 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
    return;
  }
  const SlotAt s = slot_at(a, slot);
  uint4 *kr = a.k.rows + t * a.k.row_rs, *vr = a.v.rows + t * a.v.row_rs;
  const uint2 *kc = a.k.codes + s.page * a.k.code_ps + s.row * a.k.code_rs, *vc = a.v.codes + s.page * a.v.code_ps + s.row * a.v.code_rs;
  const uint8_t *ke = a.k.exps + s.page * a.k.exp_ps + s.row, *ve = a.v.exps + s.page * a.v.exp_ps + s.row;
  for (int i0 = (int)threadIdx.x; i0 < items; i0 += 2 * step) {
    Codes16 x[2], y[2];
    unsigned kx[2], vx[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + u * step;
      if (i >= items) break;
      const int h = i / LANES, c = i % LANES;
      const uint2 *ks = kc + (h * a.k.code_hs + c), *vs = vc + (h * a.v.code_hs + c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[u].c[j] = ks[j * LANES];
        y[u].c[j] = vs[j * LANES];
      }
      kx[u] = ke[h * a.k.exp_hs];
      vx[u] = ve[h * a.v.exp_hs];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + u * step;
      if (i >= items) break;
      const int h = i / LANES, c = i % LANES;
      uint4 *kd = kr + (h * a.k.row_hs + c), *vd = vr + (h * a.v.row_hs + c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        kd[j * LANES] = values8<BF16>(x[u].c[j], __uint_as_float(kx[u] << 23));
        vd[j * LANES] = values8<BF16>(y[u].c[j], __uint_as_float(vx[u] << 23));
      }
    }
  }
}

struct RowsGrid {
  dim3 blocks, threads;
};
// each: items a thread.
RowsGrid rows_grid(int lanes, int each, const PagedFp8RowsArgs& a) {
  const int items = a.heads * lanes;
  int x = 16;   // a row's lanes lie in one warp
  while (x < kRowThreads && each * x < items) x *= 2;
  const int tokens = kRowThreads / x;   // of a block
  return RowsGrid{dim3((unsigned)(((long long)a.total + tokens - 1) / tokens)), dim3((unsigned)x, (unsigned)tokens)};
}

template <int LANES, int SM_BLOCKS>
int launch_append_rows(const RowsGrid& g, const PagedFp8RowsArgs& a, cudaStream_t stream) {
  return launch_chained(a.bf16 ? fa2_paged_append_fp8_kernel<LANES, true, SM_BLOCKS> : fa2_paged_append_fp8_kernel<LANES, false, SM_BLOCKS>,
                        g.blocks, g.threads, 0, stream, a);
}
template <int LANES>
int launch_append(const PagedFp8RowsArgs& a, cudaStream_t stream) {
  const RowsGrid g = rows_grid(LANES, 1, a);
  // up to twice what the GPU holds of three blocks an SM
  return g.blocks.x <= 2 * 3 * 152 ? launch_append_rows<LANES, 3>(g, a, stream) : launch_append_rows<LANES, 6>(g, a, stream);
}
template <int LANES>
int launch_read(const PagedFp8RowsArgs& a, cudaStream_t stream) {
  const RowsGrid g = rows_grid(LANES, 2, a);
  return launch_chained(a.bf16 ? fa2_paged_read_fp8_kernel<LANES, true> : fa2_paged_read_fp8_kernel<LANES, false>, g.blocks, g.threads, 0,
                        stream, a);
}

}  // namespace

int launch_paged_append_fp8(const PagedFp8RowsArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_append<4>(a, stream) : a.head_dim == 128 ? launch_append<8>(a, stream) : launch_append<16>(a, stream);
}

int launch_paged_read_fp8(const PagedFp8RowsArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_read<4>(a, stream) : a.head_dim == 128 ? launch_read<8>(a, stream) : launch_read<16>(a, stream);
}

}  // namespace fa2
