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
// Both kernels move 16 codes a thread (32 bytes of 16-bit values), K and V
// together; a head's row is d / 16 = 4, 8 or 16 neighbouring lanes, which find
// its maximum by shuffles.  Bound by HBM.
#include "fa2_paged_fp8.h"

#include <cuda_fp8.h>

#include "fa2_common.cuh"

namespace fa2 {
namespace {

constexpr int kRowThreads = 256;

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

template <bool BF16>
__device__ __forceinline__ void widen16(const uint4 (&w)[2], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<BF16>(u[j]);
      x[8 * i + 2 * j] = f.x;
      x[8 * i + 2 * j + 1] = f.y;
    }
  }
}

// The row's exponent from its largest |value| (0: a row of zeros).
template <bool BF16>
__device__ __forceinline__ int row_exponent(float top) {
  const unsigned bits = __float_as_uint(top);
  int e = (int)(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = BF16 ? max(-60, min(e, 60)) : max(-15, min(e, 8));
  return top == 0.f ? 0 : e;
}

// 16 codes of the row that `lanes` lanes share; e: its exponent.
template <bool BF16>
__device__ __forceinline__ uint4 quantise16(const uint4 (&w)[2], int lanes, unsigned mask, int& e) {
  float x[16];
  widen16<BF16>(w, x);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));   // a NaN is passed over
  for (int o = 1; o < lanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
  e = row_exponent<BF16>(top);
  // at the last exponent codes end at 240: past it fp16 has no value for 2^8 * code
  const float lim = e == (BF16 ? 60 : 8) ? 240.f : 448.f;
  const float f = exp2_int(-e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 y = make_float2(x[4 * i + 2 * j] * f, x[4 * i + 2 * j + 1] * f);
      // (a NaN fails both comparisons and stays)
      y.x = y.x > lim ? lim : y.x < -lim ? -lim : y.x;
      y.y = y.y > lim ? lim : y.y < -lim ? -lim : y.y;
      u |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * j);
    }
    c[i] = u;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

template <bool BF16>
__device__ __forceinline__ void values16(const uint4& codes, float f, uint4 (&w)[2]) {
  const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[i] >> (16 * j)), __NV_E4M3);
      const float2 y = __half22float2(__half2(h));
      out[2 * i + j] = pack2<BF16>(y.x * f, y.y * f);
    }
  }
  w[0] = make_uint4(out[0], out[1], out[2], out[3]);
  w[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// Threads x walk the 16-code chunks of a token's heads, threads y and the blocks
// the tokens.
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) fa2_paged_append_fp8_kernel(const PagedFp8RowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lanes = 1 << a.chunks_log2, items = a.heads << a.chunks_log2;
  const int lane = (int)((threadIdx.y * blockDim.x + threadIdx.x) & 31);
  const unsigned mask = (unsigned)((1ull << lanes) - 1) << (lane & ~(lanes - 1));   // the row's lanes
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.total) return;
  const int slot = a.slots[t];
  for (int i = (int)threadIdx.x; i < items; i += (int)blockDim.x) {
    const long long h = i >> a.chunks_log2;
    const int c = i & (lanes - 1);
    const uint4* ks = a.k.rows + t * a.k.row_rs + h * a.k.row_hs + 2 * c;
    const uint4* vs = a.v.rows + t * a.v.row_rs + h * a.v.row_hs + 2 * c;
    const uint4 x[2] = {ks[0], ks[1]}, y[2] = {vs[0], vs[1]};
    if (slot < 0 || slot >= a.num_slots) continue;
    int ke, ve;
    const uint4 kc = quantise16<BF16>(x, lanes, mask, ke), vc = quantise16<BF16>(y, lanes, mask, ve);
    const long long page = slot / a.page_size, at = slot % a.page_size;
    a.k.codes[page * a.k.code_ps + h * a.k.code_hs + at * a.k.code_rs + c] = kc;
    a.v.codes[page * a.v.code_ps + h * a.v.code_hs + at * a.v.code_rs + c] = vc;
    if (c == 0) {
      a.k.exps[page * a.k.exp_ps + h * a.k.exp_hs + at] = (uint8_t)(ke + 127);
      a.v.exps[page * a.v.exp_ps + h * a.v.exp_hs + at] = (uint8_t)(ve + 127);
    }
  }
  if (slot >= a.num_slots && threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
}

template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) fa2_paged_read_fp8_kernel(const PagedFp8RowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lanes = 1 << a.chunks_log2, items = a.heads << a.chunks_log2;
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.total) return;
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) {
    if (slot >= 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
    return;
  }
  const long long page = slot / a.page_size, at = slot % a.page_size;
  for (int i = (int)threadIdx.x; i < items; i += (int)blockDim.x) {
    const long long h = i >> a.chunks_log2;
    const int c = i & (lanes - 1);
    const uint4 kc = a.k.codes[page * a.k.code_ps + h * a.k.code_hs + at * a.k.code_rs + c];
    const uint4 vc = a.v.codes[page * a.v.code_ps + h * a.v.code_hs + at * a.v.code_rs + c];
    const int ke = a.k.exps[page * a.k.exp_ps + h * a.k.exp_hs + at], ve = a.v.exps[page * a.v.exp_ps + h * a.v.exp_hs + at];
    uint4 x[2], y[2];
    values16<BF16>(kc, __uint_as_float((unsigned)ke << 23), x);
    values16<BF16>(vc, __uint_as_float((unsigned)ve << 23), y);
    uint4* kd = a.k.rows + t * a.k.row_rs + h * a.k.row_hs + 2 * c;
    uint4* vd = a.v.rows + t * a.v.row_rs + h * a.v.row_hs + 2 * c;
    kd[0] = x[0];
    kd[1] = x[1];
    vd[0] = y[0];
    vd[1] = y[1];
  }
}

int launch_rows(void (*kernel)(PagedFp8RowsArgs), const PagedFp8RowsArgs& a, cudaStream_t stream) {
  const int items = a.heads << a.chunks_log2;
  int x = 16;   // a row's lanes lie in one warp
  while (x < kRowThreads && x < items) x *= 2;
  const int tokens = kRowThreads / x;   // of a block
  const unsigned blocks = (unsigned)(((long long)a.total + tokens - 1) / tokens);
  return launch_chained(kernel, dim3(blocks), dim3(x, tokens), 0, stream, a);
}

}  // namespace

int launch_paged_append_fp8(const PagedFp8RowsArgs& a, cudaStream_t stream) {
  return launch_rows(a.bf16 ? fa2_paged_append_fp8_kernel<true> : fa2_paged_append_fp8_kernel<false>, a, stream);
}

int launch_paged_read_fp8(const PagedFp8RowsArgs& a, cudaStream_t stream) {
  return launch_rows(a.bf16 ? fa2_paged_read_fp8_kernel<true> : fa2_paged_read_fp8_kernel<false>, a, stream);
}

}  // namespace fa2
