// fa2_paged_fp8.cuh -- attention of each sequence's new query tokens over a
// paged key/value cache of 8-bit rows (e4m3 codes and a power of two per row).
//
// S = scale Q K^T, O = softmax(S) V, L = ln sum exp S per query row, with K =
// 2^ek code, V = 2^ev code and the masks of the 16-bit paged forward.  The
// codes go to the tensor cores as they lie in memory (kind::f8f6f4): nothing is
// widened, so a key costs 2 d bytes of HBM and of shared memory.
//
// Few query rows share a key, so the keys are the long side of both products:
//
//   S^T [128 keys x rows] = K [128 x d] Q^T,   O^T [d x rows] += V^T [d x 128] P^T
//
// with M = 128 keys (or d) and N = three times the rows, in place of 128 query
// rows of which a decoding step fills four.  Keys are lanes of tensor memory:
// a softmax thread has one key and all rows' scores of it, its two exponents
// are its own, and the row maxima, which change rarely, are the only values
// that cross threads.
//
// Three times the rows: a 16-bit q (and P) is a sum of e4m3 parts,
//   x = x1 + 2^-4 x2 + 2^-8 x3,  x1 = e4m3(x), x2 = e4m3(2^4 (x - x1)), ...
// each with four significant bits and with the range of its own scale.  The
// parts are rows of the B operand; their products are joined in fp32 by the
// thread that holds them.  q is scaled by a power of two to at most 2^8, so
// bf16 and fp16 values are exact down to 2^-25 of the row's largest.  P enters
// with its value's scale, 2^(s + ev - m), under a running maximum m of s + ev
// that keeps the largest at 2^4 .. 2^8: 12 bits, down to 2^-22 of the largest
// contribution to O, also where a key of large weight has small values (the
// first tokens of a prompt) or zeros (kFp8ZeroLog2).  The sum l adds 2^(s + ev -
// m) 2^-ev in fp32, with low exponents apart (kFp8LowInv).
//
// Schedule, fragments and merging of cut pairs are the 16-bit kernel's
// (fa2_paged.cuh); a step here is two of its 64-key tiles, and pairs always lie on
// the line: with one CTA an SM nothing would overlap a pair's start and end (8
// chunks of 512 tokens over 4096 keys, d = 128, as first built: 1104 us, a CTA a pair
// 1489; now 942).  One CTA: four softmax warps for every eight rows of a tile (a
// thread has one key and eight rows), the MMA thread, the TMA warp (keys, values,
// exponents), and the planner, which walks the fragments and prepares their q parts.  What runs seldom is rolled or
// shared: a call's code comes to each SM once, and with one thread for 32 rows,
// four times the code, a call began 50 us later.
//
// Bounds.  Decoding: HBM (64 requests of 1000 .. 32000 keys, 8 K/V heads of 128:
// 331 us, 6.6 TB/s); below some thousand keys a CTA the start (6 us) and the merge
// (4 us).  With 32 rows a tile the softmax warps' instructions: some 330 a step and
// warp, 62 % of the issue slots (128 requests x heads of 8192 keys, d = 128, from an
// empty L2 cache: 84 us at 32 rows, 74 at 16, 71 at 4; a chunk of 2048 tokens over
// 16384 keys 1720 us, 340 TFLOP/s).
#pragma once

#include <cuda_fp8.h>

#include <cfloat>

#include "fa2_paged.cuh"
#include "fa2_paged_fp8.h"
#include "sm103_ptx_fp8.cuh"

namespace fa2 {

// Barriers.  Phases count steps g (of 128 keys) or fragments of the CTA.
enum : int {
  P8_Q = 0,        // + f & 1: the fragment's description and q parts are there
  P8_P = 2,        // + g & 1: P(g) is in shared memory (all softmax warps)
  P8_ODONE = 4,    // + f & 1: the softmax warps are done with O (all)
  P8_FREE = 6,     // + f & 3: and with the description (all)
  P8_PLAN = 10,    // + f & 3: the fragment's description is there
  P8_VOTE = 14,    // + row group: its four warps' votes of step g
  P8_X = 18,       // + row group: their maxima, or their sums
  P8_EXIT = 22,
  P8_EXP = 23,     // + g & 7: the exponents of step g are there (16 lanes)
  P8_HELP = 31,    // the first fragment's q parts are written (the warps that do)
  P8_RINGS = 32,   // S complete (K stages), PV complete (V stages), K landed, V landed
};

template <int D_, int R_, bool MANY_>
struct Paged8Config {
  static constexpr int D = D_;
  static constexpr int R = R_;           // query rows of a tile, padded
  static constexpr bool MANY = MANY_;
  static constexpr int BC = 128;         // keys of a step
  static constexpr int SOFT_WARPS = R / 2;         // four for eight rows
  // From nine rows on the softmax warps write the first fragment's q parts, for which
  // everything waits (windows of 1023 keys at d = 256, 32 rows: 32 us, by the
  // planner alone 40.7; with eight rows 32 requests 55.0, 54.2).
  static constexpr bool HELP = R > 8;
  static constexpr int MMA_WARP = SOFT_WARPS;
  static constexpr int TMA_WARP = SOFT_WARPS + 1;
  static constexpr int PLAN_WARP = SOFT_WARPS + 2;
  static constexpr int THREADS = 32 * (SOFT_WARPS + 3);
  static constexpr int ROW = D < 128 ? D : 128;   // bytes of a swizzled row
  static constexpr uint32_t LAYOUT = ROW == 64 ? 4 : 2;
  static constexpr int BLOCKS = D / ROW;
  static constexpr uint32_t GROUP_BYTES = 8 * D;   // 8 key rows
  static constexpr uint32_t KV_BYTES = BC * D;
  static constexpr int NB = 3 * R;                 // rows of B: the parts
  static constexpr int N = (NB + 15) / 16 * 16;    // columns of a product (those past NB are not read)
  static constexpr uint32_t Q_BYTES = NB * D;
  static constexpr uint32_t P_BYTES = NB * BC;
  // P^T with a key's bytes next to each other (no swizzle: 16 bytes of 8 keys are a
  // block of 128 bytes, N / 16 blocks in a row): a thread writes its eight rows' parts
  // as three 8-byte words in place of 24 bytes.  With eight rows N is padded to 32
  // and two CTAs' shared memory has no room for that: there a row's 128 keys are
  // next to each other, with the 128-byte swizzle.
  static constexpr bool P_KEYS = R >= 16;
  static constexpr uint32_t P_GROUP = N / 16 * 128;   // eight keys
  static constexpr int CTAS_PER_SM = D == 256 || R >= 16 ? 1 : 2;
  static constexpr int KSTAGES = R == 32 && D == 256 ? 2 : R >= 16 && D == 128 ? 5 : D == 64 ? 6 - (R == 8) : 3;
  static constexpr int VSTAGES = R == 16 && D == 256 ? 2 : KSTAGES;
  static constexpr int ESTAGES = 8;
  static constexpr int B_S = P8_RINGS, B_O = B_S + KSTAGES, B_KFULL = B_O + VSTAGES, B_VFULL = B_KFULL + KSTAGES;
  static constexpr int BARS = B_VFULL + VSTAGES;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_P = OFF_Q + 2 * Q_BYTES;
  static constexpr uint32_t OFF_K = OFF_P + 2 * P_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + KSTAGES * KV_BYTES;
  static constexpr uint32_t OFF_EXP = OFF_V + VSTAGES * KV_BYTES;   // + 256 * (g & 7): K, V
  static constexpr uint32_t OFF_FACTOR = OFF_EXP + ESTAGES * 256;   // + 4 R * (f & 1): 2^q exponent * scale * log2 e
  static constexpr uint32_t OFF_MAX = OFF_FACTOR + 2 * 4 * R;       // each softmax warp's eight rows
  static constexpr uint32_t OFF_SUM = OFF_MAX + 4 * 8 * SOFT_WARPS; // the same
  static constexpr uint32_t OFF_VOTE = OFF_SUM + 4 * 8 * SOFT_WARPS;   // two x four bytes a row group
  static constexpr uint32_t OFF_BAR = OFF_VOTE + 32;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (BARS + 1) / 2 * 16;
  static constexpr uint32_t OFF_FRAG = OFF_MISC + 16;
  static constexpr uint32_t OFF_SCAN = OFF_FRAG + 512;
  static constexpr uint32_t SMEM_BYTES = OFF_SCAN + 320 + 1024;
  static constexpr uint32_t TMEM_S = 0;   // + N * buffer
  static constexpr uint32_t TMEM_O = 2 * N;   // + N * column block
  static constexpr uint32_t TMEM_NEED = (2 + BLOCKS) * N;
  static constexpr uint32_t TMEM_COLS = TMEM_NEED <= 128 ? 128 : TMEM_NEED <= 256 ? 256 : 512;
  static_assert(ESTAGES >= VSTAGES + 2, "exponents wait for no barrier of their own");
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 233472, "shared memory per SM");
  static_assert(TMEM_NEED <= 512 && CTAS_PER_SM * TMEM_COLS <= 512, "tensor memory");
  static_assert(OFF_K % 1024 == 0 && OFF_P % 1024 == 0 && OFF_BAR % 16 == 0, "alignment");
};

// A row's m is raised when a score with its value's exponent passes it by more
// than 8, to leave the largest at 2^4: P is at most 2^8 (e4m3: 448), and a raise
// (two exchanges between the softmax warps and a pass over O) is rare.
constexpr float kFp8RaiseLog2 = 8.f;
constexpr float kFp8TopLog2 = 4.f;
// A value row of zeros adds nothing to O, whatever P is, but is stored with exponent
// 0, above ordinary rows' (values of size 1: -8): where such a key would raise m, it
// counts with this exponent instead, and the others' P keeps its bits while their
// largest s + ev lies within 88 of its s.  (P at most 2^8 and so l 2^96 a key: below
// 2^128 over 2^31 keys.)
constexpr float kFp8ZeroLog2 = 88.f;
constexpr float kFp8ZeroInv = 309485009821345068724781056.f;   // 2^88
// A key with an exponent below -20 adds its part of l by itself, 2^(s - m), not by
// way of P.  m is at least 4 below the largest s + ev and exponents end at 60: any
// other key that leaves l because its 2^(s + ev - m) is no fp32 number weighs less
// than 2^-50 of one that stays, 2^-19 over 2^31 of them.  (A branch of each thread:
// 8 chunks of 512 tokens over 4096 keys, calls in a row, 1012 us, without it 1009, by
// a warp's vote 1016, its operands kept from before S(g) 1090.)
constexpr float kFp8LowInv = 1048576.f;   // 2^20
// Sums from 2^-40 to 2^40 go to the merge as they are (their bits): what leaves the
// merge with 2^(m - max m), past 2^-126, then weighs less than 2^-46 of another part.
constexpr unsigned kFp8NearLow = (127u - 40) << 23, kFp8NearHigh = (127u + 40) << 23;
constexpr float kFp8NoMax = -FLT_MAX;   // m before a row's first key: the lowest finite score, so that -inf - m is no NaN

// 2^e; 0 below fp32's normal range.
__device__ __forceinline__ float pow2_int(int e) { return e < -126 ? 0.f : __uint_as_float((unsigned)(min(e, 127) + 127) << 23); }

// Row i's value over a warp's lanes for eight rows at once: every exchange halves
// the rows a lane still has.  The lane returns row warp_row(lane)'s.
__device__ __forceinline__ int warp_row(int lane) { return (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1); }
template <class Op>
__device__ __forceinline__ float warp_rows(const float (&v)[8], int lane, Op op) {
  float a[4], b[2];
  const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = op(h4 ? v[i + 4] : v[i], __shfl_xor_sync(0xffffffffu, h4 ? v[i] : v[i + 4], 16));
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = op(h3 ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, h3 ? a[i] : a[i + 2], 8));
  float x = op(h2 ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, h2 ? b[0] : b[1], 4));
  x = op(x, __shfl_xor_sync(0xffffffffu, x, 2));
  return op(x, __shfl_xor_sync(0xffffffffu, x, 1));
}

// The e4m3 parts of a pair of values at most 448: bits 0-7 and 8-15 of c[i] are
// x's and y's part i.
__device__ __forceinline__ void fp8_parts(float2 v, uint32_t (&c)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
    if (i < 2) {
      const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c[i], __NV_E4M3)));
      v = __ffma2_rn(back, make_float2(-16.f, -16.f), __fmul2_rn(v, make_float2(16.f, 16.f)));   // exact
    }
  }
}

template <class C>
struct Paged8Ctx {
  uint32_t base, tmem;   // shared memory
  uint8_t* smem;
  volatile int* abort_flag;
  uint32_t* status;
  PagedFrag* frags;   // four
  __device__ __forceinline__ uint32_t bar(int i) const { return base + C::OFF_BAR + 8u * (uint32_t)i; }
  __device__ __forceinline__ bool warp_wait(int i, int phase, uint32_t site) const {
    return paged_warp_wait(bar(i), (uint32_t)phase & 1, abort_flag, status, site);
  }
};

// ---------------------------------------------------------------- the planner warp

// q's parts of fragment f's rows [from, to) into buffer `buf`, and each row's factor:
// the power of two that was taken out of it, times scale log2 e.  Rows past the
// fragment's are zero.
template <class C, int AT_ONCE>   // rows whose loads are in flight together
__device__ __forceinline__ void pg8_q_parts(const Paged8Ctx<C>& t, const PagedFp8Params& a, const PagedFrag* f, int buf,
                                            int lane, int from, int to) {
  constexpr int E = C::D / 32;   // a lane's elements of a row, next to each other
  constexpr int W = E / 2;       // in 32-bit words
  const uint32_t sQ = t.base + C::OFF_Q + (uint32_t)buf * C::Q_BYTES;
  float* factor = reinterpret_cast<float*>(t.smem + C::OFF_FACTOR) + buf * C::R;
  const int group = a.p.group, head0 = f->h * group, rows = f->rows;
  const int e0 = lane * E;
  const uint32_t block = (uint32_t)(e0 / C::ROW) * (C::NB * C::ROW), in_row = (uint32_t)(e0 % C::ROW);
#pragma unroll 1
  for (int r0 = from; r0 < to; r0 += AT_ONCE) {
    uint32_t w[AT_ONCE][W];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = r0 + i, tok = r / group;
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = 0;
      if (r < rows) {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (long long)(f->row + tok) * a.q_rs +
                              (long long)(head0 + r - tok * group) * a.q_hs + e0;
        if constexpr (W == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
        } else if constexpr (W == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          w[i][0] = x.x, w[i][1] = x.y;
        } else {
          w[i][0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = r0 + i;
      float2 x[W];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        x[k] = a.bf16 ? unpack2<true>(w[i][k]) : unpack2<false>(w[i][k]);
        top = fmaxf(top, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      // largest value f 2^n, f in [1, 2): scaled by 2^(7 - n)
      const int field = min(261 - (int)(__float_as_uint(top) >> 23), 253);   // of 2^(7 - n)
      // (an infinity's products are NaN or infinite, and its row is NaN either way)
      const float up = __uint_as_float(__float_as_uint(top) >= 0x7f800000u ? 0x7fffffffu : (unsigned)field << 23);
      if (lane == 0) factor[r] = a.scale_log2 * __uint_as_float((unsigned)(254 - field) << 23);
      uint32_t parts[3][W];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        uint32_t c[3];
        fp8_parts(make_float2(x[k].x * up, x[k].y * up), c);
#pragma unroll
        for (int j = 0; j < 3; ++j) parts[j][k] = c[j];
      }
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const uint32_t n = (uint32_t)(j * C::R + r);
        const uint32_t turn = C::ROW == 64 ? (n >> 1 & 3) : (n & 7);   // 16-byte chunks, swizzled
        const uint32_t at = sQ + block + n * C::ROW + (((in_row >> 4) ^ turn) << 4 | (in_row & 15));
        if constexpr (W == 4)
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(parts[j][0] | parts[j][1] << 16),
                       "r"(parts[j][2] | parts[j][3] << 16)
                       : "memory");
        else if constexpr (W == 2)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(parts[j][0] | parts[j][1] << 16) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)parts[j][0]) : "memory");
      }
    }
  }
  fence_proxy_async_smem();
}

// Fragment nf's description goes to its slot when nf - 4 is done, its q parts to
// their buffer when nf - 2 is (so none of its waiters can be two phases behind).
// (C::HELP: the softmax warps write the first fragment's.)
template <class C>
__device__ __forceinline__ void pg8_plan(const Paged8Ctx<C>& t, const PagedFp8Params& a, const PagedPlace<C::MANY>& place,
                                         int lane) {
  const PagedParams& p = a.p;
  FragWalk<true, C::MANY> walk;
  walk.start(p, place);
  bool have = true;
#pragma unroll 1
  for (int nf = 0; have; ++nf) {
    PagedFrag* f = t.frags + (nf & 3);
    have = next_fragment(walk, p, f, lane);
    if (lane == 0) {
      if (!have) f->n = -1;
      mbar_arrive(t.bar(P8_PLAN + (nf & 3)));
      if (nf == 0) walk.tell_merge(p, place);
    }
    __syncwarp();
    if (nf >= 2 && !t.warp_wait(P8_FREE + ((nf - 2) & 3), (nf - 2) >> 2, kSiteProducerEmpty)) return;
    if (C::HELP && nf == 0) {
      if (!t.warp_wait(P8_HELP, 0, kSiteMmaQ)) return;
    } else if (have && f->n > 0) {
      pg8_q_parts<C, 4>(t, a, f, nf & 1, lane, 0, C::R);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(t.bar(P8_Q + (nf & 1)));
  }
}

// ---------------------------------------------------------------- the TMA warp

static __device__ const unsigned long long kFp8ExponentZero = 0x7f7f7f7f7f7f7f7full;   // of pages out of range

template <class C>
__device__ __forceinline__ void pg8_load(const Paged8Ctx<C>& t, const PagedFp8Params& a, const CUtensorMap* tm_k,
                                         const CUtensorMap* tm_v, int lane) {
  const PagedParams& p = a.p;
  const int my_tile = lane >> 3, my_box = lane & 7;   // of four key tiles (two steps); rows my_box * box_rows ..
  const bool has_box = my_box < kPagedKeyTile / p.box_rows;
  const int exp_box = my_box * 8 / p.box_rows, exp_row = my_box * 8 % p.box_rows;   // this lane's 8 exponents
  const uint32_t box_bytes = (uint32_t)p.box_rows * (uint32_t)C::D;
  bool ok = true, bad = false;
  struct Ahead {
    int page, row;   // row -1: no box, or no row of the query tile sees a key of it
  };
  auto fetch = [&](const PagedFrag* f, int j4) -> Ahead {
    Ahead x;
    const int k0 = f->tile(f->j0 + j4 + my_tile) * kPagedKeyTile + my_box * p.box_rows;
    const int at = (int)((__umulhi((unsigned)k0, p.page_magic) + (unsigned)k0) >> p.page_shift);   // k0 / page_size
    const bool need = j4 + my_tile < f->n && has_box &&
                      (k0 < f->km.pre_end || (k0 < f->end && k0 + p.box_rows > f->lo));
    x.page = need ? f->table[at] : 0;
    x.row = need ? k0 - at * p.page_size : -1;
    return x;
  };
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
  auto issue = [&](const At& c, unsigned lanes, int half, const CUtensorMap* tm, uint32_t s_tile, uint32_t bar) {
    const unsigned mine = lanes & (0xffffu << (16 * half));
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(mine) * box_bytes);
    if ((mine >> lane) & 1u)
      tma_load_5d(s_tile + (uint32_t)(my_tile & 1) * (kPagedKeyTile * C::D) + (uint32_t)my_box * box_bytes, tm, 0, c.c1, 0,
                  c.c3, c.c4, bar);
  };
  int g = 0, gv = 0;
  At cv_last;
  unsigned lanes_last = 0;
  int v_left = 0;   // a V step to load: 1 + its half of four key tiles
  auto load_v = [&]() {
    if (v_left == 0) return;
    const int s = gv % C::VSTAGES;
    if (gv >= C::VSTAGES) ok = t.warp_wait(C::B_O + s, gv / C::VSTAGES - 1, kSiteProducerEmpty);
    if (!ok) return;
    issue(cv_last, lanes_last, v_left - 1, tm_v, t.base + C::OFF_V + s * C::KV_BYTES, t.bar(C::B_VFULL + s));
    v_left = 0;
    ++gv;
  };
  Ahead first4;
  ok = t.warp_wait(P8_PLAN, 0, kSiteProducerEmpty);
  if (ok && t.frags[0].n > 0) first4 = fetch(t.frags, 0);
  bool ahead = true;   // fragment nf's description has been waited for, and its first boxes fetched
#pragma unroll 1
  for (int nf = 0; ok; ++nf) {
    const PagedFrag* f = t.frags + (nf & 3);
    if (!ahead) {
      ok = t.warp_wait(P8_PLAN + (nf & 3), nf >> 2, kSiteProducerEmpty);
      if (!ok) break;
      if (f->n > 0) first4 = fetch(f, 0);
    }
    ahead = false;
    const int n = f->n;
    if (n < 0) break;
    const int steps = (n + 1) >> 1, h = f->h / a.parts;
    Ahead now = first4, next4 = first4;
    At ck, cv;
    unsigned lanes = 0;
    const uint8_t *ke = nullptr, *ve = nullptr;
    bool ehave = false;
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      if ((j & 1) == 0) {
        now = next4;
        next4 = fetch(f, 2 * j + 4);
        ck = place_box(now, p.k_side, h);
        cv = place_box(now, p.v_side, h);
        lanes = __ballot_sync(0xffffffffu, now.row >= 0);
        const int from = 8 * my_tile + exp_box;
        const int page = __shfl_sync(0xffffffffu, now.page, from), row = __shfl_sync(0xffffffffu, now.row, from);
        ehave = row >= 0;
        const bool off = page < 0 || page >= p.num_pages;
        const long long at = row + exp_row;
        const uint8_t* zero = reinterpret_cast<const uint8_t*>(&kFp8ExponentZero);
        ke = off ? zero : a.k_exps + page * a.k_exp_ps + h * a.k_exp_hs + at;
        ve = off ? zero : a.v_exps + page * a.v_exp_ps + h * a.v_exp_hs + at;
      }
      const int s = g % C::KSTAGES;
      if (g >= C::KSTAGES) ok = t.warp_wait(C::B_S + s, g / C::KSTAGES - 1, kSiteProducerEmpty);
      if (!ok) break;
      issue(ck, lanes, j & 1, tm_k, t.base + C::OFF_K + s * C::KV_BYTES, t.bar(C::B_KFULL + s));
      // the exponents' slot: step g - 8's, whose softmax was done before V(g - 2)'s stage was free
      if ((my_tile >> 1) == (j & 1)) {
        const uint32_t dst = t.base + C::OFF_EXP + (uint32_t)(g & 7) * 256 + (uint32_t)(my_tile & 1) * 64 + my_box * 8;
        if (ehave) {
          cp_async_8(dst, ke);
          cp_async_8(dst + 128, ve);
        }
        cp_async_arrive(t.bar(P8_EXP + (g & 7)));
      }
      __syncwarp();
      ++g;
      load_v();
      if (!ok) break;
      cv_last = cv;
      lanes_last = lanes;
      v_left = 1 + (j & 1);
      if (j == min(steps - 1, 1)) {   // the next fragment's first boxes
        ok = t.warp_wait(P8_PLAN + ((nf + 1) & 3), (nf + 1) >> 2, kSiteProducerEmpty);
        if (!ok) break;
        ahead = true;
        const PagedFrag* fn = t.frags + ((nf + 1) & 3);
        if (fn->n > 0) first4 = fetch(fn, 0);
      }
    }
    if (ok) load_v();
  }
  if (bad) atomicOr(p.status, kStatusBadPages);
  // own copies in flight land before the CTA may exit
  cp_async_wait_all();
  if (lane == 0) {
#pragma unroll 1
    for (int s = 0; s < C::KSTAGES; ++s)
      if (g > s) paged_drain(t.bar(C::B_KFULL + s), (uint32_t)((g - 1 - s) / C::KSTAGES) & 1, t.status);
#pragma unroll 1
    for (int s = 0; s < C::VSTAGES; ++s)
      if (gv > s) paged_drain(t.bar(C::B_VFULL + s), (uint32_t)((gv - 1 - s) / C::VSTAGES) & 1, t.status);
  }
}

// ---------------------------------------------------------------- the MMA thread

// Per fragment S(0), S(1), PV(0), S(2), PV(1) ..  S(g + 2) takes the buffer of
// S(g), which was read before P(g) came.
template <class C>
__device__ __forceinline__ void pg8_mma(const Paged8Ctx<C>& t) {
  constexpr uint32_t idesc_s = make_idesc_e4m3(C::BC, C::N, false, false);
  constexpr uint32_t idesc_o = make_idesc_e4m3(C::ROW, C::N, true, C::P_KEYS);
  const uint64_t dk = make_sdesc(t.base + C::OFF_K, 16, C::GROUP_BYTES, C::LAYOUT);
  const uint64_t dq = make_sdesc(t.base + C::OFF_Q, 16, 8 * C::ROW, C::LAYOUT);
  const uint64_t dv = make_sdesc(t.base + C::OFF_V, 1024, C::GROUP_BYTES, C::LAYOUT);
  const uint64_t dp = C::P_KEYS ? make_sdesc(t.base + C::OFF_P, C::P_GROUP, 128, 0) : make_sdesc(t.base + C::OFF_P, 16, 1024, 2);
  auto wait = [&](int bar, int phase, uint32_t site) -> bool {
    return paged_wait<false>(t.bar(bar), (uint32_t)phase & 1, t.abort_flag, t.status, site);
  };
  bool ok = true;
  int g0 = 0;   // steps of the fragments before
#pragma unroll 1
  for (int nf = 0; ok; ++nf) {
    if (!wait(P8_Q + (nf & 1), nf >> 1, kSiteMmaQ)) break;
    const int n = t.frags[nf & 3].n;
    if (n < 0) break;
    const int steps = (n + 1) >> 1;
    const uint64_t b_q = dq + (uint64_t)(((nf & 1) * C::Q_BYTES) >> 4);
#pragma unroll 1
    for (int i = 0; i <= steps && ok && n > 0; ++i) {
      if (i < steps) {
        const int g = g0 + i, s = g % C::KSTAGES;
        ok = wait(C::B_KFULL + s, g / C::KSTAGES, kSiteMmaK);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a_k = dk + (uint64_t)((s * C::KV_BYTES) >> 4);
        const uint32_t tS = t.tmem + C::TMEM_S + (uint32_t)(g & 1) * C::N;
#pragma unroll
        for (int k = 0; k < C::D / 32; ++k)
          umma_f8_ss(tS, a_k + (uint64_t)(((k >> 2) * (8 * C::ROW) + (k & 3) * 32) >> 4),
                     b_q + (uint64_t)(((k >> 2) * (C::NB * C::ROW) + (k & 3) * 32) >> 4), idesc_s, k > 0 ? 1u : 0u);
        umma_commit(t.bar(C::B_S + s));
      }
      if (i > 0) {
        const int j = i - 1, g = g0 + j, s = g % C::VSTAGES;
        ok = (j > 0 || nf == 0 || wait(P8_ODONE + ((nf - 1) & 1), (nf - 1) >> 1, kSiteMmaO)) &&
             wait(P8_P + (g & 1), g >> 1, kSiteMmaP) && wait(C::B_VFULL + s, g / C::VSTAGES, kSiteMmaV);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a_v = dv + (uint64_t)((s * C::KV_BYTES) >> 4);
        const uint64_t b_p = dp + (uint64_t)(((g & 1) * C::P_BYTES) >> 4);
#pragma unroll
        for (int b = 0; b < C::BLOCKS; ++b)
#pragma unroll
          for (int k = 0; k < C::BC / 32; ++k)
            umma_f8_ss(t.tmem + C::TMEM_O + b * C::N, a_v + (uint64_t)((k * 4 * C::GROUP_BYTES + b * 8 * C::ROW) >> 4),
                       b_p + (uint64_t)((k * (C::P_KEYS ? 4 * C::P_GROUP : 32)) >> 4), idesc_o, (j > 0 || k > 0) ? 1u : 0u);
        umma_commit(t.bar(C::B_O + s));
      }
    }
    g0 += steps;
  }
  umma_commit(t.bar(P8_EXIT));
  paged_drain(t.bar(P8_EXIT), 0, t.status);
}

// ---------------------------------------------------------------- the softmax warps

// Row `key` of V stage s: rows of C::ROW bytes, 8 C::ROW apart, whose 16-byte chunks the swizzle permutes.
template <class C>
__device__ __forceinline__ uint32_t pg8_v_row(const Paged8Ctx<C>& t, int s, int key) {
  return t.base + C::OFF_V + s * C::KV_BYTES + (uint32_t)(key >> 3) * C::GROUP_BYTES + (uint32_t)(key & 7) * C::ROW;
}

// Whether that row's codes are all zero, of either sign.
template <class C>
__device__ __forceinline__ bool pg8_zero_row(uint32_t at) {
  uint32_t any = 0;
#pragma unroll 1
  for (int b = 0; b < C::BLOCKS; ++b)
#pragma unroll 1
    for (int i = 0; i < C::ROW; i += 16) {
      uint32_t x, y, z, w;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "r"(at + b * 8 * C::ROW + i) : "memory");
      any |= x | y | z | w;
    }
  return (any & 0x7f7f7f7fu) == 0;
}

// Warps 4 n .. 4 n + 3: rows 8 n .. 8 n + 7, a key a thread.
template <class C>
__device__ __forceinline__ void pg8_softmax(const Paged8Ctx<C>& t, const PagedFp8Params& a, int warp, int lane) {
  const PagedParams& p = a.p;
  const int rg = warp >> 2, r0 = rg * 8, quad = warp & 3, tid = quad * 32 + lane;
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  const uint32_t tO = t.tmem + lane_off + C::TMEM_O + r0;
  float* s_max = reinterpret_cast<float*>(t.smem + C::OFF_MAX) + rg * 32;   // four warps x eight rows
  float* s_sum = reinterpret_cast<float*>(t.smem + C::OFF_SUM) + rg * 32;
  volatile uint8_t* s_vote = t.smem + C::OFF_VOTE + rg * 8;
  const int tok0 = r0 / p.group, head0 = r0 - tok0 * p.group;   // the first row's token and head of its group
  auto wait = [&](int bar, int phase, uint32_t site) -> bool { return t.warp_wait(bar, phase, site); };
  if constexpr (C::HELP) {
    constexpr int ROWS = C::R / C::SOFT_WARPS;
    if (!wait(P8_PLAN, 0, kSiteMmaQ)) return;
    if (t.frags[0].n > 0) pg8_q_parts<C, ROWS>(t, a, t.frags, 0, lane, warp * ROWS, (warp + 1) * ROWS);
    __syncwarp();
    if (lane == 0) mbar_arrive(t.bar(P8_HELP));
  }
  int g = 0, x_phase = 0;
  for (int nf = 0;; ++nf) {
    if (!wait(P8_Q + (nf & 1), nf >> 1, kSiteMmaQ)) return;
    const PagedFrag* f = t.frags + (nf & 3);
    const int n = f->n;
    if (n < 0) return;
    const int steps = (n + 1) >> 1;
    const TileMask tmask = f->tm;
    const float4* factor = reinterpret_cast<const float4*>(t.smem + C::OFF_FACTOR + ((nf & 1) * C::R + r0) * 4);
    const float4 f0 = factor[0], f1 = factor[1];
    const float2 fr[4] = {make_float2(f0.x, f0.y), make_float2(f0.z, f0.w), make_float2(f1.x, f1.y), make_float2(f1.z, f1.w)};
    float2 neg_m[4], l[4];   // -m and the sums, rows in pairs
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      neg_m[i] = make_float2(-kFp8NoMax, -kFp8NoMax);
      l[i] = make_float2(0.f, 0.f);
    }
#pragma unroll 1
    for (int j = 0; j < steps; ++j, ++g) {
      const int half = 2 * j + (tid >> 6);   // this thread's key tile
      const bool masked = !tmask.full(2 * j) || 2 * j + 1 >= n || !tmask.full(2 * j + 1);
      bool alive = true;        // the key is seen by some row of the query tile
      unsigned seen = 0xffu;    // and by which of these eight
      if (masked) {
        const int key = f->tile(f->j0 + min(half, n - 1)) * kPagedKeyTile + (tid & 63);
        alive = half < n && (key < f->km.pre_end || (key >= f->lo && key < f->end));
        // tokens (from the first of the eight rows' on) that see it: from key - off - wr
        // to key - off + wl, or as far as the mask has no such edge there
        const KeyMask km = f->km;
        const long long at = (long long)key - km.off - (f->q0 + tok0);
        const bool all = key < p.prefix;
        const int from = all || km.wr < 0 ? 0 : (int)max(0ll, min(8ll, at - km.wr));
        const int to = all || km.wl < 0 || key < p.sinks ? 8 : (int)max(0ll, min(8ll, at + km.wl + 1));
        const int r_from = max(0, min(8, from * p.group - head0)), r_to = max(0, min(8, to * p.group - head0));
        seen = alive && r_from < r_to ? (1u << r_to) - (1u << r_from) : 0u;
      }
      if (!wait(P8_EXP + (g & 7), g >> 3, kSiteSoftmaxS)) return;
      const uint8_t* e = t.smem + C::OFF_EXP + (g & 7) * 256 + tid;
      const int ev = (int)e[128] - 127;
      const float key_scale = __uint_as_float((unsigned)e[0] << 23), value_exp = (float)ev;
      float value_inv = pow2_int(-ev);
      // S(g), which was asked for after PV(g - 2): P(g - 2), whose place P(g) takes, has been used
      if (!wait(C::B_S + g % C::KSTAGES, g / C::KSTAGES, kSiteSoftmaxS)) return;
      tc_fence_after();
      float2 x[4];
      {
        const uint32_t tS = t.tmem + lane_off + C::TMEM_S + (uint32_t)(g & 1) * C::N + r0;
        uint32_t c[3][8];
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_ld_32x32b_x8(tS + i * C::R, c[i]);
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_ld_wait_x8(c[i]);
        const float2 down = make_float2(0.0625f, 0.0625f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          auto two = [&](int part) { return make_float2(__uint_as_float(c[part][2 * i]), __uint_as_float(c[part][2 * i + 1])); };
          x[i] = __ffma2_rn(__ffma2_rn(__ffma2_rn(two(2), down, two(1)), down, two(0)),
                            __fmul2_rn(fr[i], make_float2(key_scale, key_scale)), make_float2(value_exp, value_exp));
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!(seen >> (2 * i) & 1u)) x[i].x = -INFINITY;
            if (!(seen >> (2 * i + 1) & 1u)) x[i].y = -INFINITY;
          }
        }
      }
      auto over = [&]() {   // of the rows' scores over their m, the largest (a NaN is passed over)
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = __fadd2_rn(x[i], neg_m[i]);
          top = fmaxf(top, fmaxf(y.x, y.y));
        }
        return top;
      };
      const bool raise = __any_sync(0xffffffffu, over() > kFp8RaiseLog2);
      if (lane == 0) {
        s_vote[4 * (g & 1) + quad] = raise;
        mbar_arrive(t.bar(P8_VOTE + rg));
      }
      if (!wait(P8_VOTE + rg, g, kSiteSoftmaxO)) return;
      if (*reinterpret_cast<volatile uint32_t*>(t.smem + C::OFF_VOTE + rg * 8 + 4 * (g & 1)) != 0) {
        // a value row of zeros (exponent 0) must not set the others' scale
        if (__any_sync(0xffffffffu, value_inv == 1.f)) {
          const bool asks = value_inv == 1.f && over() > kFp8RaiseLog2;
          const int s = g % C::VSTAGES;
          if (!wait(C::B_VFULL + s, g / C::VSTAGES, kSiteMmaV)) return;
          if (asks && pg8_zero_row<C>(pg8_v_row(t, s, tid))) {
            value_inv = kFp8ZeroInv;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __fadd2_rn(x[i], make_float2(-kFp8ZeroLog2, -kFp8ZeroLog2));
          }
        }
        const float rows8[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
        const float mine = warp_rows(rows8, lane, [](float u, float v) { return fmaxf(u, v); });
        if ((lane & 3) == 0) s_max[quad * 8 + warp_row(lane)] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(t.bar(P8_X + rg));
        if (!wait(P8_X + rg, x_phase, kSiteSoftmaxO)) return;
        ++x_phase;
        float alpha[8];
        auto up = [&](int i, float& neg, float& sum) {
          const float top = fmaxf(fmaxf(s_max[i], s_max[8 + i]), fmaxf(s_max[16 + i], s_max[24 + i]));
          alpha[i] = 1.f;
          if (top + neg > kFp8RaiseLog2) {
            const float neg_new = kFp8TopLog2 - top;
            const float half = ex2_approx(0.5f * (neg_new - neg));   // (l may be far above 1 where alpha is no fp32 number)
            alpha[i] = half * half;
            sum = sum * half * half;
            neg = neg_new;
          }
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          up(2 * i, neg_m[i].x, l[i].x);
          up(2 * i + 1, neg_m[i].y, l[i].y);
        }
        if (j > 0) {
          if (!wait(C::B_O + (g - 1) % C::VSTAGES, (g - 1) / C::VSTAGES, kSiteSoftmaxO)) return;
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < C::BLOCKS * 3; ++b) {
            const uint32_t at = tO + (uint32_t)(b / 3) * C::N + (uint32_t)(b % 3) * C::R;
            uint32_t o[8];
            tmem_ld_32x32b_x8(at, o);
            tmem_ld_wait_x8(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[i]);
            tmem_st_32x32b_x8(at, o);
          }
          tmem_st_wait();
        }
      }
      if (value_inv > kFp8LowInv) {   // this key's part of l by itself
        const float shift = (float)((int)(__float_as_uint(value_inv) >> 23) - 127);   // -ev
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = __fadd2_rn(__fadd2_rn(x[i], neg_m[i]), make_float2(shift, shift));
          l[i] = __fadd2_rn(l[i], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
        }
        value_inv = 0.f;
      }
      uint32_t c[4][3];   // parts of two rows
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 y = __fadd2_rn(x[i], neg_m[i]);
        y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        l[i] = __ffma2_rn(y, make_float2(value_inv, value_inv), l[i]);
        fp8_parts(y, c[i]);
      }
      if constexpr (C::P_KEYS) {
        const uint32_t sP = t.base + C::OFF_P + (uint32_t)(g & 1) * C::P_BYTES + (uint32_t)(tid >> 3) * C::P_GROUP +
                            (uint32_t)(tid & 7) * 16;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const int at = part * C::R + r0;
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(sP + (uint32_t)(at / 16 * 128 + at % 16)),
                       "r"(c[0][part] | c[1][part] << 16), "r"(c[2][part] | c[3][part] << 16)
                       : "memory");
        }
      } else {
        const uint32_t sP = t.base + C::OFF_P + (uint32_t)(g & 1) * C::P_BYTES + (uint32_t)(r0 * 128 + (tid & 15));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t at = sP + ((uint32_t)((tid >> 4) ^ i) << 4);
#pragma unroll
          for (int part = 0; part < 3; ++part)
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(at + (uint32_t)((part * C::R + i) * 128)), "r"(c[i / 2][part] >> (8 * (i & 1)))
                         : "memory");
        }
      }
      if (rg == 0 && __any_sync(0xffffffffu, !alive)) {
        // a row of V that no query row sees may hold anything, and 0 x NaN would reach the sums
        const int s = g % C::VSTAGES;
        if (!wait(C::B_VFULL + s, g / C::VSTAGES, kSiteMmaV)) return;
        if (!alive) {
          const uint32_t at = pg8_v_row(t, s, tid);
#pragma unroll 1
          for (int b = 0; b < C::BLOCKS; ++b)
#pragma unroll
            for (int i = 0; i < C::ROW; i += 16)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + b * 8 * C::ROW + i), "r"(0u) : "memory");
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(t.bar(P8_P + (g & 1)));
    }
    // the rows' sums over all keys: over the lanes, then over the four warps
    float sum[8] = {};
    if (n > 0) {
      const float rows8[8] = {l[0].x, l[0].y, l[1].x, l[1].y, l[2].x, l[2].y, l[3].x, l[3].y};
      const float mine = warp_rows(rows8, lane, [](float u, float v) { return u + v; });
      if ((lane & 3) == 0) s_sum[quad * 8 + warp_row(lane)] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(t.bar(P8_X + rg));
      if (!wait(P8_X + rg, x_phase, kSiteEpilogueO)) return;
      ++x_phase;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = (s_sum[i] + s_sum[8 + i]) + (s_sum[16 + i] + s_sum[24 + i]);
      if (!wait(C::B_O + (g - 1) % C::VSTAGES, (g - 1) / C::VSTAGES, kSiteEpilogueO)) return;
      tc_fence_after();
    }
    const int rows = f->rows - r0, slot = f->slot;   // of these eight
    if (rows > 0) {
      const bool has_d = C::ROW == 128 || lane < 16;   // (64 rows of O^T lie in 16 lanes of each warp)
      float inv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) inv[i] = slot >= 0 ? 1.f : sum[i] == 0.f ? 0.f : 1.f / sum[i];   // 0: sees no key (a NaN sum is no such row's)
      // A partial's weight is l 2^m.  Where l is far from 1, by its keys' exponents, m is
      // raised by l's power of two, so that the merge's 2^(m - max m) says the weight.
      bool far = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) far |= __float_as_uint(sum[i]) - kFp8NearLow > kFp8NearHigh - kFp8NearLow;
      if (slot >= 0 && far) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& neg = i & 1 ? neg_m[i / 2].y : neg_m[i / 2].x;
          const float n = sum[i] == 0.f ? neg : neg - (float)((int)(__float_as_uint(sum[i]) >> 23) - 127);
          inv[i] = ex2_approx(n - neg);   // (as far as m could be raised: it may be a large number)
          sum[i] *= inv[i];
          neg = n;
        }
      }
      const long long wrap = p.o_rs - (long long)(p.group - 1) * p.o_hs;   // from a token's last head to the next token's first
#pragma unroll 1
      for (int b = 0; b < C::BLOCKS; ++b) {
        uint32_t c[3][8];
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_ld_32x32b_x8(tO + b * C::N + i * C::R, c[i]);   // n = 0: not used
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_ld_wait_x8(c[i]);
        const int d = C::ROW == 128 ? b * 128 + tid : quad * 16 + lane;
        float* part = p.ws_o + (((size_t)slot * (C::D / 4) + d / 4) * (size_t)p.slot_rows + r0) * 4 + (d & 3);
        uint16_t* dst = reinterpret_cast<uint16_t*>(paged_o_row(p, f->row + tok0, f->h * p.group + head0)) + d;
        int head = head0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = fmaf(fmaf(__uint_as_float(c[2][i]), 0.0625f, __uint_as_float(c[1][i])), 0.0625f,
                               __uint_as_float(c[0][i]));
          const float y = sum[i] == 0.f ? 0.f : o * inv[i];
          if (i < rows && has_d) {
            if (slot >= 0)
              part[4 * i] = y;
            else
              *dst = (uint16_t)(a.bf16 ? pack2<true>(y, 0.f) : pack2<false>(y, 0.f));
          }
          const bool last = ++head == p.group;
          dst += last ? wrap : p.o_hs;
          head = last ? 0 : head;
        }
      }
      float my_m = 0.f, my_l = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        my_m = lane == i ? -(i & 1 ? neg_m[i / 2].y : neg_m[i / 2].x) : my_m;
        my_l = lane == i ? sum[i] : my_l;
      }
      if (quad == 0 && lane < min(rows, 8)) {
        const int r = r0 + lane;
        if (slot >= 0) {
          *reinterpret_cast<float2*>(p.ws_ml + ((size_t)slot * (size_t)p.slot_rows + r) * 2) = make_float2(my_m, my_l);
        } else {
          const int tok = r / p.group;
          p.lse[(long long)(f->h * p.group + r - tok * p.group) * p.lse_hs + f->row + tok] =
              my_l == 0.f ? -INFINITY : (my_m + log2f(my_l)) * 0.6931471805599453f;
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(t.bar(P8_ODONE + (nf & 1)));
      mbar_arrive(t.bar(P8_FREE + (nf & 3)));
    }
  }
}

// SMALL: at most 32 sequences, each of one query tile (see fa2_paged_kernel).
template <int D, int R, bool MANY, bool SMALL>
__global__ void __launch_bounds__(Paged8Config<D, R, MANY>::THREADS, Paged8Config<D, R, MANY>::CTAS_PER_SM)
    fa2_paged_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PagedFp8Params a) {
  using C = Paged8Config<D, R, MANY>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const PagedParams& p = a.p;
  Paged8Ctx<C> t;
  t.smem = smem;
  t.base = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  t.abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  t.status = p.status;
  t.frags = reinterpret_cast<PagedFrag*>(smem + C::OFF_FRAG);
  PagedScan<MANY>* scan = reinterpret_cast<PagedScan<MANY>*>(smem + C::OFF_SCAN);
  static_assert(sizeof(PagedScan<MANY>) <= 320 && C::OFF_SCAN % 8 == 0, "scan area");
  static_assert(4 * sizeof(PagedFrag) <= 512, "fragment descriptions");
  const int warp = (int)(threadIdx.x >> 5);
  const int lane = (int)(threadIdx.x & 31);
  grid_launch_dependents();   // the merge may be scheduled once every CTA has started; it waits for the partials
  if (warp == C::TMA_WARP && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < C::BARS; ++i) {
      mbar_init(t.bar(i), i == P8_HELP ? C::SOFT_WARPS : i >= P8_EXP && i < P8_HELP ? 16 : i >= P8_P && i < P8_PLAN ? C::SOFT_WARPS
                                                         : i >= P8_VOTE && i < P8_EXIT ? 4 : 1);
    }
    *t.abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_dependency_wait();   // what precedes this kernel is complete
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  PagedPlace<MANY> place;
  if constexpr (SMALL) {
    if (warp == C::PLAN_WARP) {
      place = find_place_small(p, (int)blockIdx.x, blockIdx.x == 0);
      if (lane == 0) scan->place = place;
    }
    __syncthreads();
    place = scan->place;
  } else {
    // (seven warps of any number sum the sequences, with their barriers)
    const LineScan<MANY> sums = line_scan<224, MANY, 0>(p, (int)threadIdx.x, scan, blockIdx.x == 0, [] {});
    place = line_place<MANY, 0>(p, sums, (int)blockIdx.x, p.ctas, scan);
  }
  tc_fence_after();
  t.tmem = *tmem_slot;
  if (place.seq < 0) {   // nothing for this CTA
    if (threadIdx.x == 0 && place.line && place.piece < p.ctas) p.merges[place.piece].count = -1;
  } else if (warp == C::TMA_WARP) {
    pg8_load<C>(t, a, &tm_k, &tm_v, lane);
  } else if (warp == C::MMA_WARP) {
    if (lane == 0) pg8_mma<C>(t);
    __syncwarp();
  } else if (warp == C::PLAN_WARP) {
    pg8_plan<C>(t, a, place, lane);
  } else {
    pg8_softmax<C>(t, a, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(t.tmem, C::TMEM_COLS);
  }
}

template <int D>
int launch_paged_fp8_merge(const PagedParams& p, bool bf16, cudaStream_t stream) {
  if constexpr (D == 64) return launch_paged_merge_d64(p, bf16, stream);
  if constexpr (D == 128) return launch_paged_merge_d128(p, bf16, stream);
  return launch_paged_merge_d256(p, bf16, stream);
}

template <int D, int R, bool MANY, bool SMALL>
int launch_paged_fp8_kernels(const PagedFp8LaunchArgs& x) {
  using C = Paged8Config<D, R, MANY>;
  auto kern = fa2_paged_fp8_kernel<D, R, MANY, SMALL>;
  static std::atomic<unsigned long long> configured{0};
  const int e = once_per_device(configured, [&]() -> int {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_BYTES);
    if (r != cudaSuccess) return (int)r;
    return (int)cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  if (e != 0) return e;
  const PagedParams& p = x.a.p;
  const int r = launch_chained(kern, dim3((unsigned)p.ctas), C::THREADS, C::SMEM_BYTES, x.stream, x.tm_k, x.tm_v, x.a);
  if (r != 0) return r;
  return launch_paged_fp8_merge<D>(p, x.a.bf16 != 0, x.stream);
}

template <int D, int R>
int launch_paged_fp8_rows(const PagedFp8LaunchArgs& x) {
  return x.a.p.batch <= 32 ? launch_paged_fp8_kernels<D, R, false, true>(x)
                           : launch_paged_fp8_kernels<D, R, false, false>(x);
}

template <int D>
int launch_paged_fp8(const PagedFp8LaunchArgs& x) {
  if (x.many) return launch_paged_fp8_kernels<D, kPagedFp8Rows, true, false>(x);
  if (x.a.p.slot_rows <= 8) return launch_paged_fp8_rows<D, 8>(x);
  if (x.a.p.slot_rows <= 16) return launch_paged_fp8_rows<D, 16>(x);
  return launch_paged_fp8_rows<D, kPagedFp8Rows>(x);
}

}  // namespace fa2
