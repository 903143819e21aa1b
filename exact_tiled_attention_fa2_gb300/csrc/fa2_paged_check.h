// fa2_paged_check.h -- argument checks the paged-cache entry points share.  Not
// part of the public interface.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/fa2.h"

namespace fa2 {

constexpr long long kMaxStride = 1ll << 39;   // elements: 16-bit strides stay below the TMA limit of 2^40 bytes

constexpr int kPagedMaxHeads = 65536;
constexpr long long kPagedMaxKeys = (1ll << 31) - 4096;   // keys of a sequence, rounded up to tiles, stay below 2^31

struct Range {
  uintptr_t at;
  size_t bytes;
};

inline Range range(const void* p, size_t bytes) { return Range{reinterpret_cast<uintptr_t>(p), bytes}; }
inline bool overlap(const Range& a, const Range& b) { return a.at < b.at + b.bytes && b.at < a.at + a.bytes; }
inline bool misaligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Bytes a strided tensor can touch: dims[i] with strides st[i] (elements), and
// `inner` contiguous elements.
template <int N>
Range extent(const void* p, const long long (&dims)[N], const long long (&st)[N], long long inner, int elem) {
  long long last = inner - 1;
  for (int i = 0; i < N; ++i)
    if (dims[i] > 1) last += (dims[i] - 1) * st[i];
  return range(p, (size_t)(last + 1) * (size_t)elem);
}

// Strides of dimensions larger than 1: positive multiples of `unit` elements (a
// power of two).
template <int N>
int check_strides(const long long (&dims)[N], const long long (&st)[N], int unit = 8) {
  for (int i = 0; i < N; ++i) {
    if (dims[i] <= 1) continue;
    if (st[i] <= 0 || st[i] >= kMaxStride) return FA2_ERR_INVALID_ARG;
    if (st[i] & (unit - 1)) return FA2_ERR_MISALIGNED;
  }
  return FA2_OK;
}

// One cache tensor: (pages, heads, rows).
struct CacheView {
  long long dims[3], st[3];
  Range bytes;
};

}  // namespace fa2
