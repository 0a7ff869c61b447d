// The key-value cache's layout on the device (include/pwq_cache.h), shared by
// the kernels that write, read and attend to it.
#pragma once

#include "pwq_internal.h"

namespace pwq {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// A record: 32 tokens of one head.
template <int D, int BITS>
struct Record {
  static constexpr int codes = 4 * D * BITS;            // bytes of the key (or value) codes
  static constexpr int words = 2 * codes;               // where the key words start
  static constexpr int bytes = 2 * codes + 256;
  static constexpr int lane_bytes = codes / 64;         // a lane's key (or value) codes
  // Byte of the key codes that holds token p's channels d .. d + 7 (d % 8 == 0),
  // which are BITS consecutive bytes.
  static __device__ __forceinline__ int key_at(int p, int d) {
    const int n = (p / 16 * (D / 32) + d / 32) * BITS;
    return n / 16 * 1024 + (d % 32 / 8 * 16 + p % 16) * 16 + n % 16;
  }
  // Byte of the value codes that holds token p's channel d (4 bits: in the half
  // that d / 16 % 2 says).
  static __device__ __forceinline__ int value_at(int p, int d) {
    const int key = p / 16 * 4 + p % 4;
    const int n = (BITS == 8 ? d / 16 : d / 32) * 8 + key;
    return n / 16 * 1024 + (p % 16 / 4 * 16 + d % 16) * 16 + n % 16;
  }
};

// One sequence of a batch: rows r0 .. r1 - 1 of the tensors are its tokens
// len - (r1 - r0) .. len - 1.
struct Seq {
  int r0, r1, len;
};
__device__ __forceinline__ int clamp_row(int r, int ntok) { return min(max(r, 0), ntok); }
__device__ __forceinline__ Seq sequence(const CacheBatch& b, int s) {
  Seq q;
  q.r0 = clamp_row(b.starts[(int64_t)s * b.starts_step], b.ntok);
  q.r1 = max(q.r0, clamp_row(b.starts[(int64_t)(s + 1) * b.starts_step], b.ntok));
  q.len = max(b.lengths[s], 0);
  return q;
}

// The sequence whose rows hold t, -1 for none.
__device__ __forceinline__ int find_sequence(const CacheBatch& b, int t) {
  int lo = 0, hi = b.nseq;                    // starts[lo] <= t < starts[hi], where there are any
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  if (b.nseq == 0 || t < b.starts[lo] || t >= b.starts[lo + 1]) return -1;
  return lo;
}

// The same for a wave whose lanes all ask for row t: 64 starts at a time.
__device__ __forceinline__ int find_sequence_wave(const CacheBatch& b, int t, int lane) {
  int lo = 0, count = b.nseq;
  while (count > 1) {
    const int step = (count + 63) >> 6, at = lane * step;
    const int below = __popcll(__ballot(at < count && b.starts[lo + min(at, count - 1)] <= t));
    if (below == 0) return -1;
    lo += (below - 1) * step;
    count = min(step, count - (below - 1) * step);
  }
  if (count < 1 || t < b.starts[lo] || t >= b.starts[lo + 1]) return -1;
  return lo;
}

// Address of the record of head h that holds block `block` (of 32 tokens) of a
// table row; NULL for a hole.
__device__ __forceinline__ const uint8_t* record_of(const CacheView& c, const int32_t* row,
                                                    int width, int block, int h) {
  const int entry = block >> c.blocks_shift;
  if (entry >= width) return nullptr;
  const int page = row[entry];
  if (page < 0 || page >= c.pages) return nullptr;
  const int64_t at = ((int64_t)page * c.heads + h) << c.blocks_shift;
  return c.records + (at + (block & ((1 << c.blocks_shift) - 1))) * c.record_bytes;
}

struct __attribute__((packed, aligned(1))) any16 { uint32_t v[4]; };

// Eight consecutive elements (any alignment) in float32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (std::is_same_v<T, float>) {
    const any16 a = ((const any16*)p)[0], b = ((const any16*)p)[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(a.v[e]), x[4 + e] = __uint_as_float(b.v[e]);
  } else {
    const any16 a = *(const any16*)p;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(a.v[e] << 16);
      x[2 * e + 1] = __uint_as_float(a.v[e] & 0xffff0000u);
    }
  }
}

// A word's parts.
__device__ __forceinline__ float word_step(uint32_t w) { return __uint_as_float(w & ~255u); }
__device__ __forceinline__ int word_zero(uint32_t w) { return (int)(w & 255u); }

}  // namespace pwq
