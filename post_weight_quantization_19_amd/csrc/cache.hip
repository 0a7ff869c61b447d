// Writing to the key-value cache and reading it back (include/pwq_cache.h).
//
// A head of a token becomes codes of one step and zero point, which depend on its own
// values only: everything is read once, reduced over the D / 8 lanes that hold the head, and
// written once.  The bound is memory for many tokens, and the time of a launch with its chain
// of three dependent loads (starts, table, record) for few.  Codes lie as the matrix
// cores take them, a token's value codes in single bytes 8 or 16 apart: row by row those are
// stores of single bytes, which is right for a token or two per record, and a block of 32
// tokens is put together in LDS and leaves in whole pieces of 16 bytes where there are many.
//
// Measured with the caches' own bytes warm, us (writing, reading; bf16, 8 key heads of 128
// channels in 8 bits unless said otherwise): one token 3.5, 2.5; 256 sequences' next tokens in
// 4 bits 5.7, 4.5; 10589 tokens of 6 prompts 22.6 and 14.8 (66 MB each, 2.9 and 4.5 TB/s;
// writing's quantization, and its byte stores to LDS, not memory, are what is left), in
// float32 23.6 and 22.0 (109 MB, 4.6 and 5.0 TB/s); 65536 tokens read 89.6 (407 MB, 4.5 TB/s,
// where a large copy reaches 5.03).
#include "cache_device.h"

namespace pwq {
namespace {

// Eight float32 to consecutive elements (any alignment).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (std::is_same_v<T, float>) {
    any16 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) a.v[e] = __float_as_uint(x[e]), b.v[e] = __float_as_uint(x[4 + e]);
    ((any16*)p)[0] = a, ((any16*)p)[1] = b;
  } else {
    any16 a;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __bf16 two[2] = {(__bf16)x[2 * e], (__bf16)x[2 * e + 1]};
      a.v[e] = __builtin_bit_cast(uint32_t, two);
    }
    *(any16*)p = a;
  }
}

// rint(x / s) of the exact quotient, |quotient| < 256, s of 16 significant bits
// and at least 2^-100, inv = 1 / s.  r = rint(x inv) is at most one off, and only
// where the quotient is within 2^-14 of a tie; x - r s is exact in float32 (r s has
// 24 bits, and the difference is a multiple of the smaller unit, below s), so
// that it says which side of the tie x is on.
__device__ __forceinline__ float nearest(float x, float s, float inv) {
  float r = __builtin_rintf(x * inv);
  const float d = fabsf(fmaf(-r, s, x)) * 2.0f;
  const float toward = copysignf(1.0f, fmaf(-r, s, x));
  if (d > s || (d == s && (((int)r) & 1))) r += toward;
  return r;
}

// A token's head: D / 8 lanes, eight channels each, codes of 8 channels in
// `code`.  Returns the head's word.
template <int D, int BITS>
__device__ __forceinline__ uint32_t quantize(float (&x)[8], int (&code)[8]) {
  constexpr float TOP = (1 << BITS) - 1;
  float lo = 0.0f, hi = 0.0f, sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, x[e]), hi = fmaxf(hi, x[e]);
    sum = fmaf(x[e], 0.0f, sum);                          // NaN after a NaN or an infinity
  }
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, o, 64));
    hi = fmaxf(hi, __shfl_xor(hi, o, 64));
    sum += __shfl_xor(sum, o, 64);
  }
  const float range = hi - lo;
  uint32_t word = (__float_as_uint(range / TOP) + 128u) & ~255u;
  float s = __uint_as_float(word);
  const bool bad = sum != 0.0f || !(range <= __FLT_MAX__);
  if (bad || s == 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = 0;
    return bad ? 0x7fc00000u : 0u;
  }
  // small steps: 2^64 times everything, so that 1 / s stays finite
  const float up = s < 0x1p-100f ? 0x1p64f : 1.0f;
  s *= up;
  const float inv = 1.0f / s;
  const float z = fminf(nearest(-lo * up, s, inv), TOP);
  // Away from ties the product with 1 / s rounds like the quotient.
  float off = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = x[e] * up * inv, r = __builtin_rintf(v);
    off = fmaxf(off, fabsf(v - r));
    code[e] = (int)__builtin_amdgcn_fmed3f(r + z, 0.0f, TOP);
  }
  if (off > 0.5f - 0x1p-13f)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      code[e] = (int)__builtin_amdgcn_fmed3f(nearest(x[e] * up, s, inv) + z, 0.0f, TOP);
  return word | (uint32_t)(int)z;
}

// D / 8 threads write one token's head of keys, or of values.
template <typename T, int D, int BITS>
__global__ __launch_bounds__(256) void write_rows(const CacheRowsLaunch a) {
  using R = Record<D, BITS>;
  constexpr int TH = D / 8;                               // threads of a head
  const int64_t head = block_index() * (256 / TH) + threadIdx.x / TH;
  const int d = (int)(threadIdx.x % TH) * 8;
  const int of = (int)(head & 1);
  const int t = (int)((head >> 1) / a.cache.heads), h = (int)((head >> 1) % a.cache.heads);
  if (t >= a.batch.ntok) return;                          // all threads of a head alike
  const int s = find_sequence(a.batch, t);
  if (s < 0) return;
  const Seq q = sequence(a.batch, s);
  const int p = q.len - (q.r1 - t);
  if (p < 0) return;
  const uint8_t* rec = record_of(a.cache, a.batch.table + s * a.batch.ldt, a.batch.width, p >> 5, h);
  if (!rec) return;
  uint8_t* out = a.cache.records + (rec - a.cache.records);
  const CacheTensor& src = of ? a.v : a.k;
  float x[8];
  int c[8];
  load8((const T*)src.p + t * src.ts + h * src.hs + d, x);
  const uint32_t word = quantize<D, BITS>(x, c);
  if (d == 0) ((uint32_t*)(out + R::words + of * 128))[p & 31] = word;
  if (of == 0) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BITS == 8) w[e / 4] |= (uint32_t)c[e] << (8 * (e % 4));
      else w[0] |= (uint32_t)c[e] << (4 * (e / 2) + 16 * (e % 2));
    }
    uint32_t* to = (uint32_t*)(out + R::key_at(p & 31, d));
    if constexpr (BITS == 8) *(uint2*)to = make_uint2(w[0], w[1]);
    else *to = w[0];
  } else if constexpr (BITS == 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[R::codes + R::value_at(p & 31, d + e)] = (uint8_t)c[e];
  } else {
    // channels d .. d + 7 and d + 16 .. d + 23 share bytes
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int other = __shfl_xor(c[e], 2, 64);
      if (d % 32 < 16)
        out[R::codes + R::value_at(p & 31, d + e)] = (uint8_t)(c[e] | other << 4);
    }
  }
}

template <typename T, int D, int BITS>
__global__ __launch_bounds__(256) void read_rows(const CacheRowsLaunch a) {
  using R = Record<D, BITS>;
  constexpr int TH = D / 8;
  const int64_t head = block_index() * (256 / TH) + threadIdx.x / TH;
  const int d = (int)(threadIdx.x % TH) * 8;
  const int of = (int)(head & 1);
  const int t = (int)((head >> 1) / a.cache.heads), h = (int)((head >> 1) % a.cache.heads);
  if (t >= a.batch.ntok) return;
  const int s = find_sequence(a.batch, t);
  if (s < 0) return;
  const Seq q = sequence(a.batch, s);
  const int p = q.len - (q.r1 - t);
  const uint8_t* rec = p < 0 ? nullptr : record_of(a.cache, a.batch.table + s * a.batch.ldt,
                                                   a.batch.width, p >> 5, h);
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (rec) {
    const uint32_t word = ((const uint32_t*)(rec + R::words + of * 128))[p & 31];
    const float step = word_step(word);
    const int z = word_zero(word);
    int c[8];
    if (of == 0) {
      const uint32_t* from = (const uint32_t*)(rec + R::key_at(p & 31, d));
      uint32_t w[2] = {from[0], BITS == 8 ? from[1] : 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        c[e] = BITS == 8 ? (w[e / 4] >> (8 * (e % 4))) & 255
                         : (w[0] >> (4 * (e / 2) + 16 * (e % 2))) & 15;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int byte = rec[R::codes + R::value_at(p & 31, d + e)];
        c[e] = BITS == 8 ? byte : (byte >> (d % 32 < 16 ? 0 : 4)) & 15;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)(c[e] - z) * step;
  }
  const CacheTensor& dst = of ? a.v : a.k;
  store8((T*)dst.p + t * dst.ts + h * dst.hs + d, x);
}

// Blocks of 32 tokens that a batch's rows touch, sequence after sequence: at least one of
// a sequence with rows, at most rows / 32 + 2.
__device__ __forceinline__ int blocks_of(const Seq& q) {
  const int rows = q.r1 - q.r0, from = max(q.len - rows, 0);
  return rows > 0 ? (max(q.len - 1, 0) >> 5) - (from >> 5) + 1 : 0;
}
struct Window {
  int seq, block;
};
// The window-th block; seq -1 past the last.
__device__ __forceinline__ Window find_window(const CacheBatch& b, int64_t window) {
  __shared__ int64_t sums[4];
  __shared__ Window found;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x == 0) found.seq = -1;
  int64_t before = 0;
  for (int base = 0; base < b.nseq; base += 256) {
    const int s = base + threadIdx.x;
    Seq q{0, 0, 0};
    if (s < b.nseq) q = sequence(b, s);
    const int64_t n = blocks_of(q);
    int64_t in = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t u = __shfl_up(in, o, 64);
      if (lane >= o) in += u;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = in;
    __syncthreads();
    int64_t at = before + in - n;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += sums[w];
      before += sums[w];
    }
    if (window >= at && window < at + n)
      found = Window{s, (int)(window - at) + (max(q.len - (q.r1 - q.r0), 0) >> 5)};
    if (before > window) break;
  }
  __syncthreads();
  return found;
}

// A workgroup per block and head: its record is put together in LDS, and written in pieces
// of 16 bytes where all of its tokens are the call's.
template <typename T, int D, int BITS>
__global__ __launch_bounds__(256) void write_blocks(const CacheRowsLaunch a) {
  using R = Record<D, BITS>;
  constexpr int TH = D / 8, AT_ONCE = 256 / TH, TURNS = 32 / AT_ONCE;
  __shared__ __align__(16) uint8_t image[R::bytes];
  const int h = (int)(block_index() % a.cache.heads);
  const Window w = find_window(a.batch, block_index() / a.cache.heads);
  if (w.seq < 0) return;
  const Seq q = sequence(a.batch, w.seq);
  const uint8_t* rec = record_of(a.cache, a.batch.table + w.seq * a.batch.ldt, a.batch.width,
                                 w.block, h);
  if (!rec) return;
  const int first = q.len - (q.r1 - q.r0) - w.block * 32;    // tokens first .. end - 1 are new
  const int end = min(q.len - w.block * 32, 32);
  if (end <= max(first, 0)) return;
  const int d = (int)(threadIdx.x % TH) * 8, p0 = (int)threadIdx.x / TH;
  float x[2][TURNS][8];
#pragma unroll
  for (int of = 0; of < 2; ++of)
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int p = min(max(p0 + AT_ONCE * i, first), end - 1);
      const CacheTensor& src = of ? a.v : a.k;
      load8((const T*)src.p + (int64_t)(q.r0 + p - first) * src.ts + h * src.hs + d, x[of][i]);
    }
#pragma unroll
  for (int of = 0; of < 2; ++of)
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int p = p0 + AT_ONCE * i;
      int c[8];
      const uint32_t word = quantize<D, BITS>(x[of][i], c);
      if (d == 0) *(uint32_t*)(image + R::words + of * 128 + 4 * p) = word;
      if (of == 0) {
        uint32_t v[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (BITS == 8) v[e / 4] |= (uint32_t)c[e] << (8 * (e % 4));
          else v[0] |= (uint32_t)c[e] << (4 * (e / 2) + 16 * (e % 2));
        }
#pragma unroll
        for (int e = 0; e < BITS / 4; ++e) *(uint32_t*)(image + R::key_at(p, d) + 4 * e) = v[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          int byte = c[e];
          if constexpr (BITS == 4) byte |= __shfl_xor(c[e], 2, 64) << 4;
          if (BITS == 8 || d % 32 < 16)
            image[R::codes + R::value_at(p, d + e)] = (uint8_t)byte;
        }
      }
    }
  __syncthreads();
  uint8_t* out = a.cache.records + (rec - a.cache.records);
  if (first <= 0 && end == 32) {
    for (int i = threadIdx.x; i < R::bytes / 16; i += 256)
      ((uint4*)out)[i] = ((const uint4*)image)[i];
    return;
  }
  // the new tokens' words and key codes, and single bytes of the value codes
  for (int i = threadIdx.x; i < 64; i += 256)
    if ((i & 31) >= first && (i & 31) < end)
      ((uint32_t*)(out + R::words))[i] = ((const uint32_t*)(image + R::words))[i];
  for (int i = threadIdx.x; i < 32 * TH; i += 256) {
    const int p = i / TH;
    if (p < first || p >= end) continue;
    const int at = R::key_at(p, i % TH * 8);
#pragma unroll
    for (int e = 0; e < BITS / 4; ++e)
      *(uint32_t*)(out + at + 4 * e) = *(const uint32_t*)(image + at + 4 * e);
  }
  for (int i = threadIdx.x; i < R::codes; i += 256) {
    const int n = i / 1024 * 16 + i % 16;                    // byte of lane i / 16 % 64
    const int p = n % 8 / 4 * 16 + i / 256 % 4 * 4 + n % 4;
    if (p >= first && p < end) out[R::codes + i] = image[R::codes + i];
  }
}

// A workgroup per block and head: the record through LDS.
template <typename T, int D, int BITS>
__global__ __launch_bounds__(256) void read_blocks(const CacheRowsLaunch a) {
  using R = Record<D, BITS>;
  constexpr int TH = D / 8, AT_ONCE = 256 / TH, TURNS = 32 / AT_ONCE;
  __shared__ __align__(16) uint8_t image[R::bytes];
  const int h = (int)(block_index() % a.cache.heads);
  const Window w = find_window(a.batch, block_index() / a.cache.heads);
  if (w.seq < 0) return;
  const Seq q = sequence(a.batch, w.seq);
  const uint8_t* rec = record_of(a.cache, a.batch.table + w.seq * a.batch.ldt, a.batch.width,
                                 w.block, h);
  const int first = q.len - (q.r1 - q.r0) - w.block * 32, end = min(q.len - w.block * 32, 32);
  for (int i = threadIdx.x; i < R::bytes / 16; i += 256)
    ((uint4*)image)[i] = rec ? ((const uint4*)rec)[i] : make_uint4(0, 0, 0, 0);
  __syncthreads();
  const int d = (int)(threadIdx.x % TH) * 8, p0 = (int)threadIdx.x / TH;
  if (w.block == 0 && first < 0) {                    // rows before the first token
    const float none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int p = first + p0; p < 0 && p - first < q.r1 - q.r0; p += AT_ONCE) {
      store8((T*)a.k.p + (int64_t)(q.r0 + p - first) * a.k.ts + h * a.k.hs + d, none);
      store8((T*)a.v.p + (int64_t)(q.r0 + p - first) * a.v.ts + h * a.v.hs + d, none);
    }
  }
#pragma unroll
  for (int of = 0; of < 2; ++of)
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int p = p0 + AT_ONCE * i;
      if (p < first || p >= end) continue;
      const uint32_t word = *(const uint32_t*)(image + R::words + of * 128 + 4 * p);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        int c;
        if (of == 0) {
          const uint32_t v = *(const uint32_t*)(image + R::key_at(p, d) + (BITS == 8 ? e / 4 * 4 : 0));
          c = BITS == 8 ? (v >> (8 * (e % 4))) & 255 : (v >> (4 * (e / 2) + 16 * (e % 2))) & 15;
        } else {
          c = image[R::codes + R::value_at(p, d + e)];
          if constexpr (BITS == 4) c = (c >> (d % 32 < 16 ? 0 : 4)) & 15;
        }
        x[e] = (float)(c - word_zero(word)) * word_step(word);
      }
      const CacheTensor& dst = of ? a.v : a.k;
      store8((T*)dst.p + (int64_t)(q.r0 + p - first) * dst.ts + h * dst.hs + d, x);
    }
}

template <typename T, int D, int BITS>
void launch_rows_of(const CacheRowsLaunch& a, bool write, hipStream_t st) {
  // Whole blocks where there are enough values to fill the card with them and enough rows to
  // a sequence to fill most of a block; else row by row.  Measured, us, rows and blocks (bf16,
  // 8 key heads of 128 channels in 8 bits; f32 with 2 of 64 crosses at as many values):
  //   write, sequences x rows    1x256     8x128     64x32       64x64       8x1024
  //                              4.9, 8.9  8.7, 9.9  13.6, 13.8  22.2, 16.8  34.1, 21.5
  //                              256x4      256x16      256x32
  //                              9.5, 19.4  24.4, 33.3  39.2, 34.0
  //   read                       1x256     8x64      1x1024    64x32      8x1024
  //                              3.9, 4.8  4.7, 4.8  5.8, 5.1  10.2, 6.2  29.2, 12.2
  //                              256x4     256x8      256x32
  //                              7.1, 8.2  11.8, 9.5  34.1, 15.3
  const int64_t values = (int64_t)a.batch.ntok * a.cache.heads * D;
  if (values >= (write ? 3 << 19 : 1 << 19) &&
      a.batch.ntok >= (write ? 32 : 8) * (int64_t)a.batch.nseq) {
    const int64_t windows = a.batch.ntok / 32 + 2 * (int64_t)a.batch.nseq;
    const dim3 grid = block_grid(windows * a.cache.heads);
    if (write) write_blocks<T, D, BITS><<<grid, 256, 0, st>>>(a);
    else read_blocks<T, D, BITS><<<grid, 256, 0, st>>>(a);
    return;
  }
  const int64_t heads = (int64_t)a.batch.ntok * a.cache.heads * 2;
  const dim3 grid = block_grid((heads * (D / 8) + 255) / 256);
  if (write) write_rows<T, D, BITS><<<grid, 256, 0, st>>>(a);
  else read_rows<T, D, BITS><<<grid, 256, 0, st>>>(a);
}

template <typename T, int D>
void launch_bits(const CacheRowsLaunch& a, bool write, hipStream_t st) {
  if (a.bits == 8) launch_rows_of<T, D, 8>(a, write, st);
  else launch_rows_of<T, D, 4>(a, write, st);
}

template <typename T>
void launch_dim(const CacheRowsLaunch& a, bool write, hipStream_t st) {
  if (a.head_dim == 64) launch_bits<T, 64>(a, write, st);
  else if (a.head_dim == 128) launch_bits<T, 128>(a, write, st);
  else launch_bits<T, 256>(a, write, st);
}

hipError_t launch(const CacheRowsLaunch& a, bool write, hipStream_t st) {
  if (a.batch.ntok == 0 || a.batch.nseq == 0) return hipSuccess;
  if (a.dtype == PWQ_F32) launch_dim<float>(a, write, st);
  else launch_dim<uint16_t>(a, write, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const CacheRowsLaunch& a, hipStream_t st) {
  return launch(a, true, st);
}
hipError_t launch_cache_read(const CacheRowsLaunch& a, hipStream_t st) {
  return launch(a, false, st);
}

}  // namespace pwq
