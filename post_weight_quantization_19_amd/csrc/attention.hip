// Attention over the quantized key-value cache (include/pwq_cache.h).
//
//   out = sum_p w_p V_p / sum_p w_p,  w_p = 2^(t_p f - m),
//   t_p = s_p (c_p - z_p) . q',  f = scale log2(e) / 2^k,  q' = q 2^k,
// with the running maximum m of t_p f over the tokens p seen so far.  A row is a
// query head of a token; the rows of one key head and sequence share its keys.
//
// Keys times queries: 16x16x32 float16 matrix products, 16 keys x 32 channels of
// codes (exact: |c - z| <= 255) by 32 channels x 16 rows of q' (scaled so that a row's
// largest is in 2^13 .. 2^14, in attend_tiles the largest of rows taken together where all
// are near it; float32 queries in two float16 parts).  The result has a lane for four keys
// of one row, which is where the next product, values times weights, wants its weights: P
// never leaves the registers.  Weights are held as 2^8 at the running maximum, up to 2^12 before it is
// raised, so that sums are rescaled rarely.  A partial result is the maximum less 8, and a
// 256th of the total and of the sums (weights of 16 at most, so that many add up in float32).
//
// Two kernels, for few rows of a sequence and for many, and one that joins what the
// workers of a row have found.  attend_rows is bound by memory where the cache is long,
// and by the chain of launch, batch lookup, table, records and join where it is short:
// one token behind 131071 (277 MB at 8 key heads of 128 channels in 8 bits) takes 60 us
// with cold caches, 4.6 TB/s, where a large copy reaches 5.03; one token behind 512 takes
// 10.9, of which 3.8 are a launch and 0.9 each tile of 128 tokens (workgroups of eight
// waves there gain 0.7, and lose up to 8 us with 64 sequences).  In 4 bits (64 sequences of 1
// .. 16384 tokens, 45 us) it does twice the work per byte, and spreading codes to float16,
// not memory, is what bounds it.  attend_tiles' matrix and vector instructions issue for 42%
// and 49% of the cycles, and do not overlap: 2048 bf16 tokens behind 8192, 32 heads, 347 us at
// the clock that lasting work has (420 at first), 890 TFLOP/s, where a large bf16 product
// of the library reaches 1206.
#include "cache_device.h"

#include <algorithm>

namespace pwq {
namespace {

// Native vectors: what is stored as one type and loaded as another goes through
// these, which alias everything.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;              // rows of an item: query heads of a sequence's tokens
constexpr int kTile = 128;             // tokens of a tile: 32 for each of the four waves
// What starting an item costs, in tiles: without it a worker that gets many short sequences
// is the last (64 sequences of 1 to 15000 tokens in 4 bits: 72 us with 0, 59 with 1, 47 with
// 2, 44 with 3, 44 with 5).
constexpr int kStart = 3;
constexpr float kNone = -__builtin_inff();

// Between LDS writes of a wave's lanes and reads by its other lanes: the LDS takes a
// wave's accesses in order, but the compiler must be told that they meet.
__device__ __forceinline__ void wave_meets() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ f32x4_t mfma(f16x8_t a, f16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// Weights 2^(t - base) of scores t = acc sk, two ways.  One fma gives the exact product less
// base.  The maximum is a rounded product, off by half of float32's spacing: from 2^25 on
// that is 2 and more, and at 2^30 the largest weight may be anything in 2^-56 .. 2^72 (a
// single token gave 0 or NaN).  weight_of takes the rounded product too, so that the largest
// score less the maximum is exact.  It is for rows whose maximum is that far from 0, and used
// where a maximum has just been raised.  Weights are held as 2^8 at the maximum as far as
// float32 tells scores 8 apart.
constexpr float kFar = 0x1p25f;
__device__ __forceinline__ bool is_far(float base) {
  return fabsf(base) >= kFar && base != kNone;
}
__device__ __forceinline__ float weight_of(float acc, float sk, float base) {
#pragma clang fp contract(off)
  const float t = acc * sk;            // (not an fma after all)
  return __builtin_amdgcn_exp2f(t - base);
}
__device__ __forceinline__ float base_of(float most) {
  return fabsf(most) < 4.0f * kFar ? most - 8.0f : most;
}
// In place of the number of tokens that all rows see: every record is looked at as one with
// hidden tokens, where weights are taken by weight_of.  (Another branch for each record makes
// a prompt chunk 2% slower; so it is the same, 4 short float32 prompts in 4 bits 4%.)
constexpr int kAlways = INT32_MIN;

__device__ __forceinline__ f16x2_t as_half2(uint32_t w) { return __builtin_bit_cast(f16x2_t, w); }
__device__ __forceinline__ uint32_t as_word(f16x2_t h) { return __builtin_bit_cast(uint32_t, h); }
__device__ __forceinline__ f16x8_t as_half8(uint4 w) { return __builtin_bit_cast(f16x8_t, w); }

__device__ __forceinline__ uint32_t two_halves(float a, float b) {
  const f16x2_t h = {(_Float16)a, (_Float16)b};
  return as_word(h);
}

// Codes less their zero points in float16.  A byte c below 0x64 in the upper half
// is 1024 + c; 4 bits at bit 4 are 1024 + 16 c there.  b0 = -(1024 + z) of both
// elements, b4 = -(64 + z).
__device__ __forceinline__ uint32_t bytes_less(uint32_t w, uint32_t sel, uint32_t b0) {
  return as_word(as_half2(__builtin_amdgcn_perm(0x64646464u, w, sel)) + as_half2(b0));
}
__device__ __forceinline__ uint32_t low_less(uint32_t w, uint32_t b0) {
  return as_word(as_half2((w & 0x000f000fu) | 0x64006400u) + as_half2(b0));
}
__device__ __forceinline__ uint32_t high_less(uint32_t w, uint32_t b4) {
  const f16x2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  return as_word(__builtin_elementwise_fma(as_half2((w & 0x00f000f0u) | 0x64006400u), sixteenth,
                                           as_half2(b4)));
}
// -(1024 + z) and -(64 + z) of two zero points (the second: z below 16).
__device__ __forceinline__ uint32_t bias0(int z0, int z1) {
  return 0xe400e400u | (uint32_t)z0 | (uint32_t)z1 << 16;
}
__device__ __forceinline__ uint32_t bias4(int z0, int z1) {
  return 0xd400d400u | (uint32_t)(z0 & 15) << 4 | (uint32_t)(z1 & 15) << 20;
}

// A lane's eight codes of keys (4 bits: of w0 alone), or of values (4 bits: channels 16 n + a
// of an even n, or odd), less their zero points, as a fragment of float16.
template <int BITS>
__device__ __forceinline__ uint4 key_fragment(uint32_t w0, uint32_t w1, uint32_t b0, uint32_t b4) {
  if constexpr (BITS == 8)
    return make_uint4(bytes_less(w0, 0x04010400u, b0), bytes_less(w0, 0x04030402u, b0),
                      bytes_less(w1, 0x04010400u, b0), bytes_less(w1, 0x04030402u, b0));
  else
    return make_uint4(low_less(w0, b0), high_less(w0, b4), low_less(w0 >> 8, b0),
                      high_less(w0 >> 8, b4));
}
template <int BITS>
__device__ __forceinline__ uint4 value_fragment(uint32_t w0, uint32_t w1, bool odd,
                                                const uint32_t (&z0)[4], const uint32_t (&z4)[4]) {
  if constexpr (BITS == 8)
    return make_uint4(bytes_less(w0, 0x04010400u, z0[0]), bytes_less(w0, 0x04030402u, z0[1]),
                      bytes_less(w1, 0x04010400u, z0[2]), bytes_less(w1, 0x04030402u, z0[3]));
  else if (!odd)
    return make_uint4(low_less(w0, z0[0]), low_less(w0 >> 8, z0[1]), low_less(w1, z0[2]),
                      low_less(w1 >> 8, z0[3]));
  else
    return make_uint4(high_less(w0, z4[0]), high_less(w0 >> 8, z4[1]), high_less(w1, z4[2]),
                      high_less(w1 >> 8, z4[3]));
}
// -(1024 + z) and -(64 + z) of values' zero points, two tokens to a word in the order of a
// fragment; vx the words of tokens 4 g + i, 16 + 4 g + i.
template <int BITS>
__device__ __forceinline__ void value_zeros(const u32x4_t (&vx)[2], uint32_t (&z0)[4],
                                            uint32_t (&z4)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int first = BITS == 8 ? k % 2 * 2 : k % 2, other = BITS == 8 ? 1 : 2;
    const uint32_t z = __builtin_amdgcn_perm(vx[k / 2][first + other], vx[k / 2][first],
                                             0x0c040c00u);
    z0[k] = z | 0xe400e400u, z4[k] = (z & 0x000f000fu) << 4 | 0xd400d400u;
  }
}

// Weights of a record's tokens 4 g + i (x[i]) and 16 + 4 g + i (x[4 + i]) in the order of
// a value fragment; x becomes what float16 leaves of it.  (REST: x is held in a register
// first.  Where the compiler sees the product that x is, it rounds it to float16 twice,
// once through float32 and once not, and loses a last place of the first part.)
template <int BITS, bool REST>
__device__ __forceinline__ uint4 weight_part(float (&x)[8]) {
  constexpr int B = BITS == 8 ? 1 : 2, C = BITS == 8 ? 2 : 1;
  if constexpr (REST)
#pragma unroll
    for (int i = 0; i < 8; ++i) pin(x[i]);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int a = k / 2 * 4 + (k % 2 ? C : 0), b = k / 2 * 4 + (k % 2 ? 3 : B);
    w[k] = two_halves(x[a], x[b]);
    const f16x2_t h = as_half2(w[k]);
    x[a] -= (float)h[0], x[b] -= (float)h[1];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Exponent field of the power of two that brings `top` to 2^13 .. 2^14.
__device__ __forceinline__ int up_field(float top) {
  return max(min(267 - (int)(__float_as_uint(top) >> 23), 253), 1);
}

struct __attribute__((packed, aligned(1))) any8 { uint32_t v[2]; };
// Four elements of out (any alignment).
__device__ __forceinline__ void store_row4(float* p, const float (&y)[4]) {
  *(any16*)p = any16{{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                      __float_as_uint(y[3])}};
}
__device__ __forceinline__ void store_row4(uint16_t* p, const float (&y)[4]) {
  const __bf16 v[4] = {(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
  *(any8*)p = __builtin_bit_cast(any8, v);
}

// Partial results: a slot has ROWS rows of D sums, then their maxima, then their totals.
template <int D> constexpr int kSlot = kRows * (D + 2);
// Where the slots of a row are: n of them from `first` on (of its key head), row k of each.
// n -1: the result is in out already.
struct __attribute__((aligned(16))) Found {
  int first, n, k, unused;
};

struct Walk {
  CacheBatch batch;
  int group, capacity;
  __device__ __forceinline__ Seq seq(int s) const { return sequence(batch, s); }
  __device__ __forceinline__ int items(const Seq& q) const {
    return (int)(((int64_t)(q.r1 - q.r0) * group + kRows - 1) / kRows);
  }
  // Tiles of an item, kStart more than its tokens have; 0 without tokens.
  __device__ __forceinline__ int tiles(const Seq& q) const {
    const int held = min(q.len, capacity);
    return held > 0 ? (held + kTile - 1) / kTile + kStart : 0;
  }
};

// Sums over the workgroup's first 256 threads of two numbers (others give 0); before: the
// sums of the threads before this one.
__device__ __forceinline__ void scan2(int64_t a, int64_t b, int64_t* before_a, int64_t* before_b,
                                      int64_t* all_a, int64_t* all_b, int64_t (*red)[2]) {
  int64_t ia = a, ib = b;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t ua = __shfl_up(ia, o, 64), ub = __shfl_up(ib, o, 64);
    if (lane >= o) ia += ua, ib += ub;
  }
  __syncthreads();
  if (lane == 63) red[wave][0] = ia, red[wave][1] = ib;
  __syncthreads();
  int64_t pa = 0, pb = 0, ta = 0, tb = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) pa += red[w][0], pb += red[w][1];
    ta += red[w][0], tb += red[w][1];
  }
  *before_a = pa + ia - a, *before_b = pb + ib - b;
  *all_a = ta, *all_b = tb;
}

struct Scan {
  int64_t red[8][2];
  int64_t found[3];
};

// A value that all lanes have alike, for the scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
         (int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32;
}

// Worker w's share of all tiles of a key head: c tiles (at least one) from w c on.
struct Share {
  int seq;                 // that holds the first of them; -1: there are none
  int64_t c, total;
  int64_t item, tile;      // the sequence's first item and tile
};
__device__ __forceinline__ Share share_of(const Walk& w, int64_t worker, int64_t workers,
                                          Scan& sc) {
  auto counts = [&](int s, int64_t* it, int64_t* ti) {
    *it = *ti = 0;
    if (s < w.batch.nseq) {
      const Seq q = w.seq(s);
      *it = w.items(q), *ti = *it * w.tiles(q);
    }
  };
  if (threadIdx.x == 0) sc.found[0] = -1;
  int64_t it, ti, bi, bt, ai, at;
  counts(threadIdx.x, &it, &ti);
  scan2(it, ti, &bi, &bt, &ai, &at, sc.red);
  int64_t total = at;
  if (w.batch.nseq > 256) {
    int64_t mine = 0, x, y, none;
    for (int s = 256 + threadIdx.x; s < w.batch.nseq; s += 256) {
      counts(s, &x, &y);
      mine += y;
    }
    int64_t all;
    scan2(mine, 0, &x, &y, &all, &none, sc.red);
    total += all;
  }
  Share r;
  total = uniform(total);
  r.total = total;
  r.c = max((total + workers - 1) / workers, (int64_t)1);
  const int64_t tile = worker * r.c;
  int64_t item0 = 0, tile0 = 0;
  for (int base = 0;; base += 256) {
    if (base > 0) {
      counts(base + threadIdx.x, &it, &ti);
      scan2(it, ti, &bi, &bt, &ai, &at, sc.red);
    }
    bi += item0, bt += tile0;
    if (tile >= bt && tile < bt + ti)
      sc.found[0] = base + threadIdx.x, sc.found[1] = bi, sc.found[2] = bt;
    item0 += ai, tile0 += at;
    if (tile < tile0 || base + 256 >= w.batch.nseq) break;
  }
  __syncthreads();
  r.seq = __builtin_amdgcn_readfirstlane((int)sc.found[0]);
  r.item = uniform(sc.found[1]), r.tile = uniform(sc.found[2]);
  return r;
}

// The sequence of an item (in units of ROWS rows), and the item's number in it; -1
// past the last.
template <int ROWS>
__device__ __forceinline__ int64_t items_of(const Seq& q, int group) {
  return ((int64_t)(q.r1 - q.r0) * group + ROWS - 1) / ROWS;
}
template <int ROWS>
__device__ __forceinline__ int find_item(const CacheBatch& b, int group, int64_t item, int* in,
                                         Scan& sc) {
  if (threadIdx.x == 0) sc.found[0] = -1;
  int64_t before = 0;
  for (int base = 0; base < b.nseq; base += 256) {
    const int s = threadIdx.x < 256 ? base + (int)threadIdx.x : b.nseq;
    const int64_t n = s < b.nseq ? items_of<ROWS>(sequence(b, s), group) : 0;
    int64_t at, unused, all, none;
    scan2(n, 0, &at, &unused, &all, &none, sc.red);
    at += before;
    if (item >= at && item < at + n) sc.found[0] = s, sc.found[1] = item - at;
    before += all;
  }
  __syncthreads();
  *in = (int)sc.found[1];
  return (int)sc.found[0];
}

struct RowsArgs {
  CacheView cache;
  CacheBatch batch;
  CacheTensor q, out;
  int group, causal, capacity, direct, whole;   // whole: a worker for each item
  int64_t workers, items;
  float scale;
  float* slots;
  Found* found;            // of each row: token * group + query head of the key head's
};

// The batch's, and the prefix's (workers 0: none).
struct RowsPair {
  RowsArgs a[2];
};

// Attention of 16 rows at a time: worker w of a key head takes the tiles w c .. w c + c - 1
// of all items in a row, and each of its waves 32 tokens of a tile, by itself: a record
// is spread in the registers of the wave that multiplies by it, with the next one's codes
// on the way.  (Records through LDS by asynchronous copies, several in flight, was slower.)
template <typename T, int D, int BITS>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attend_rows(const RowsPair both) {
  using R = Record<D, BITS>;
  constexpr int PARTS = std::is_same_v<T, float> ? 2 : 1;
  constexpr int J = D / 32, N = D / 16, KW = R::lane_bytes / 16;
  __shared__ Scan sc;
  __shared__ int entries[4][64];
  __shared__ float sm[4][kRows], sl[4][kRows];
  __shared__ float so[4][kRows][D + 4];
  const int64_t own_blocks = both.a[0].workers * both.a[0].cache.heads;
  const RowsArgs a = both.a[block_index() >= own_blocks];
  const int64_t block = block_index() - (block_index() >= own_blocks ? own_blocks : 0);
  const int h = (int)(block % a.cache.heads);
  const int64_t w = block / a.cache.heads;
  if (w >= a.workers) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  const Walk walk{a.batch, a.group, a.capacity};
  Share sh;
  int64_t at, end;
  if (a.whole) {                                       // item w
    int in;
    sh.seq = find_item<kRows>(a.batch, a.group, w, &in, sc);
    if (sh.seq < 0) return;
    const Seq mine = walk.seq(sh.seq);
    const int per = max(walk.tiles(mine), kStart + 1);
    sh.item = w - in, sh.tile = 0, sh.c = per;
    at = (int64_t)in * per, end = at + per;
  } else {
    sh = share_of(walk, w, a.workers, sc);
    end = min(sh.total, (w + 1) * sh.c);
    at = w * sh.c;
    if (at >= end || sh.seq < 0) return;
  }
  int s = sh.seq;
  int64_t item0 = sh.item, tile0 = sh.tile;
  Seq q = walk.seq(s);
  int per = a.whole ? (int)sh.c : walk.tiles(q), count = walk.items(q);
  const uint8_t* head_base = a.cache.records + (((int64_t)h << a.cache.blocks_shift) * R::bytes);
  const int64_t page_bytes = ((int64_t)a.cache.heads << a.cache.blocks_shift) * R::bytes;
  const int in_page = (1 << a.cache.blocks_shift) - 1;
  while (at < end) {
    while (at >= tile0 + (int64_t)per * count) {       // the next sequence with tiles
      tile0 += (int64_t)per * count, item0 += count;
      if (++s >= a.batch.nseq) return;
      q = walk.seq(s);
      per = walk.tiles(q), count = walk.items(q);
    }
    const int in = count == 1 ? 0 : (int)((at - tile0) / per);     // item of the sequence
    const int64_t item_tile = tile0 + (int64_t)in * per;
    const int ta = max((int)(at - item_tile) - kStart, 0);
    const int tb = (int)min((int64_t)per, end - item_tile) - kStart;
    const int64_t item = item0 + in;
    at = item_tile + tb + kStart;
    if (item >= a.items) return;                       // starts that descend
    if (tb <= 0) return;                               // the next worker starts it
    const int rows = (int)min((int64_t)kRows, (int64_t)(q.r1 - q.r0) * a.group - in * kRows);
    const bool whole = a.direct && ta == 0 && tb == per - kStart;
    if (!a.whole && ta == 0 && h == 0 && threadIdx.x < rows) {
      const int64_t last = (item_tile + per - 1) / sh.c;
      a.found[(int64_t)q.r0 * a.group + in * kRows + threadIdx.x] =
          Found{(int)(w + item), whole ? -1 : (int)(last - w) + 1, (int)threadIdx.x, 0};
    }
    // this lane's row
    const int r = in * kRows + min(col, rows - 1);
    const int token = r / a.group, head = h * a.group + r % a.group;
    const int held = min(q.len, a.capacity);
    const int visible = min(held, a.causal ? q.len - (q.r1 - q.r0) + token + 1 : q.len);
    int least = __builtin_amdgcn_readfirstlane(visible);
    const int most = __builtin_amdgcn_readlane(visible, rows - 1);
    f16x8_t qf[PARTS][J];
    float f;
    {
      const T* src = (const T*)a.q.p + (int64_t)(q.r0 + token) * a.q.ts +
                     (int64_t)head * a.q.hs + 8 * g;
      float x[J][8], mine = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) load8(src + 32 * j, x[j]);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          mine = fmaxf(mine, fabsf(x[j][e]));
          if (x[j][e] != x[j][e]) mine = __builtin_inff();
        }
      mine = fmaxf(mine, __shfl_xor(mine, 16, 64));
      mine = fmaxf(mine, __shfl_xor(mine, 32, 64));
      const bool bad = !(mine <= __FLT_MAX__);
      // (the row's own largest: its neighbours may be of any size)
      const int field = up_field(bad ? 0.0f : mine);
      const float up = __uint_as_float((uint32_t)field << 23);
      f = __uint_as_float((uint32_t)(254 - field) << 23) * a.scale * 1.44269504088896340736f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = bad ? __builtin_nanf("") : x[j][e] * up;
          const _Float16 hi = (_Float16)v;
          qf[0][j][e] = hi;
          if constexpr (PARTS == 2) qf[1][j][e] = (_Float16)(v - (float)hi);
        }
    }
    float base = kNone, l = 0.0f, ref = 0.0f, unit = 0.0f;
    f32x4_t o[N];
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = f32x4_t{0, 0, 0, 0};
    // this wave's records: block 4 tile + wave of every tile, up to the last that a row sees
    const int32_t* table = a.batch.table + s * a.batch.ldt;
    const int records = min(tb, (max(most, 0) + 31 - 32 * wave + 96) / 128);
    int entries_from = -64, next_page = -1, next_tile = ta;
    auto look_up = [&]() __attribute__((always_inline)) {
      const int entry = (4 * next_tile + wave) >> a.cache.blocks_shift;
      if (__builtin_expect(entry - entries_from >= 64, 0)) {
        entries_from = entry & ~63;
        wave_meets();
        entries[wave][lane] = entries_from + lane < a.batch.width ? table[entries_from + lane] : -1;
        wave_meets();
      }
      next_page = entries[wave][entry - entries_from];
    };
    struct Where {
      const uint8_t* rec;
      int there, p0;
    };
    auto next_record = [&]() __attribute__((always_inline)) {
      const int page = __builtin_amdgcn_readfirstlane(next_page), block = 4 * next_tile + wave;
      const bool hole = page < 0 || page >= a.cache.pages;
      Where at;
      at.p0 = block * 32;
      at.there = hole ? 0 : min(most - block * 32, 32);
      // (a hole: any record, its tokens count for nothing)
      at.rec = head_base + (hole ? 0 : page) * page_bytes + (block & in_page) * R::bytes;
      next_tile = min(next_tile + 1, records - 1);
      return at;
    };
    // Loads are the same for every record, without branches, and past the last record
    // repeat it: the compiler can wait for exactly those that are used.
    u32x4_t kr[KW], vr[KW], kx[2], vx[2];
    uint32_t kw[2];
    auto load_keys = [&](const Where& at) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < KW; ++i)
        kr[i] = *(const u32x4_t*)(at.rec + (uint32_t)(i * 1024 + lane * 16));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        kw[t] = *(const uint32_t*)(at.rec + (uint32_t)(R::words + 64 * t + 4 * col));
        kx[t] = *(const u32x4_t*)(at.rec + (uint32_t)(R::words + 64 * t + 16 * g));
      }
    };
    auto load_values = [&](const Where& at) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        vx[t] = *(const u32x4_t*)(at.rec + (uint32_t)(R::words + 128 + 64 * t + 16 * g));
#pragma unroll
      for (int i = 0; i < KW; ++i)
        vr[i] = *(const u32x4_t*)(at.rec + (uint32_t)(R::codes + i * 1024 + lane * 16));
    };
    if (ta < records) {
      look_up();
      Where now = next_record();
      load_keys(now);
      load_values(now);
      look_up();
      for (int tile = ta; tile < records; ++tile) {
        const int p0 = now.p0, n = now.there;
        // scores
        f32x4_t acc[2], sk[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          acc[t] = f32x4_t{0, 0, 0, 0};
          const int z = word_zero(kw[t]);
          const uint32_t b0 = bias0(z, z), b4 = bias4(z, z);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int k = (t * J + j) * (BITS / 4);
            const uint4 frag = key_fragment<BITS>(kr[k / 4][k % 4],
                                                  BITS == 8 ? kr[k / 4][k % 4 + 1] : 0, b0, b4);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              acc[t] = mfma(as_half8(frag), qf[part][j], acc[t]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sk[t][i] = word_step(kx[t][i]) * f;
        }
        const Where ahead = next_record();
        load_keys(ahead);
        float e[8];
        auto exps = [&]() __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            e[i] = __builtin_amdgcn_exp2f(fmaf(acc[i / 4][i % 4], sk[i / 4][i % 4], -base));
        };
        const int seen = min(visible - p0, n) - 4 * g;
        auto hide = [&]() __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i / 4 * 16 + i % 4 >= seen) e[i] = 0.0f;
        };
        exps();
        const bool masked = p0 + 32 > least || n < 32;
        if (masked) {
          if (least == kAlways)
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = weight_of(acc[i / 4][i % 4], sk[i / 4][i % 4], base);
          hide();
        }
        float top = 0.0f, sv[8], most_step = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top = fmaxf(top, e[i]);
          sv[i] = word_step(vx[i / 4][i % 4]);
        }
        if (masked) {
          // tokens that are not there, or that the row does not see: their steps do not count
          // for its unit, and those that read as NaN must not meet a weight of 0
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i / 4 * 16 + i % 4 >= seen) sv[i] = 0.0f;
            if (sv[i] != sv[i]) e[i] = sv[i], sv[i] = 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) most_step = fmaxf(most_step, sv[i]);
        if (__builtin_expect(__any(top > 4096.0f || most_step > ref * 8.0f), 0)) {
          // the maximum is raised once a score is 4 above it, a row's ref where a step is 8 of it
          float m = kNone;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i / 4 * 16 + i % 4 < seen) m = fmaxf(m, acc[i / 4][i % 4] * sk[i / 4][i % 4]);
          m = fmaxf(m, __shfl_xor(m, 16, 64));
          m = fmaxf(m, __shfl_xor(m, 32, 64));
          const float next = __any(top > 4096.0f) ? fmaxf(base, base_of(m)) : base;
          float factor = base == kNone ? 0.0f : __builtin_amdgcn_exp2f(base - next);
          l *= factor;
          base = next;
          if (__any(is_far(base))) least = kAlways;
          float largest = fmaxf(most_step, __shfl_xor(most_step, 16, 64));
          largest = fmaxf(largest, __shfl_xor(largest, 32, 64));
          if (largest > ref * 8.0f) {
            const float to = __uint_as_float(
                __float_as_uint(fminf(fmaxf(largest, 0x1p-126f), 0x1p127f)) & 0x7f800000u);
            factor *= ref / to;
            ref = to, unit = 1.0f / to;
          }
#pragma unroll
          for (int k = 0; k < N; ++k) o[k] *= factor;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool poisoned = e[i] != e[i];
            const float x = weight_of(acc[i / 4][i % 4], sk[i / 4][i % 4], base);
            if (!poisoned) e[i] = masked && i / 4 * 16 + i % 4 >= seen ? 0.0f : x;
          }
        }
        uint4 pf[PARTS];
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          l += e[i];
          x[i] = e[i] * (sv[i] * unit);
        }
#pragma unroll
        for (int part = 0; part < PARTS; ++part) pf[part] = weight_part<BITS, PARTS == 2>(x);
        // values
        uint32_t z0[4], z4[4];
        value_zeros<BITS>(vx, z0, z4);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int at = BITS == 8 ? k : k / 2;
          const uint32_t w0 = vr[at / 2][at % 2 * 2], w1 = vr[at / 2][at % 2 * 2 + 1];
          const uint4 frag = value_fragment<BITS>(w0, w1, k % 2, z0, z4);
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
            o[k] = mfma(as_half8(frag), as_half8(pf[part]), o[k]);
        }
        load_values(ahead);
        look_up();
        now = ahead;
      }
    }
    // the four waves' results
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    __syncthreads();
    if (g == 0) sm[wave][col] = base, sl[wave][col] = l * (1.0f / 256.0f);
    __syncthreads();
    float all = kNone, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) all = fmaxf(all, sm[i][col]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += sm[i][col] == kNone ? sl[i][col] : sl[i][col] * exp2f(sm[i][col] - all);
    // the whole result's weights are divided by here
    const float back = ref * (1.0f / 256.0f);
    const float part = (base == kNone ? 1.0f : exp2f(base - all)) *
                       (whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f);
#pragma unroll
    for (int n = 0; n < N; ++n)
      *(f32x4_t*)&so[wave][col][16 * n + 4 * g] = o[n] * part * back;
    __syncthreads();
    float* slot = a.slots + ((int64_t)h * (a.workers + a.items) + w + item) * kSlot<D>;
    for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      f32x4_t v = *(const f32x4_t*)&so[0][row][d];
#pragma unroll
      for (int k = 1; k < 4; ++k) v += *(const f32x4_t*)&so[k][row][d];
      if (whole) {
        const int rr = in * kRows + row;
        const int64_t to = (int64_t)(q.r0 + rr / a.group) * a.out.ts +
                           (int64_t)(h * a.group + rr % a.group) * a.out.hs + d;
        const float y[4] = {v[0], v[1], v[2], v[3]};
        store_row4((T*)a.out.p + to, y);
      } else {
        *(f32x4_t*)&slot[row * D + d] = v;
      }
    }
    if (!whole && wave == 0 && g == 0) {
      slot[kRows * D + col] = all;
      slot[kRows * D + kRows + col] = sum;
    }
  }
}

struct TilesArgs {
  CacheView cache;
  CacheBatch batch;
  CacheTensor q, out;
  int group, causal, capacity;
  int64_t splits, items;
  float scale;
  float* slots;            // NULL: one split, results written to out
  Found* found;            // as for attend_rows; NULL: not wanted
};

// Attention of 128 RT rows, 16 RT to each of eight waves: all waves take the same
// records of 32 tokens one after the other, spread to float16 by the workgroup once and
// kept in LDS as fragments.  The waves of a SIMD, w and w + 4, take turns: one
// multiplies (values of the record before, keys of this) while the other turns its
// scores into weights and spreads its share of the record after next.
template <typename T, int D, int BITS, int RT>
__global__ __launch_bounds__(512, 1) void attend_tiles(const TilesArgs a) {
  using R = Record<D, BITS>;
  constexpr int PARTS = std::is_same_v<T, float> ? 2 : 1;
  constexpr int J = D / 32, N = D / 16, WAVES = 8, ROWS = 16 * RT * WAVES;
  // A record's codes are spread in tasks of FT fragments from 4 WORDS bytes a lane: the
  // keys', then the values', eight or more where there are as many.
  constexpr int PIECES = 2 * R::codes / 1024, SPLIT = PIECES < WAVES ? 2 : 1;
  constexpr int TASKS = PIECES * SPLIT, TURNS = (TASKS + WAVES - 1) / WAVES, WORDS = 4 / SPLIT;
  constexpr int FT = (BITS == 8 ? 2 : 4) / SPLIT;
  // A weight is held as 2^8 of them (up to 2^12), a value's step over ref as kUnit (up to
  // 8 kUnit, which times 255 has to stay in float16 where the steps are folded in).
  constexpr float kUnit = PARTS == 1 ? 32.0f : 1.0f;
  __shared__ Scan sc;
  __shared__ float tops[WAVES], lows[WAVES];
  __shared__ float row_scale[ROWS], row_ref[ROWS];   // (ref of a row's sums: of what it sees)
  __shared__ u32x4_t frags[4][2 * J + N][64];    // [record % 4][keys (t, j), values n]
  // Of a record's tokens: keys' steps times f; zero points as -(1024 + z), a key's four times
  // twice, values' in the order of a fragment's tokens; values' steps over ref, float16 in
  // that order (folded into the values, PARTS 1) or float32.
  __shared__ __align__(16) float step_k[4][32], step_v[4][32];
  __shared__ __align__(16) uint32_t zero_k[4][32][4];
  __shared__ __align__(16) uint16_t zero_v[4][32];
  __shared__ __align__(16) _Float16 step_h[4][32];
  __shared__ __align__(16) uint32_t one_h[4];  // four times two ones
  __shared__ float2 about[4];                  // of a record: its ref; its tokens that are there
  __shared__ int entries[WAVES][64];           // table entries, a wave's own
  __shared__ int apart[16], apart_count;       // records left to the end
  const int h = (int)(block_index() % a.cache.heads);
  const int64_t rest = block_index() / a.cache.heads;
  const int64_t split = rest % a.splits, item = a.items - 1 - rest / a.splits;
  if (item < 0) return;
  int in;
  const int s = find_item<ROWS>(a.batch, a.group, item, &in, sc);
  if (s < 0) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 7;
  const Seq q = sequence(a.batch, s);
  const int rows = (int)min((int64_t)ROWS, (int64_t)(q.r1 - q.r0) * a.group - (int64_t)in * ROWS);
  const int first = in * ROWS;
  const int held = min(q.len, a.capacity);
  auto visible_of = [&](int row) {               // tokens that a row of the item sees
    return min(held, a.causal ? q.len - (q.r1 - q.r0) + (first + row) / a.group + 1 : q.len);
  };
  const int most = max(visible_of(rows - 1), 0);
  if (a.found && h == 0 && split == 0)
    for (int i = threadIdx.x; i < rows; i += 512)
      a.found[(int64_t)q.r0 * a.group + first + i] =
          Found{(int)(item * a.splits), (int)a.splits, i, 0};
  const int records = (most + 31) / 32;
  const int i0 = (int)(records * split / a.splits), i1 = (int)(records * (split + 1) / a.splits);

  // This wave's rows of queries: on their way while the first records are found.
  f16x8_t qf[RT][PARTS][J];
  int visible[RT];
  float raw[RT][J][8];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = min((rt * WAVES + wave) * 16 + col, rows - 1);
    visible[rt] = visible_of(row);
    const int r = first + row;
    const T* src = (const T*)a.q.p + (int64_t)(q.r0 + r / a.group) * a.q.ts +
                   (int64_t)(h * a.group + r % a.group) * a.q.hs + 8 * g;
#pragma unroll
    for (int j = 0; j < J; ++j) load8(src + 32 * j, raw[rt][j]);
  }
  int least = __builtin_amdgcn_readfirstlane(visible[0]);   // the first row sees least
  const int least_of_all = visible_of(0);
  if (threadIdx.x == 0) apart_count = 0;
  float f = 0.0f;
  // All rows are scaled alike, by their largest, where none is more than 2^8 below it (rows of
  // zeros aside): f goes into the keys' steps, for all.  Else each by its own, scores are brought
  // back by row_scale, and f is of a size that neither they nor the steps leave float32:
  // a row 2^40 below another would be zeros.  Records then go the way of those with hidden
  // tokens, so that even rows pay nothing.
  auto scale_queries = [&]() __attribute__((always_inline)) {
    float top = 0.0f, low = __FLT_MAX__, mine[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      mine[rt] = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          mine[rt] = fmaxf(mine[rt], fabsf(raw[rt][j][e]));
          if (raw[rt][j][e] != raw[rt][j][e]) mine[rt] = __builtin_inff();
        }
      mine[rt] = fmaxf(mine[rt], __shfl_xor(mine[rt], 16, 64));
      mine[rt] = fmaxf(mine[rt], __shfl_xor(mine[rt], 32, 64));
      if (mine[rt] > 0.0f && mine[rt] <= __FLT_MAX__) {
        top = fmaxf(top, mine[rt]);
        low = fminf(low, mine[rt]);
      }
    }
    top = wave_max(top);
    low = wave_min(low);
    if (lane == 0) tops[wave] = top, lows[wave] = low;
    __syncthreads();
    top = tops[0], low = lows[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) top = fmaxf(top, tops[i]), low = fminf(low, lows[i]);
    const bool uneven = __builtin_amdgcn_readfirstlane(low < top * 0x1p-8f);
    const int field = uneven ? min(up_field(top) + 96, 127) : up_field(top);
    if (uneven) least = kAlways;
    f = __uint_as_float((uint32_t)(254 - field) << 23) * a.scale * 1.44269504088896340736f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const bool bad = !(mine[rt] <= __FLT_MAX__);
      const int own = uneven ? up_field(bad ? 0.0f : mine[rt]) : field;
      const float up = __uint_as_float((uint32_t)own << 23);
      row_scale[(rt * WAVES + wave) * 16 + col] = ldexpf(1.0f, field - own);
      row_ref[(rt * WAVES + wave) * 16 + col] = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = bad ? __builtin_nanf("") : raw[rt][j][e] * up;
          const _Float16 hi = (_Float16)v;
          qf[rt][0][j][e] = hi;
          if constexpr (PARTS == 2) qf[rt][1][j][e] = (_Float16)(v - (float)hi);
        }
    }
  };

  // ---- staging
  // Records one after the other, up to the last.  Table entries come 64 at a time, and
  // that of the next record is read from LDS while this one is loaded.
  const int32_t* table = a.batch.table + s * a.batch.ldt;
  const uint8_t* head_base = a.cache.records + (((int64_t)h << a.cache.blocks_shift) * R::bytes);
  const int64_t page_bytes = ((int64_t)a.cache.heads << a.cache.blocks_shift) * R::bytes;
  const int in_page = (1 << a.cache.blocks_shift) - 1;
  int entries_from = -64, next_page = -1, next_block = i0;
  auto look_up = [&]() __attribute__((always_inline)) {
    const int entry = next_block >> a.cache.blocks_shift;
    if (__builtin_expect(entry - entries_from >= 64, 0)) {
      entries_from = entry & ~63;
      wave_meets();
      entries[wave][lane] = entries_from + lane < a.batch.width ? table[entries_from + lane] : -1;
      wave_meets();
    }
    next_page = entries[wave][entry - entries_from];
  };
  struct Where {
    const uint8_t* rec;
    int there;                               // its tokens that are there
  };
  auto next_record = [&]() __attribute__((always_inline)) {
    const int page = __builtin_amdgcn_readfirstlane(next_page);
    const bool hole = page < 0 || page >= a.cache.pages;
    Where w;
    w.there = hole ? 0 : min(most - next_block * 32, 32);
    // (a hole: any record, its tokens count for nothing)
    w.rec = head_base + (hole ? 0 : page) * page_bytes + (next_block & in_page) * R::bytes;
    next_block = min(next_block + 1, i1 - 1);
    return w;
  };
  // What a wave loads of a record: its part of the codes, two records ahead of spreading
  // it, and the words, three ahead.  Every wave loads alike, without branches, and indexes
  // past the last record are brought back to it: otherwise the compiler waits for all
  // loads in flight at each use (a fifth more time for 2048 bf16 tokens behind 8192).
  struct Codes {
    uint32_t c[TURNS][WORDS];
  };
  struct Words {
    uint32_t word;                           // lanes 0 .. 31 a token's key word, 32 .. its value's
    int there;
  };
  auto load_codes = [&](Codes& st, const Where& w) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int task = min(wave + WAVES * i, TASKS - 1);
      const uint8_t* from = w.rec + (uint32_t)(task / SPLIT * 1024 + task % SPLIT * (4 * WORDS) +
                                               lane * 16);
      if constexpr (SPLIT == 1) {
        const u32x4_t x = *(const u32x4_t*)from;
        st.c[i][0] = x[0], st.c[i][1] = x[1], st.c[i][2] = x[2], st.c[i][3] = x[3];
      } else {
        const u32x2_t x = *(const u32x2_t*)from;
        st.c[i][0] = x[0], st.c[i][1] = x[1];
      }
    }
  };
  auto load_words = [&](Words& st, const Where& w) __attribute__((always_inline)) {
    st.word = *(const uint32_t*)(w.rec + (uint32_t)(R::words + 4 * lane));
    st.there = w.there;
  };
  // Wave 0: a record's steps and zero points for all; ref is raised where a value's step is
  // above 8 of it.  The unit is one for all rows: a record of which some rows do not see all
  // tokens, whose values' steps are further apart than 2^8, is one without tokens here (there
  // are 9 of them at most), and is left to the end, where each row has its own unit.
  float ref = 0.0f, staged_ref = 0.0f, unit = 0.0f;     // of the sums; of the values staged
  int staged = i0, parted = 0;                          // the record; those left
  auto steps = [&](const Words& st, int buf) __attribute__((always_inline)) {
    if (wave != 0) return;
    const float step = word_step(st.word);
    const int k = lane & 31;
    int count = st.there;
    float sv = lane >= 32 && k < count && step == step ? step : 0.0f;
    if (__builtin_expect(staged * 32 + count > least_of_all && staged < i1, 0)) {
      if (wave_min(sv > 0.0f ? sv : __FLT_MAX__) * 256.0f < wave_max(sv)) {
        if (lane == 0) apart[parted] = staged, apart_count = parted + 1;
        ++parted, count = 0, sv = 0.0f;
      }
    }
    ++staged;
    const bool there = k < count;
    const uint64_t nan = __ballot(step != step) >> 32;
    if (__builtin_expect(__any(sv > staged_ref * 8.0f), 0)) {
      staged_ref = __uint_as_float(
          __float_as_uint(fminf(fmaxf(wave_max(sv), 0x1p-126f * kUnit), 0x1p127f)) & 0x7f800000u);
      unit = kUnit / staged_ref;
    }
    const uint32_t zero = 0xe400u | (uint32_t)word_zero(st.word);
    // token 16 t + 4 g + i of a fragment: 8 g + 4 t, then the order of weight_part
    const int i = BITS == 8 ? k & 3 : (k & 1) << 1 | (k & 2) >> 1;
    const int at = (k >> 2 & 3) * 8 + (k >> 4) * 4 + i;
    if (lane < 32) {
      // whoever sees a token whose values are NaN gets a NaN
      step_k[buf][k] = !there ? 0.0f : nan >> k & 1 ? __builtin_nanf("") : step * f;
      const uint32_t two = zero | zero << 16;
      *(u32x4_t*)&zero_k[buf][k][0] = u32x4_t{two, two, two, two};
    } else {
      if constexpr (PARTS == 2) step_v[buf][k] = sv * unit;
      else step_h[buf][at] = (_Float16)(sv * unit);
      zero_v[buf][at] = (uint16_t)zero;
    }
    if (lane == 0) about[buf] = make_float2(staged_ref, (float)count);
    __builtin_amdgcn_s_waitcnt(0xc07f);        // there before the barrier (lgkmcnt(0))
  };
  // What a task needs of them, read a turn ahead.
  struct Zeros {
    u32x4_t zero[TURNS], step[TURNS];
  };
  Zeros zs;
  auto fetch_zeros = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int first = min(wave + WAVES * i, TASKS - 1) * FT;
      const bool values = first >= 2 * J;
      zs.zero[i] = *(const u32x4_t*)(values ? (const void*)&zero_v[buf][8 * g]
                                            : (const void*)&zero_k[buf][first / J * 16 + col][0]);
      if constexpr (PARTS == 1)
        zs.step[i] =
            *(const u32x4_t*)(values ? (const void*)&step_h[buf][8 * g] : (const void*)&one_h[0]);
    }
  };
  auto spread = [&](const Codes& st, int buf, int i) __attribute__((always_inline)) {
    {
      const int task = min(wave + WAVES * i, TASKS - 1), first = task * FT;
      const uint32_t(&c)[WORDS] = st.c[i];
      const u32x4_t z0 = zs.zero[i];
      u32x4_t v[FT];
      if constexpr (BITS == 8) {
#pragma unroll
        for (int k = 0; k < FT; ++k)
          v[k] = u32x4_t{bytes_less(c[2 * k], 0x04010400u, z0[0]),
                         bytes_less(c[2 * k], 0x04030402u, z0[1]),
                         bytes_less(c[2 * k + 1], 0x04010400u, z0[2]),
                         bytes_less(c[2 * k + 1], 0x04030402u, z0[3])};
      } else {
        u32x4_t z4;
#pragma unroll
        for (int k = 0; k < 4; ++k) z4[k] = (z0[k] & 0x000f000fu) << 4 | 0xd400d400u;
        if (first >= 2 * J) {
#pragma unroll
          for (int k = 0; k < FT; k += 2) {
            v[k] = u32x4_t{low_less(c[k], z0[0]), low_less(c[k] >> 8, z0[1]),
                           low_less(c[k + 1], z0[2]), low_less(c[k + 1] >> 8, z0[3])};
            v[k + 1] = u32x4_t{high_less(c[k], z4[0]), high_less(c[k] >> 8, z4[1]),
                               high_less(c[k + 1], z4[2]), high_less(c[k + 1] >> 8, z4[3])};
          }
        } else {
#pragma unroll
          for (int k = 0; k < FT; ++k)
            v[k] = u32x4_t{low_less(c[k], z0[0]), high_less(c[k], z4[0]),
                           low_less(c[k] >> 8, z0[0]), high_less(c[k] >> 8, z4[0])};
        }
      }
#pragma unroll
      for (int k = 0; k < FT; ++k) {
        if constexpr (PARTS == 1)              // (keys: times 1)
#pragma unroll
          for (int n = 0; n < 4; ++n) v[k][n] = as_word(as_half2(v[k][n]) * as_half2(zs.step[i][n]));
        frags[buf][first + k][lane] = v[k];
      }
    }
  };

  // ---- sums
  f32x4_t o[RT][N], l[RT];
  float base[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    base[rt] = kNone;
    l[rt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < N; ++n) o[rt][n] = f32x4_t{0, 0, 0, 0};
  }
  u32x4_t one_words = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
  asm("" : "+v"(one_words));                 // kept, not made again for each record
  const f16x8_t ones = __builtin_bit_cast(f16x8_t, one_words);
  const bool busy = wave * 16 < rows;

  f32x4_t score[RT][2], sk[2];             // of a record's tokens, and the tokens' steps
  float2 now = make_float2(0.0f, 0.0f);    // about the record
  float e[RT][8];
  auto far_exps = [&](int rt) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e[rt][i] = weight_of(score[rt][i / 4][i % 4], sk[i / 4][i % 4], base[rt]);
  };
  auto exps = [&](int rt) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        e[rt][4 * t + i] = __builtin_amdgcn_exp2f(fmaf(score[rt][t][i], sk[t][i], -base[rt]));
  };
  auto hide = [&](int rt, int p0, int n) __attribute__((always_inline)) {
    const int end = min(visible[rt] - p0, n) - 4 * g;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i / 4 * 16 + i % 4 >= end) e[rt][i] = 0.0f;
  };
  // Weights 2^(score - maximum + 8) of a record's tokens; p0 its first token, n those
  // that are there.  The maximum is raised once a score is 4 above it.
  uint4 weight[RT][PARTS];
  // (e as exps left them)
  auto weights = [&](int buf, int p0, int n) __attribute__((always_inline)) {
    const bool masked = p0 + 32 > least || n < 32;
    if (masked)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (least == kAlways) {
          const float scale = row_scale[(rt * WAVES + wave) * 16 + col];
#pragma unroll
          for (int t = 0; t < 2; ++t) score[rt][t] *= scale;
          far_exps(rt);
        }
        hide(rt, p0, n);
      }
    float top = 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, e[rt][i]);
    if (__builtin_expect(__any(top > 4096.0f), 0)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int end = min(visible[rt] - p0, n) - 4 * g;
        float m = kNone;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = score[rt][i / 4][i % 4] * sk[i / 4][i % 4];
          if (i / 4 * 16 + i % 4 < end) m = fmaxf(m, x);
        }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float next = fmaxf(base[rt], base_of(m));
        const float factor = base[rt] == kNone ? 0.0f : __builtin_amdgcn_exp2f(base[rt] - next);
        base[rt] = next;
        if (__any(is_far(next))) least = kAlways;
        l[rt] *= factor;
#pragma unroll
        for (int nn = 0; nn < N; ++nn) o[rt][nn] *= factor;
        far_exps(rt);
        if (masked) hide(rt, p0, n);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = e[rt][i];
      if constexpr (PARTS == 1) {
        weight[rt][0] = weight_part<BITS, false>(x);
        l[rt] = mfma(ones, as_half8(weight[rt][0]), l[rt]);
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const f32x4_t y = *(const f32x4_t*)&step_v[buf][16 * t + 4 * g];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            l[rt][0] += x[4 * t + i];
            x[4 * t + i] *= y[i];
          }
        }
#pragma unroll
        for (int part = 0; part < PARTS; ++part) weight[rt][part] = weight_part<BITS, true>(x);
      }
    }
  };
  // Values of record `vb` (of 4) times weights into o, keys of `kb` times queries into
  // score: fragments come from LDS kAhead before they are used, the first of them before
  // the barrier that starts the turn.  (3: 2% slower; 5, 6, 8: the same as 4.)
  constexpr int kAhead = 4, kFrags = N + 2 * J;
  f16x8_t ahead[kAhead];
  auto fragment = [&](int k, int vb, int kb) __attribute__((always_inline)) {
    const int i = k - N;                       // keys: j, then t
    return __builtin_bit_cast(
        f16x8_t, k < N ? frags[vb][2 * J + k][lane] : frags[kb][i % 2 * J + i / 2][lane]);
  };
  auto fetch = [&](int vb) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ahead[k] = fragment(k, vb, 0);
  };
  auto multiply = [&](int vb, int kb, auto keys, auto&& between) __attribute__((always_inline)) {
    constexpr int TOTAL = decltype(keys)::value ? kFrags : N;
    if constexpr (TOTAL > N) {
      now = about[kb];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sk[t] = *(const f32x4_t*)&step_k[kb][16 * t + 4 * g];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) score[rt][t] = f32x4_t{0, 0, 0, 0};
      }
    }
    static_for_up<TOTAL>([&](auto kc) __attribute__((always_inline)) {
      constexpr int k = decltype(kc)::value;
      const f16x8_t x = ahead[k % kAhead];
      if constexpr (k + kAhead < TOTAL) ahead[k % kAhead] = fragment(k + kAhead, vb, kb);
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if constexpr (k < N) o[rt][k] = mfma(x, as_half8(weight[rt][part]), o[rt][k]);
          else
            score[rt][(k - N) % 2] = mfma(x, qf[rt][part][(k - N) / 2], score[rt][(k - N) % 2]);
        }
      between(kc);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  auto turn = [&](auto wait) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(wait)::value) lds_barrier();
    else {
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_barrier();
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto yes = std::true_type{};
  const auto no = std::false_type{};
  if (i0 < i1) {
    // Wave 0 prepares a record's steps three records ahead of its turn, and the record is
    // spread two ahead, into the place of the one two before: the last reads of that
    // were a barrier ago, the first reads are one ahead.  What a turn of weights writes to
    // LDS is waited for at the end of the next turn, of products.
    Codes st[2];
    Words wq[4];                             // two from the loop on
    look_up();
    Where at[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      at[k] = next_record();
      look_up();
      if (k < 4) load_words(wq[k], at[k]);
      if (k < 2) load_codes(st[k], at[k]);
    }
    scale_queries();
#pragma unroll
    for (int k = 0; k < 3; ++k) steps(wq[k], k);
    wq[1] = wq[3];                           // of the fourth record; the fifth's
    load_words(wq[0], at[4]);
    // the first turn multiplies weights of 0 by values of a record before the first
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int part = 0; part < PARTS; ++part) weight[rt][part] = make_uint4(0, 0, 0, 0);
    for (int n = wave; n < N; n += WAVES) frags[3][2 * J + n][lane] = u32x4_t{0, 0, 0, 0};
    if (threadIdx.x < 4) one_h[threadIdx.x] = 0x3c003c00u;
    turn(yes);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      fetch_zeros(k);
#pragma unroll
      for (int n = 0; n < TURNS; ++n) spread(st[k], k, n);
      load_codes(st[k], at[k + 2]);
    }
    Where ahead_of = at[4];
    turn(yes);
    fetch(3);
    if (wave >= 4) turn(no);
    // Larger values in record i: the sums in their unit, but for rows that are done.
    auto rescale = [&](int i) __attribute__((always_inline)) {
      if (__builtin_expect(now.x != ref, 0)) {
        const float factor = ref / now.x;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (visible[rt] > 32 * i) {
            row_ref[(rt * WAVES + wave) * 16 + col] = now.x;
#pragma unroll
            for (int n = 0; n < N; ++n) o[rt][n] *= factor;
          }
        ref = now.x;
      }
    };
    auto one = [&](int i, auto u) __attribute__((always_inline)) {
      constexpr int U = decltype(u)::value;             // (i - i0) % 4
      rescale(i - 1);
      fetch_zeros((U + 2) & 3);
      Words& wn = wq[(U + 3) & 1];
      const Words old = wn;
      multiply((U + 3) & 3, U, yes, [&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value;
        // between the products, once the zero points have come from LDS
        if constexpr (k >= kFrags / 2 && k < kFrags / 2 + TURNS)
          spread(st[U & 1], (U + 2) & 3, k - kFrags / 2);
        if constexpr (k == kFrags / 2 + TURNS) load_codes(st[U & 1], ahead_of);
        if constexpr (k == kFrags / 2 + TURNS + 1) ahead_of = next_record();
        if constexpr (k == kFrags / 2 + TURNS + 2) load_words(wn, ahead_of);
      });
      turn(yes);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) exps(rt);
      weights(U, i * 32, __builtin_amdgcn_readfirstlane((int)now.y));
      steps(old, (U + 3) & 3);
      look_up();
      fetch(U);
      turn(no);
    };
    int i = i0;
    for (;;) {
      one(i, std::integral_constant<int, 0>{});
      if (++i == i1) break;
      one(i, std::integral_constant<int, 1>{});
      if (++i == i1) break;
      one(i, std::integral_constant<int, 2>{});
      if (++i == i1) break;
      one(i, std::integral_constant<int, 3>{});
      if (++i == i1) break;
    }
    if (wave < 4) turn(no);
    {
      const int last = (i1 - 1 - i0) & 3;
      rescale(i1 - 1);
      multiply(last, 0, no, [](auto) {});
    }
    // The records left, as attend_rows takes them: spread in this wave's registers.
    const int left = __builtin_amdgcn_readfirstlane(apart_count);
    for (int a_record = 0; a_record < left; ++a_record) {
      const int i = __builtin_amdgcn_readfirstlane(apart[a_record]), p0 = 32 * i;
      const int page = __builtin_amdgcn_readfirstlane(table[i >> a.cache.blocks_shift]);
      const uint8_t* rec = head_base + page * page_bytes + (i & in_page) * R::bytes;
      const int n = min(most - p0, 32);
      const uint8_t* mine = rec + (uint32_t)(lane * 16);
      u32x4_t kx[2], vx[2];
      uint32_t kw[2], z0[4], z4[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        kw[t] = *(const uint32_t*)(rec + (uint32_t)(R::words + 64 * t + 4 * col));
        kx[t] = *(const u32x4_t*)(rec + (uint32_t)(R::words + 64 * t + 16 * g));
        vx[t] = *(const u32x4_t*)(rec + (uint32_t)(R::words + 128 + 64 * t + 16 * g));
      }
      value_zeros<BITS>(vx, z0, z4);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma clang fp contract(off)                 // (as in weight_of)
        const int row = (rt * WAVES + wave) * 16 + col;
        const int seen = min(visible[rt] - p0, n) - 4 * g;
        const float scale = row_scale[row];
        float x[8], sv[8], t[8], m = kNone, largest = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4_t acc = {0, 0, 0, 0};
          const int z = word_zero(kw[h]);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int k = (h * J + j) * BITS;
            const uint32_t* w = (const uint32_t*)(mine + k / 16 * 1024 + k % 16);
            const f16x8_t frag = as_half8(key_fragment<BITS>(w[0], BITS == 8 ? w[1] : 0,
                                                             bias0(z, z), bias4(z, z)));
#pragma unroll
            for (int part = 0; part < PARTS; ++part) acc = mfma(frag, qf[rt][part][j], acc);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 4 * h + e;
            t[k] = acc[e] * scale * (word_step(kx[h][e]) * f);
            sv[k] = word_step(vx[h][e]);
            if (16 * h + e >= seen) sv[k] = 0.0f, t[k] = kNone;
            if (sv[k] != sv[k]) t[k] = sv[k], sv[k] = 0.0f;
            m = fmaxf(m, t[k]), largest = fmaxf(largest, sv[k]);
          }
        }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        largest = fmaxf(largest, __shfl_xor(largest, 16, 64));
        largest = fmaxf(largest, __shfl_xor(largest, 32, 64));
        const float next = fmaxf(base[rt], base_of(m));
        float factor = base[rt] == kNone ? 0.0f : __builtin_amdgcn_exp2f(base[rt] - next);
        base[rt] = next;
        l[rt] *= factor;
        float own = row_ref[row];
        if (largest > own * 8.0f) {
          const float to = __uint_as_float(
              __float_as_uint(fminf(fmaxf(largest, 0x1p-126f * kUnit), 0x1p127f)) & 0x7f800000u);
          factor *= own / to;
          own = to;
          row_ref[row] = to;
        }
        float sum = 0.0f;
        const float over = own > 0.0f ? 1.0f / own : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = t[k] == kNone ? 0.0f : __builtin_amdgcn_exp2f(t[k] - next);
          sum += e;
          x[k] = e * (sv[k] * over);
        }
        if constexpr (PARTS == 1) {                // (l: the whole row's in every lane)
          sum += __shfl_xor(sum, 16, 64);
          sum += __shfl_xor(sum, 32, 64);
        }
        l[rt] += sum;
        uint4 pf[PARTS];
#pragma unroll
        for (int part = 0; part < PARTS; ++part) pf[part] = weight_part<BITS, PARTS == 2>(x);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int at = (BITS == 8 ? k : k / 2) * 8;
          const uint32_t* w = (const uint32_t*)(mine + R::codes + at / 16 * 1024 + at % 16);
          const f16x8_t frag = as_half8(value_fragment<BITS>(w[0], w[1], k % 2, z0, z4));
          f32x4_t y = {0, 0, 0, 0};
#pragma unroll
          for (int part = 0; part < PARTS; ++part) y = mfma(frag, as_half8(pf[part]), y);
          o[rt][k] = o[rt][k] * factor + y * kUnit;
        }
      }
    }
  }
  if (!busy) return;
  float* slot = a.slots + (((int64_t)h * a.items + item) * a.splits + split) * (ROWS * (D + 2));
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = (rt * WAVES + wave) * 16 + col;
    float sum = l[rt][0];
    const float back = i0 < i1 ? row_ref[row] / (kUnit * 256.0f) : 0.0f;
    if constexpr (PARTS == 2) {
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
    }
    sum *= 1.0f / 256.0f;
    if (row >= rows) continue;
    if (a.slots == nullptr) {
      const float part = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int r = first + row;
      const int64_t to = (int64_t)(q.r0 + r / a.group) * a.out.ts +
                         (int64_t)(h * a.group + r % a.group) * a.out.hs + 4 * g;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = sum == 0.0f ? 0.0f : o[rt][n][i] * part * back;
        store_row4((T*)a.out.p + to + 16 * n, y);
      }
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) slot[row * D + 16 * n + 4 * g + i] = o[rt][n][i] * back;
      if (g == 0) {
        slot[ROWS * D + row] = base[rt];
        slot[ROWS * (D + 1) + row] = sum;
      }
    }
  }
}

struct JoinArgs {
  CacheBatch batch;
  CacheTensor out;
  int heads, group, capacity;
  // the batch's own slots: per key head, rows of a slot, where a row's are
  const float* own;
  const Found* found;
  int64_t own_per_head;
  int own_rows, own_tiles;     // own_tiles: by attend_tiles, which has slots for every row
  // the prefix's, NULL: none: all of its splits of the row's tile, or (before_found) as
  // the batch's own
  const float* before;
  const Found* before_found;
  int64_t before_per_head;
  int before_rows, before_splits, before_capacity;
  const int32_t* before_length;
};
constexpr int kMostParts = 1024;   // of a row

// A row's results from the workers that had tiles of its item, and from the splits of the
// prefix: WAVES waves a row, 4 / WAVES rows a workgroup.  All maxima and totals are read at
// once, then the sums with as many loads in flight.  A row of few parts is a chain of three
// loads (5.2 us for 32 rows of 8 chats' prefix and own tokens); many rows are bytes: 128
// tokens x 32 heads of a 32768-token prefix in 16 splits, 34 MB, 11.6 us.
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(256) void join_rows(const JoinArgs j) {
  constexpr int ROWS = 4 / WAVES, MOST = kMostParts / ROWS, PER = MOST / (64 * WAVES);
  __shared__ float fac[ROWS][MOST], red[2][4], so[4][D];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int mine = ROWS == 1 ? 0 : wave, first = ROWS == 1 ? wave : 0;
  const int64_t b = block_index() * ROWS + mine;
  const int head = (int)(b % j.heads), h = head / j.group;
  // (rows of one workgroup are independent: no barrier between them)
  if (b / j.heads >= j.batch.ntok) return;
  const int t = (int)(b / j.heads);
  const int s = find_sequence_wave(j.batch, t, lane);
  if (s < 0) return;
  const int64_t row = (int64_t)t * j.group + head % j.group;
  int n = 0, k = 0, m = 0, kb = 0;
  const float *own = nullptr, *before = nullptr;
  const int64_t own_slot = (int64_t)j.own_rows * (D + 2);
  const int64_t before_slot = (int64_t)j.before_rows * (D + 2);
  // (with starts that descend, nothing may have been found)
  auto good = [](const Found& at, int rows, int64_t per_head) {
    return at.first >= 0 && at.n >= 0 && at.k >= 0 && at.k < rows &&
           at.first + (int64_t)at.n <= per_head && at.n <= kMostParts / 2;
  };
  if (j.own_tiles || min(sequence(j.batch, s).len, j.capacity) > 0) {
    const Found at = j.found[row];
    if (at.n == -1) return;                            // written already
    if (good(at, j.own_rows, j.own_per_head)) {
      n = at.n, k = at.k;
      own = j.own + ((int64_t)h * j.own_per_head + at.first) * own_slot;
    }
  }
  if (j.before_found) {
    if (min(j.before_length[0], j.before_capacity) > 0) {
      const Found at = j.before_found[row];
      if (good(at, j.before_rows, j.before_per_head)) {
        m = at.n, kb = at.k;
        before = j.before + ((int64_t)h * j.before_per_head + at.first) * before_slot;
      }
    }
  } else if (j.before) {
    const int64_t r = row - (int64_t)clamp_row(j.batch.starts[0], j.batch.ntok) * j.group;
    const int64_t first_slot = r / j.before_rows * j.before_splits;
    kb = (int)(r % j.before_rows);
    if (first_slot < j.before_per_head) {
      m = j.before_splits;
      before = j.before + ((int64_t)h * j.before_per_head + first_slot) * before_slot;
    }
  }
  auto part = [&](int i, int* rows, int* at) {
    *rows = i < n ? j.own_rows : j.before_rows;
    *at = i < n ? k : kb;
    return i < n ? own + i * own_slot : before + (i - n) * before_slot;
  };
  const int all = n + m, step = 64 * WAVES, me = first * 64 + lane;
  float top = kNone, sum = 0.0f;
  float o[D / 64] = {};
  // (one wave takes parts MOST at a time, with the maximum and total so far)
  for (int from = 0; from < all; from += MOST) {
    const int count = min(all - from, MOST);
    float mx[PER], lx[PER], next = kNone;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
      const int i = me + step * c;
      mx[c] = kNone, lx[c] = 0.0f;
      if (i < count) {
        int rows, at;
        const float* slot = part(from + i, &rows, &at);
        mx[c] = slot[(int64_t)rows * D + at], lx[c] = slot[(int64_t)rows * (D + 1) + at];
      }
      next = fmaxf(next, mx[c]);
    }
    next = wave_max(next);
    if constexpr (WAVES > 1) {
      __syncthreads();
      if (lane == 0) red[0][wave] = next;
      __syncthreads();
      next = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    }
    next = fmaxf(next, top);
    const float before_factor = top == kNone ? 1.0f : exp2f(top - next);
    float add = 0.0f;
    if constexpr (WAVES == 1) wave_meets();
#pragma unroll
    for (int c = 0; c < PER; ++c) {
      const int i = me + step * c;
      if (i >= count) break;
      const float x = mx[c] == kNone ? 1.0f : exp2f(mx[c] - next);     // (NaN sums stay)
      fac[mine][i] = x;
      add += lx[c] * x;
    }
#pragma unroll
    for (int u = 32; u >= 1; u >>= 1) add += __shfl_xor(add, u, 64);
    if constexpr (WAVES > 1) {
      if (lane == 0) red[1][wave] = add;
      __syncthreads();
      add = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    } else {
      wave_meets();
    }
    sum = sum * before_factor + add;
    top = next;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) o[e] *= before_factor;
    constexpr int AT_ONCE = 8;
    for (int i0 = first; i0 < count; i0 += WAVES * AT_ONCE) {
      float x[AT_ONCE][D / 64];
#pragma unroll
      for (int c = 0; c < AT_ONCE; ++c) {
        int rows, at;
        const float* slot = part(from + min(i0 + WAVES * c, count - 1), &rows, &at);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) x[c][e] = slot[(int64_t)at * D + 64 * e + lane];
      }
#pragma unroll
      for (int c = 0; c < AT_ONCE; ++c)
        if (i0 + WAVES * c < count)
#pragma unroll
          for (int e = 0; e < D / 64; ++e) o[e] = fmaf(x[c][e], fac[mine][i0 + WAVES * c], o[e]);
    }
  }
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int e = 0; e < D / 64; ++e) so[wave][64 * e + lane] = o[e];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      const int d = 64 * e + lane;
      o[e] = so[0][d] + so[1][d] + so[2][d] + so[3][d];
    }
  }
  const int64_t to = (int64_t)t * j.out.ts + (int64_t)head * j.out.hs + lane;
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const float y = sum == 0.0f ? 0.0f : o[e] / sum;
    if constexpr (std::is_same_v<T, float>) ((float*)j.out.p)[to + 64 * e] = y;
    else ((__bf16*)j.out.p)[to + 64 * e] = (__bf16)y;
  }
}

// 16 rows of attend_tiles' waves: what the registers hold of queries and sums.
template <typename T, int D>
struct Shape {
  static constexpr int rt = D == 256 || (D == 128 && std::is_same_v<T, float>) ? 1 : 2;
  static constexpr int rows = 128 * rt;
};
template <typename T>
int rows_of_dim(int dim) {
  return dim == 64 ? Shape<T, 64>::rows : dim == 128 ? Shape<T, 128>::rows : Shape<T, 256>::rows;
}
int tile_rows_of(int32_t dtype, int dim) {
  return dtype == PWQ_F32 ? rows_of_dim<float>(dim) : rows_of_dim<uint16_t>(dim);
}

// Tokens that a table row's pages hold.
int capacity_of(const CacheBatch& b, const CacheView& c) {
  if (c.pages == 0) return 0;
  return (int)std::min<int64_t>((int64_t)b.width << (c.blocks_shift + 5), INT32_MAX - 65535);
}

struct Launch {
  JoinArgs join;
  RowsPair rows;               // workers 0: none
  TilesArgs tiles[2];          // the batch's, the prefix's; splits 0: none
  bool joined;
  int64_t parts;               // of a row, about
};

template <typename T, int D, int BITS>
void launch_all(const Launch& l, hipStream_t st) {
  for (const TilesArgs& t : l.tiles)
    if (t.splits)
      attend_tiles<T, D, BITS, Shape<T, D>::rt>
          <<<block_grid(t.items * t.splits * t.cache.heads), 512, 0, st>>>(t);
  const int64_t blocks = l.rows.a[0].workers * l.rows.a[0].cache.heads +
                         l.rows.a[1].workers * l.rows.a[1].cache.heads;
  if (blocks) attend_rows<T, D, BITS><<<block_grid(blocks), 256, 0, st>>>(l.rows);
  if (!l.joined) return;
  const int64_t rows = (int64_t)l.join.batch.ntok * l.join.heads;
  if (l.parts > 32) join_rows<T, D, 4><<<block_grid(rows), 256, 0, st>>>(l.join);
  else join_rows<T, D, 1><<<block_grid((rows + 3) / 4), 256, 0, st>>>(l.join);
}

template <typename T, int D>
void launch_bits(const Launch& l, int bits, hipStream_t st) {
  if (bits == 8) launch_all<T, D, 8>(l, st);
  else launch_all<T, D, 4>(l, st);
}

template <typename T>
void launch_dim(const Launch& l, int dim, int bits, hipStream_t st) {
  if (dim == 64) launch_bits<T, 64>(l, bits, st);
  else if (dim == 128) launch_bits<T, 128>(l, bits, st);
  else launch_bits<T, 256>(l, bits, st);
}

}  // namespace

AttentionPlan attention_plan(const AttentionLaunch& a) {
  AttentionPlan p{};
  const int64_t heads = a.cache.heads, group = a.heads / heads;
  const int64_t rows = a.batch.ntok * group, seqs = std::min(a.batch.nseq, a.batch.ntok);
  const int64_t tile = tile_rows_of(a.dtype, a.head_dim), slot = (a.head_dim + 2) * 4;
  // Tiles of rows, or 16 rows at a time, by their estimated time, us, for the tokens that the
  // tables have room for: per row and token in float16 products of 128 channels, tiles
  // half of the other's, but of whole tiles and 12 us longer to start; an item of 16 rows
  // starts in the time of 384 tokens.  Measured, us, 16 rows at a time and tiles (bf16,
  // 8 key heads of 128 channels in 8 bits):
  //   rows of a sequence      64         128        256        512        1024
  //   1 sequence, 2500 tokens 18, 25     19, 27     23, 35     32, 37     43, 45
  //   1, 16000                29, 43     41, 46     63, 53     106, 72    185, 107
  //   8, 2500                 34, 45     41, 53     77, 65     148, 101   299, 124
  //   64, 300                 52, 50     94, 58     178, 70    351, 138   759, 299
  auto by_tiles = [&](int64_t rows_each, int64_t n, int64_t tokens) {
    const double unit = a.head_dim / 128.0 * (a.dtype == PWQ_F32 ? 2 : 1) * n * heads;
    const double whole = (double)((rows_each + tile - 1) / tile * tile);
    return 1.25e-6 * unit * rows_each * (tokens + 384) > 0.65e-6 * unit * whole * tokens + 12;
  };
  // Splits of the tokens: workgroups for every CU, where items alone are fewer, of
  // at least 64 tokens (128: 1111 tokens before 8 sequences 28.9 us instead of 28.3, 256:
  // 33.7).
  auto splits = [&](int64_t items, int64_t tokens) {
    return std::min(std::max<int64_t>(1, 256 / (items * heads)),
                    std::max<int64_t>(1, tokens / 64));
  };
  const int64_t workers = std::max<int64_t>(1, 512 / heads);
  const int64_t tokens = capacity_of(a.batch, a.cache);
  p.tiles = by_tiles((rows + seqs - 1) / seqs, seqs, tokens);
  if (p.tiles) {
    p.items = rows / tile + seqs;
    p.splits = splits((rows / seqs + tile - 1) / tile * seqs, tokens);
    if (p.splits > 1 || a.prefix.nseq) p.own_bytes = p.items * p.splits * heads * tile * slot;
  } else {
    p.items = rows / kRows + seqs;
    // Few tokens: a worker for each item and nothing to join.  Us, joined and so (bf16, 8 key
    // heads of 128 channels in 8 bits): one sequence of 250 tokens 13.6, 9.7, of 500 13.8,
    // 11.5, of 900 14.0, 14.8, of 1900 14.2, 20.2; 64 of 900 29.6, 26.3, of 1900 48.9, 44.0;
    // of 256 channels one of 250 15.3, 12.0, of 900 15.8, 19.6.
    p.whole = tokens <= std::min<int64_t>(1024, 131072 / a.head_dim) && !a.prefix.nseq;
    p.workers = p.whole ? p.items : workers;
    if (!p.whole) p.own_bytes = (p.workers + p.items) * heads * kRows * slot;
  }
  if (p.own_bytes) p.found_bytes = rows * sizeof(Found);
  if (a.prefix.nseq) {
    const int64_t before = capacity_of(a.prefix, a.cache);
    p.prefix_tiles = by_tiles(rows, 1, before);
    if (p.prefix_tiles) {
      p.prefix_items = (rows + tile - 1) / tile;
      p.prefix_splits = splits(p.prefix_items, before);
      p.prefix_bytes = p.prefix_items * p.prefix_splits * heads * tile * slot;
    } else {
      p.prefix_workers = workers;
      p.prefix_items = (rows + kRows - 1) / kRows;
      p.prefix_bytes = (workers + p.prefix_items) * heads * kRows * slot;
      p.prefix_found_bytes = rows * sizeof(Found);
    }
  }
  return p;
}

hipError_t launch_cached_attention(const AttentionLaunch& a, const AttentionPlan& p,
                                   const AttentionWs& w, hipStream_t st) {
  if (a.batch.ntok == 0 || a.batch.nseq == 0) return hipSuccess;
  const int group = a.heads / a.cache.heads;
  const int tile = tile_rows_of(a.dtype, a.head_dim);
  const int capacity = capacity_of(a.batch, a.cache);
  Launch l{};
  l.joined = p.own_bytes > 0;
  l.parts = (p.tiles ? p.splits : p.workers / std::max<int64_t>(1, p.items)) +
            p.prefix_splits + p.prefix_workers / std::max<int64_t>(1, p.prefix_items);
  l.join.batch = a.batch, l.join.out = a.out;
  l.join.heads = a.heads, l.join.group = group, l.join.capacity = capacity;
  l.join.own = (const float*)w.own, l.join.found = (const Found*)w.found;
  l.join.own_per_head = p.tiles ? p.items * p.splits : p.workers + p.items;
  l.join.own_rows = p.tiles ? tile : kRows, l.join.own_tiles = p.tiles;
  if (p.tiles)
    l.tiles[0] = TilesArgs{a.cache, a.batch, a.q, a.out, group, a.causal, capacity,
                           p.splits, p.items, a.scale, p.own_bytes ? (float*)w.own : nullptr,
                           p.own_bytes ? (Found*)w.found : nullptr};
  else
    l.rows.a[0] = RowsArgs{a.cache, a.batch, a.q, a.out, group, a.causal, capacity,
                           a.prefix.nseq == 0, p.whole, p.workers, p.items, a.scale,
                           (float*)w.own, (Found*)w.found};
  l.rows.a[1].cache = a.cache;
  if (a.prefix.nseq) {
    CacheBatch b = a.prefix;
    b.starts = a.batch.starts, b.starts_step = a.batch.nseq, b.ntok = a.batch.ntok;
    const int before = capacity_of(a.prefix, a.cache);
    if (p.prefix_tiles)
      l.tiles[1] = TilesArgs{a.cache, b, a.q, a.out, group, 0, before, p.prefix_splits,
                             p.prefix_items, a.scale, (float*)w.prefix, nullptr};
    else
      l.rows.a[1] = RowsArgs{a.cache, b, a.q, a.out, group, 0, before, 0, 0,
                             p.prefix_workers, p.prefix_items, a.scale, (float*)w.prefix,
                             (Found*)w.prefix_found};
    l.join.before = (const float*)w.prefix;
    l.join.before_found = (const Found*)w.prefix_found;
    l.join.before_per_head = p.prefix_tiles ? p.prefix_items * p.prefix_splits
                                            : p.prefix_workers + p.prefix_items;
    l.join.before_rows = p.prefix_tiles ? tile : kRows;
    l.join.before_splits = (int)p.prefix_splits;
    l.join.before_capacity = before, l.join.before_length = a.prefix.lengths;
  }
  if (a.dtype == PWQ_F32) launch_dim<float>(l, a.head_dim, a.bits, st);
  else launch_dim<uint16_t>(l, a.head_dim, a.bits, st);
  return hipGetLastError();
}

}  // namespace pwq
