// Attention over the quantized key-value cache (include/pwq_cache.h).
//
//   out = sum_p w_p V_p / sum_p w_p,  w_p = 2^(t_p f - m),
//   t_p = s_p (c_p - z_p) . q',  f = scale log2(e) / 2^k,  q' = q 2^k,
// with the running maximum m of t_p f over the tokens p seen so far.  A row is a
// query head of a token; the rows of one key head and sequence share its keys.
//
// Keys times queries: 16x16x32 float16 matrix products, 16 keys x 32 channels of
// codes (exact: |c - z| <= 255) by 32 channels x 16 rows of q' (scaled so that
// the row's largest is in 2^13 .. 2^14).  The result has a lane for four keys of one
// row, which is where the next product, values times weights, wants its weights:
// P never leaves the registers.  The steps of the values go into the weights,
// w_p s_p / ref (ref a power of two), 256 at the largest steps seen, up to 2^15.
#include "cache_device.h"

#include <algorithm>

namespace pwq {
namespace {

constexpr int kRows = 16;              // rows of an item: query heads of a sequence's tokens
constexpr int kTile = 128;             // tokens of a tile: 32 for each of the four waves
constexpr float kNone = -__builtin_inff();

__device__ __forceinline__ f32x4_t mfma(f16x8_t a, f16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
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

// The rows of an item.
struct Item {
  int seq, first;          // row `first` of the sequence's (r1 - r0) * group rows
  Seq s;
  int keys;                // tokens that any row sees, within the table
};

// Partial results: a slot has 16 rows of D sums, then 16 maxima, then 16 totals.
template <int D> constexpr int kSlot = kRows * (D + 2);

struct Walk {
  CacheBatch batch;
  const CacheView* cache;
  int group, capacity;
  __device__ __forceinline__ Seq seq(int s) const { return sequence(batch, s); }
  __device__ __forceinline__ int items(const Seq& q) const {
    return (int)(((int64_t)(q.r1 - q.r0) * group + kRows - 1) / kRows);
  }
  __device__ __forceinline__ int tiles(const Seq& q) const {
    return (min(q.len, capacity) + kTile - 1) / kTile;
  }
};

// Sums over the workgroup's 256 threads of two numbers; before: the sums of the
// threads before this one.
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

// Where a tile, or a sequence, stands among all items of a key head.
struct Place {
  int seq;                 // -1: past the end
  int64_t item, tile;      // first item and first tile of the sequence
};
struct Scan {
  int64_t red[4][2];
  int64_t found[3];
};
// Total tiles of a key head.
__device__ __forceinline__ int64_t total_tiles(const Walk& w, Scan& sc) {
  int64_t mine = 0;
  for (int s = threadIdx.x; s < w.batch.nseq; s += 256) {
    const Seq q = w.seq(s);
    mine += (int64_t)w.items(q) * w.tiles(q);
  }
  int64_t b0, b1, all, none;
  scan2(mine, 0, &b0, &b1, &all, &none, sc.red);
  return all;
}
// The sequence that holds tile `tile` (want < 0), or the place of sequence `want`.
__device__ __forceinline__ Place locate(const Walk& w, int64_t tile, int want, Scan& sc) {
  if (threadIdx.x == 0) sc.found[0] = -1;
  int64_t item0 = 0, tile0 = 0;
  for (int base = 0; base < w.batch.nseq; base += 256) {
    const int s = base + threadIdx.x;
    int64_t it = 0, ti = 0;
    if (s < w.batch.nseq) {
      const Seq q = w.seq(s);
      it = w.items(q), ti = it * w.tiles(q);
    }
    int64_t bi, bt, ai, at;
    scan2(it, ti, &bi, &bt, &ai, &at, sc.red);
    bi += item0, bt += tile0;
    if (s < w.batch.nseq && (want >= 0 ? s == want : tile >= bt && tile < bt + ti))
      sc.found[0] = s, sc.found[1] = bi, sc.found[2] = bt;
    item0 += ai, tile0 += at;
  }
  __syncthreads();
  return Place{(int)sc.found[0], sc.found[1], sc.found[2]};
}

struct RowsArgs {
  CacheView cache;
  CacheBatch batch;
  CacheTensor q, out;
  int group, heads, causal, capacity, direct;
  int64_t workers, items;
  float scale;
  float* slots;
};

// Tiles of a worker: at least one.
__device__ __forceinline__ int64_t share(int64_t total, int64_t workers) {
  return max((total + workers - 1) / workers, (int64_t)1);
}

// Attention of 16 rows at a time: worker w of a key head takes the tiles w c ..
// w c + c - 1 of all items in a row, and each of its waves 32 tokens of a tile.
template <typename T, int D, int BITS>
__global__ __launch_bounds__(256) void attend_rows(const RowsArgs a) {
  using R = Record<D, BITS>;
  constexpr int PARTS = std::is_same_v<T, float> ? 2 : 1;
  constexpr int J = D / 32, N = D / 16, KW = R::lane_bytes / 4;
  __shared__ Scan sc;
  __shared__ float sm[4][kRows], sl[4][kRows];
  __shared__ float so[4][kRows][D + 4];
  const int h = (int)(block_index() % a.cache.heads);
  const int64_t w = block_index() / a.cache.heads;
  if (w >= a.workers) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, col = lane & 15;
  const Walk walk{a.batch, &a.cache, a.group, a.capacity};
  const int64_t total = total_tiles(walk, sc);
  const int64_t c = share(total, a.workers);
  const int64_t end = min(total, (w + 1) * c);
  int64_t at = w * c;
  if (at >= end) return;
  __syncthreads();
  const Place place = locate(walk, at, -1, sc);
  if (place.seq < 0) return;
  int s = place.seq;
  int64_t item0 = place.item, tile0 = place.tile;
  Seq q = walk.seq(s);
  int per = walk.tiles(q), count = walk.items(q);
  while (at < end) {
    while (at >= tile0 + (int64_t)per * count) {       // the next sequence with tiles
      tile0 += (int64_t)per * count, item0 += count;
      if (++s >= a.batch.nseq) return;
      q = walk.seq(s);
      per = walk.tiles(q), count = walk.items(q);
    }
    const int in = (int)((at - tile0) / per);          // item of the sequence
    const int64_t item_tile = tile0 + (int64_t)in * per;
    const int ta = (int)(at - item_tile), tb = (int)min((int64_t)per, end - item_tile);
    const int64_t item = item0 + in;
    at = item_tile + tb;
    if (item >= a.items) return;                       // starts that descend
    const int rows = (int)min((int64_t)kRows, (int64_t)(q.r1 - q.r0) * a.group - in * kRows);
    // this lane's row
    const int r = in * kRows + min(col, rows - 1);
    const int token = r / a.group, head = h * a.group + r % a.group;
    const int visible = min(min(q.len, a.capacity),
                            a.causal ? q.len - (q.r1 - q.r0) + token + 1 : q.len);
    const int least = __shfl(visible, 0, 64), most = __shfl(visible, rows - 1, 64);
    f16x8_t qf[PARTS][J];
    float f;
    {
      const T* src = (const T*)a.q.p + (int64_t)(q.r0 + token) * a.q.ts + head * a.q.hs;
      float x[J][8], top = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[j][e] = load1<T>(src, 32 * j + 8 * g + e);
          top = fmaxf(top, fabsf(x[j][e]));
          if (x[j][e] != x[j][e]) top = __builtin_inff();
        }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const int field = min(267 - (int)(__float_as_uint(top) >> 23), 253);
      const float up = __uint_as_float((uint32_t)max(field, 1) << 23);
      f = top <= __FLT_MAX__ ? fmaxf(__uint_as_float((uint32_t)(254 - max(field, 1)) << 23) *
                                         a.scale * 1.44269504088896340736f, __FLT_MIN__)
                             : __builtin_nanf("");
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = x[j][e] * up;
          const _Float16 hi = (_Float16)v;
          qf[0][j][e] = hi;
          if constexpr (PARTS == 2) qf[1][j][e] = (_Float16)(v - (float)hi);
        }
    }
    float m = kNone, l = 0.0f, ref = 0.0f, inv_ref = 0.0f;
    f32x4_t o[N];
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = f32x4_t{0, 0, 0, 0};
    const int32_t* table = a.batch.table + s * a.batch.ldt;
    for (int tile = ta; tile < tb; ++tile) {
      const int block = tile * 4 + wave, p0 = block * 32;
      if (p0 >= most) continue;
      const uint8_t* rec = record_of(a.cache, table, a.batch.width, block, h);
      if (!rec) continue;
      uint32_t kr[KW], vr[KW], kw[2], kx[2][4], vx[2][4];
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        kr[i] = ((const uint32_t*)(rec + i / 4 * 1024 + lane * 16))[i % 4];
        vr[i] = ((const uint32_t*)(rec + R::codes + i / 4 * 1024 + lane * 16))[i % 4];
      }
      const uint32_t* words = (const uint32_t*)(rec + R::words);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        kw[t] = words[16 * t + col];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          kx[t][i] = words[16 * t + 4 * g + i];
          vx[t][i] = words[32 + 16 * t + 4 * g + i];
        }
      }
      if (p0 + 32 > most) {                              // tokens that no row sees
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p0 + 16 * t + 4 * g + i >= most) kx[t][i] = vx[t][i] = 0;
      }
      // scores
      float p[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4_t acc{0, 0, 0, 0};
        const int z = word_zero(kw[t]);
        const uint32_t b0 = bias0(z, z), b4 = bias4(z, z);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          uint4 frag;
          if constexpr (BITS == 8) {
            const uint32_t w0 = kr[(t * J + j) * 2], w1 = kr[(t * J + j) * 2 + 1];
            frag = make_uint4(bytes_less(w0, 0x04010400u, b0), bytes_less(w0, 0x04030402u, b0),
                              bytes_less(w1, 0x04010400u, b0), bytes_less(w1, 0x04030402u, b0));
          } else {
            const uint32_t w0 = kr[t * J + j], w1 = w0 >> 8;
            frag = make_uint4(low_less(w0, b0), high_less(w0, b4), low_less(w1, b0),
                              high_less(w1, b4));
          }
#pragma unroll
          for (int part = 0; part < PARTS; ++part) acc = mfma(as_half8(frag), qf[part][j], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[t][i] = acc[i] * word_step(kx[t][i]);
          if (p0 + 16 * t + 4 * g + i >= visible) p[t][i] = kNone;
        }
      }
      float top = kNone;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, p[t][i]);
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float next = fmaxf(m, top), base = next == kNone ? 0.0f : next * f;
      // larger steps of the values than ref allows
      float most_step = 0.0f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) most_step = fmaxf(most_step, word_step(vx[t][i]));
      float scale_o = m == kNone ? 0.0f : exp2f(fmaf(m, f, -base));
      l *= scale_o;
      if (__any(most_step > ref * 128.0f)) {
        most_step = fmaxf(most_step, __shfl_xor(most_step, 16, 64));
        most_step = fmaxf(most_step, __shfl_xor(most_step, 32, 64));
        const float old = ref;
        // 2^e <= most_step, within 2^-100 .. 2^100
        ref = __uint_as_float(__float_as_uint(fminf(fmaxf(most_step, 0x1p-100f), 0x1p100f)) &
                              0x7f800000u);
        inv_ref = 256.0f / ref;
        scale_o *= old / ref;
      }
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] *= scale_o;
      m = next;
      uint4 pf[PARTS];
      {
        float x[8], y[8];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = exp2f(fmaf(p[t][i], f, -base));
            l += e;
            const bool seen = p0 + 16 * t + 4 * g + i < visible;
            x[4 * t + i] = seen ? e * (word_step(vx[t][i]) * inv_ref) : 0.0f;
          }
        // the order of a value fragment's tokens
        constexpr int B = BITS == 8 ? 1 : 2, C = BITS == 8 ? 2 : 1;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = (float)(_Float16)x[e];
          pf[part] = make_uint4(two_halves(x[0], x[B]), two_halves(x[C], x[3]),
                                two_halves(x[4], x[4 + B]), two_halves(x[4 + C], x[7]));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] -= y[e];
        }
      }
      // values
      uint32_t z0[4], z4[4];
      {
        constexpr int B = BITS == 8 ? 1 : 2, C = BITS == 8 ? 2 : 1;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          int z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = word_zero(vx[t][i]);
          z0[2 * t] = bias0(z[0], z[B]), z0[2 * t + 1] = bias0(z[C], z[3]);
          z4[2 * t] = bias4(z[0], z[B]), z4[2 * t + 1] = bias4(z[C], z[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        uint4 frag;
        if constexpr (BITS == 8) {
          const uint32_t w0 = vr[2 * n], w1 = vr[2 * n + 1];
          frag = make_uint4(bytes_less(w0, 0x04010400u, z0[0]), bytes_less(w0, 0x04030402u, z0[1]),
                            bytes_less(w1, 0x04010400u, z0[2]), bytes_less(w1, 0x04030402u, z0[3]));
        } else {
          const uint32_t w0 = vr[n / 2 * 2], w1 = vr[n / 2 * 2 + 1];
          if (n % 2 == 0)
            frag = make_uint4(low_less(w0, z0[0]), low_less(w0 >> 8, z0[1]), low_less(w1, z0[2]),
                              low_less(w1 >> 8, z0[3]));
          else
            frag = make_uint4(high_less(w0, z4[0]), high_less(w0 >> 8, z4[1]),
                              high_less(w1, z4[2]), high_less(w1 >> 8, z4[3]));
        }
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
          o[n] = mfma(as_half8(frag), as_half8(pf[part]), o[n]);
      }
    }
    // the four waves' results
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    const float m2 = m == kNone ? kNone : m * f;
    __syncthreads();
    if (g == 0) sm[wave][col] = m2, sl[wave][col] = l;
    __syncthreads();
    float all = kNone, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) all = fmaxf(all, sm[i][col]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += sm[i][col] == kNone ? sl[i][col] : sl[i][col] * exp2f(sm[i][col] - all);
    const float part = m2 == kNone ? 1.0f : exp2f(m2 - all);
    const float back = ref * (1.0f / 256.0f);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) so[wave][col][16 * n + 4 * g + i] = o[n][i] * part * back;
    __syncthreads();
    const bool whole = a.direct && ta == 0 && tb == per;
    float* slot = a.slots + ((int64_t)h * (a.workers + a.items) + w + item) * kSlot<D>;
    for (int i = threadIdx.x; i < rows * D; i += 256) {
      const int row = i / D, d = i % D;
      const float v = so[0][row][d] + so[1][row][d] + so[2][row][d] + so[3][row][d];
      if (whole) {
        float total_l = 0.0f, top = kNone;
        for (int k = 0; k < 4; ++k) top = fmaxf(top, sm[k][row]);
        for (int k = 0; k < 4; ++k)
          total_l += sm[k][row] == kNone ? sl[k][row] : sl[k][row] * exp2f(sm[k][row] - top);
        const int rr = in * kRows + row;
        const int64_t to = (int64_t)(q.r0 + rr / a.group) * a.out.ts +
                           (int64_t)(h * a.group + rr % a.group) * a.out.hs + d;
        const float y = total_l == 0.0f ? 0.0f : v / total_l;
        if constexpr (std::is_same_v<T, float>) ((float*)a.out.p)[to] = y;
        else ((__bf16*)a.out.p)[to] = (__bf16)y;
      } else {
        slot[i] = v;
      }
    }
    if (!whole && wave == 0 && g == 0) {
      slot[kRows * D + col] = all;
      slot[kRows * D + kRows + col] = sum;
    }
  }
}

struct JoinArgs {
  RowsArgs own, before;        // before.workers 0: no prefix
};

// A row's results from the workers that had tiles of its item, and from those of
// the prefix: a workgroup per row.
template <typename T, int D>
__global__ __launch_bounds__(256) void join_rows(const JoinArgs j) {
  const RowsArgs& a = j.own;
  __shared__ Scan sc;
  __shared__ float sm[4], sl[4], so[4][D];
  const int64_t b = block_index();
  const int head = (int)(b % a.heads), h = head / a.group;
  if (b / a.heads >= a.batch.ntok) return;
  const int t = (int)(b / a.heads);
  const int s = find_sequence(a.batch, t);
  if (s < 0) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  constexpr int E = D / 64;
  float m = kNone, l = 0.0f, o[E] = {};
  bool any = false;
  for (int of = 0; of < 2; ++of) {
    const RowsArgs& r = of ? j.before : j.own;
    if (r.workers == 0) continue;
    const Walk walk{r.batch, &r.cache, r.group, r.capacity};
    const int own = of ? 0 : s;
    const Seq q = walk.seq(own);
    const int per = walk.tiles(q);
    const int64_t row = (int64_t)(t - q.r0) * r.group + head % r.group;
    const int64_t total = total_tiles(walk, sc);
    __syncthreads();
    const Place place = locate(walk, 0, own, sc);
    __syncthreads();
    if (per == 0) continue;
    const int64_t c = share(total, r.workers), item = place.item + row / kRows;
    const int64_t first = place.tile + row / kRows * per;
    const int64_t w0 = first / c, w1 = (first + per - 1) / c;
    if (item >= r.items) continue;
    if (w0 == w1 && r.direct) return;                  // written already
    any = true;
    for (int64_t w = w0 + wave; w <= w1; w += 4) {
      const float* slot = r.slots + ((int64_t)h * (r.workers + r.items) + w + item) * kSlot<D>;
      const int k = (int)(row % kRows);
      const float pm = slot[kRows * D + k], pl = slot[kRows * D + kRows + k];
      const float next = fmaxf(m, pm), base = next == kNone ? 0.0f : next;
      const float fm = exp2f(m - base), fp = pm == kNone ? 1.0f : exp2f(pm - base);
      l = l * fm + pl * fp;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * fm + slot[k * D + lane * E + e] * fp;
      m = next;
    }
  }
  if (lane == 0) sm[wave] = m, sl[wave] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[wave][lane * E + e] = o[e];
  __syncthreads();
  float all = kNone, sum = 0.0f;
  for (int i = 0; i < 4; ++i) all = fmaxf(all, sm[i]);
  float fac[4];
  for (int i = 0; i < 4; ++i) {
    fac[i] = sm[i] == kNone ? 1.0f : exp2f(sm[i] - all);
    sum += sl[i] * fac[i];
  }
  for (int d = threadIdx.x; d < D; d += 256) {
    float v = 0.0f;
    for (int i = 0; i < 4; ++i) v += so[i][d] * fac[i];
    const float y = !any || sum == 0.0f ? 0.0f : v / sum;
    const int64_t to = (int64_t)t * a.out.ts + (int64_t)head * a.out.hs + d;
    if constexpr (std::is_same_v<T, float>) ((float*)a.out.p)[to] = y;
    else ((__bf16*)a.out.p)[to] = (__bf16)y;
  }
}

int capacity_of(const CacheBatch& b, int blocks_shift) {
  return (int)std::min<int64_t>((int64_t)b.width << (blocks_shift + 5), INT32_MAX - 65535);
}

template <typename T, int D, int BITS>
void launch_all(const JoinArgs& j, hipStream_t st) {
  for (const RowsArgs* r : {&j.before, &j.own})
    if (r->workers)
      attend_rows<T, D, BITS><<<block_grid(r->workers * r->cache.heads), 256, 0, st>>>(*r);
  join_rows<T, D><<<block_grid((int64_t)j.own.batch.ntok * j.own.heads), 256, 0, st>>>(j);
}

template <typename T, int D>
void launch_bits(const JoinArgs& j, int bits, hipStream_t st) {
  if (bits == 8) launch_all<T, D, 8>(j, st);
  else launch_all<T, D, 4>(j, st);
}

template <typename T>
void launch_dim(const JoinArgs& j, int dim, int bits, hipStream_t st) {
  if (dim == 64) launch_bits<T, 64>(j, bits, st);
  else if (dim == 128) launch_bits<T, 128>(j, bits, st);
  else launch_bits<T, 256>(j, bits, st);
}

}  // namespace

AttentionPlan attention_plan(const AttentionLaunch& a) {
  AttentionPlan p{};
  const int64_t group = a.heads / a.cache.heads, rows = (int64_t)a.batch.ntok * group;
  p.workers = std::max<int64_t>(1, 512 / a.cache.heads);
  p.items = rows / kRows + std::min<int64_t>(a.batch.nseq, a.batch.ntok) + 1;
  p.prefix_items = a.prefix.nseq ? (rows + kRows - 1) / kRows : 0;
  const int64_t slot = kRows * (a.head_dim + 2) * 4;
  p.own_bytes = (p.workers + p.items) * a.cache.heads * slot;
  p.prefix_bytes = p.prefix_items ? (p.workers + p.prefix_items) * a.cache.heads * slot : 0;
  return p;
}

hipError_t launch_cached_attention(const AttentionLaunch& a, const AttentionPlan& p, void* own,
                                   void* prefix, hipStream_t st) {
  if (a.batch.ntok == 0 || a.batch.nseq == 0) return hipSuccess;
  JoinArgs j{};
  j.own = RowsArgs{a.cache, a.batch, a.q, a.out, a.heads / a.cache.heads, a.heads, a.causal,
                   capacity_of(a.batch, a.cache.blocks_shift), a.prefix.nseq == 0, p.workers,
                   p.items, a.scale, (float*)own};
  if (a.prefix.nseq) {
    j.before = j.own;
    j.before.batch = a.prefix;
    j.before.batch.starts = a.batch.starts;
    j.before.batch.starts_step = a.batch.nseq;
    j.before.batch.ntok = a.batch.ntok;
    j.before.causal = 0;
    j.before.direct = 0;
    j.before.capacity = capacity_of(a.prefix, a.cache.blocks_shift);
    j.before.items = p.prefix_items;
    j.before.slots = (float*)prefix;
  }
  if (a.dtype == PWQ_F32) launch_dim<float>(j, a.head_dim, a.bits, st);
  else launch_dim<uint16_t>(j, a.head_dim, a.bits, st);
  return hipGetLastError();
}

}  // namespace pwq
