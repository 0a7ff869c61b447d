// y = x W^^T of a packed layer for more than 16 tokens: tiles of BT tokens x
// BR rows on the matrix cores.
//
//   y[t, r] = x_scale[t] * sum_g s[r, g] * sum_{k in g} x[t, k] (c - z)[r, k]
//
// The inner sum runs over integers c - z: v_mfma_i32_16x16x64_i8 for 8-bit x
// (exact int32 sums), v_mfma_f32_16x16x32_bf16 otherwise (c - z is exact in
// bf16, products are exact in float32).  A float32 x is the sum of three bf16
// parts (the top, middle and last 8 bits of its significand), each of which
// runs over the same weights.
//
// Up to a few hundred tokens batch_tiles reads the packed codes and spreads them
// itself.  With more, every tile of tokens would repeat that on the vector
// unit, which the multiplication by the steps already fills: spread_weights
// writes the integers c - z (overflow entries added) once per call in the
// operands' order, a wave's operand a contiguous kilobyte, and prompt_tiles
// multiplies.
//
// A step of prompt_tiles covers 128 bytes of every x row (128 8-bit or 64 bf16
// columns).  Two steps ahead of their use, x goes HBM -> LDS by asynchronous
// copies through three slots (LDS rows are 128 bytes, their 16-byte units
// permuted by the row so that 16 rows' reads of one column block cover every
// bank) and weights straight to registers.  A wave works on all of the tile's
// tokens and 32 rows, so that a workgroup reads every weight once; waves of 64
// x 64 read each twice, and a CU's 2 x 24 instead of 2 x 16 KB of a step took
// 512 bf16 tokens of up_proj from 63 to 72 us.  Two workgroups' waves to a
// SIMD at most: with that bound the compiler sums in vector registers, without
// it in accumulation registers, whose reads double the vector instructions (81
// us).
//
// What bounds it: the matrix instructions and the multiplications of their sums
// by the steps on the vector unit, which follow each other more than they
// overlap, and the wait at every step's barrier.  Of a tile's cycles the matrix
// unit is busy 37% and the vector unit 44% for 2048 8-bit tokens of up_proj
// (groups of 128), 44% and 26% for 1024 bf16 tokens of down_proj (64).  Tiles alone take 254 to 296 us (as the clock
// goes) for 2048 bf16 tokens of up_proj and 146 to 163 us in 8 bits (0.95 and
// 1.65 P(FL)OP/s at best), 206 and 105 us with one step per row; 8192 tokens 961
// and 596 us with everything (1.00 and 1.61 P(FL)OP/s).  The library's products
// of the first size take 207 us (bf16) and, at its 8192^3 rate, 115 us (8 bits).
#include "pwq_internal.h"

#include <algorithm>

namespace pwq {
namespace {

constexpr int KB = 128;            // bytes of an x row per step

// Byte of 16-byte unit c of LDS row r.
__device__ __forceinline__ uint32_t unit_at(int r, int c) {
  return (uint32_t)(r * KB + ((c ^ ((r >> 1) & 7)) << 4));
}

template <bool I8> using sum_t = std::conditional_t<I8, i32x4_t, f32x4_t>;

template <bool I8>
__device__ __forceinline__ sum_t<I8> mma(const i32x4_t& x, const i32x4_t& w, const sum_t<I8>& c) {
  if constexpr (I8) return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, w, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x),
                                                   __builtin_bit_cast(bf16x8_t, w), c, 0, 0, 0);
}

// What a group's sum starts from, and its value.  1.5 2^23 as an integer: int32
// sums below 2^22 that start here read as 1.5 2^23 + sum when taken for a
// float32.
constexpr int kMagic = 0x4b400000;
template <bool I8> __device__ __forceinline__ sum_t<I8> sum_start() {
  if constexpr (I8) return i32x4_t{kMagic, kMagic, kMagic, kMagic};
  else return f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
}
__device__ __forceinline__ float sum_value(const i32x4_t& c, int e) {
  return __int_as_float(c[e]) - 12582912.0f;
}
__device__ __forceinline__ float sum_value(const f32x4_t& c, int e) { return c[e]; }

struct PromptArgs {
  const char* x;          // rows of `steps` * 128 bytes, 16-byte aligned
  int64_t xrow;           // bytes between x rows
  int steps;              // steps over the whole row
  int reps;               // steps per weight block: 1, or 3 parts of float32
  int per;                // steps (batch_tiles: tiles of 128 columns) per split
  int tiles_t, tiles_r;
  const float* x_scales;
  // packed weights (batch_tiles)
  const uint8_t* qweight;
  int64_t ldq;
  const float* scales;
  const uint8_t* zeros;
  const int32_t* off;
  const int32_t* outliers;
  int n_out;
  const i32x4_t* spread;  // [strip of 16 rows][weight block][half][lane]
  int blocks;             // weight blocks (steps / reps)
  const float* steps_t;   // [group][16 strips' rows], times what the operands leave out
  int64_t rows16;         // rows of it: 16 strips
  int ntok, m, n, ng;
  uint32_t per_group;     // 2^31 / half steps of a group, rounded up: 2 u per_group / 2^32 is
                          // the group of half step u < 2^16 (at most 2^15 to a group)
  void* y;
  int ydtype;
  int64_t ldy;
  float* partial;         // splits x ntok x m, or NULL
};

// First token and row of this workgroup's tile; false past the last one.  XCD b
// % 8 owns a contiguous range of tiles, tokens fastest, so that its L2 holds
// the weights of a few row tiles.
__device__ __forceinline__ bool tile_of(const PromptArgs& a, int bt, int br, int& t0, int& r0) {
  const int tiles = a.tiles_t * a.tiles_r;
  const int b = blockIdx.x, x = b & 7, q = tiles / 8, r = tiles % 8;
  const int tile = x * q + min(x, r) + (b >> 3);
  t0 = tile % a.tiles_t * bt;
  r0 = tile / a.tiles_t * br;
  return (b >> 3) < q + (x < r ? 1 : 0);
}

// The operand integers of 16 rows x 128 columns (one wave each) in 8 bits or
// bf16, and the steps of the groups that start there, group by group.
template <bool I8>
__global__ __launch_bounds__(256) void spread_weights(
    const uint8_t* __restrict__ qweight, int64_t ldq, const float* __restrict__ scales,
    const uint8_t* __restrict__ zeros, const int32_t* __restrict__ off,
    const int32_t* __restrict__ outliers, int n_out, int64_t m, int n, int G, int ng,
    int across, int64_t tiles, i32x4_t* __restrict__ spread, int blocks,
    float* __restrict__ steps_t, int64_t rows16) {
  constexpr int ROW = 128 + 16;                        // bytes of a row in LDS
  __shared__ __attribute__((aligned(16))) char smem[4][16 * ROW];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = block_index() * 4 + wave;
  if (tile >= tiles) return;
  char* const L = smem[wave];
  const int64_t strip = tile / across;
  const int kt = (int)(tile - strip * across), k0 = kt * 128;
  // packed bytes: lane -> row lane / 4, 32 columns
  const int r = lane >> 2, kc = k0 + 32 * (lane & 3);
  const int64_t row = min(strip * 16 + r, m - 1);
  uint4 w = make_uint4(0, 0, 0, 0);
  if (kc / 2 < ldq) w = *(const uint4*)(qweight + row * ldq + kc / 2);
  const int z = zeros ? zeros[row * ng + min(kc / G, ng - 1)] : 8;
  const uint32_t z4 = (uint32_t)z * 0x01010101u, flip = zeros ? 0u : 0x88888888u;
  {
    const uint2 p0 = steps_i8(w.x ^ flip, z4), p1 = steps_i8(w.y ^ flip, z4);
    const uint2 p2 = steps_i8(w.z ^ flip, z4), p3 = steps_i8(w.w ^ flip, z4);
    char* d = L + r * ROW + 32 * (lane & 3);
    *(uint4*)d = make_uint4(p0.x, p0.y, p1.x, p1.y);
    *(uint4*)(d + 16) = make_uint4(p2.x, p2.y, p3.x, p3.y);
  }
  if (n_out > 0) {
    // the wave's own LDS: its writes above are in order with these
    const int e0 = max(off[tile], 0), e1 = min(off[tile + 1], n_out);
    for (int e = e0 + lane; e < e1; e += 64) {
      const int v = outliers[e];
      int8_t* d = (int8_t*)(L + ((v >> 7) & 15) * ROW + (v & 127));
      *d = (int8_t)(*d + (v >> 16));
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int lr = lane & 15, lq = lane >> 4;
  if constexpr (I8) {
    i32x4_t* const o = spread + (strip * blocks + kt) * 128 + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) o[64 * h] = *(const i32x4_t*)(L + lr * ROW + 64 * h + 16 * lq);
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (2 * kt + b >= blocks) break;
      i32x4_t* const o = spread + (strip * blocks + 2 * kt + b) * 128 + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int8_t c[8];
        __builtin_memcpy(c, L + lr * ROW + 64 * b + 32 * h + 8 * lq, 8);
        i32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i)                    // (small integers: exact in bf16)
          v[i] = (int)__builtin_amdgcn_perm(__float_as_uint((float)c[2 * i + 1]),
                                            __float_as_uint((float)c[2 * i]), 0x07060302u);
        o[64 * h] = v;
      }
    }
  }
  // steps, transposed: groups starting in the tile
  for (int g = (k0 + G - 1) / G; g < ng && g * G < k0 + 128; ++g)
    if (lane < 16) steps_t[g * rows16 + strip * 16 + lane] =
        scales[min(strip * 16 + lane, m - 1) * ng + g];
}

// A tile's sums to y, or to its split's part of the partial sums.  Lane l holds
// tokens 4 (l / 16) + e, row l % 16 of every block; smem: BT rows of y, free.
template <int BT, int BR> constexpr int kYBytes = BT * (2 * BR + 32);
template <int BT, int BR, int NT>
__device__ __forceinline__ void store_tile(const PromptArgs& a,
                                           float (&acc)[BT / 16][BR / 16 * 64 / NT][4], char* smem,
                                           int t0, int r0, int split) {
  constexpr int NI = BT / 16, NJ = BR / 16 * 64 / NT, YROW = 2 * BR + 32;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool split_sum = a.partial != nullptr;
  if (a.x_scales && !split_sum) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float xsc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        xsc[e] = a.x_scales[min(t0 + 16 * i + 4 * lq + e, a.ntok - 1)];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] *= xsc[e];
    }
  }
  if (split_sum || a.ydtype == PWQ_F32) {
    float* const y = split_sum ? a.partial + (int64_t)split * a.ntok * a.m : (float*)a.y;
    const int64_t ld = split_sum ? a.m : a.ldy;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + 16 * i + 4 * lq + e;
        if (t < a.ntok)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int r = r0 + 16 * (wave * NJ + j) + lr;
            if (r < a.m) y[t * ld + r] = acc[i][j][e];
          }
      }
    return;
  }
  // bf16: through LDS, so that rows of y are written 16 bytes a lane.  Two
  // neighbouring lanes trade halves: the even one packs both their rows of
  // token e, the odd one of token e + 1.
  const bool odd = lane & 1;
  const uint32_t sel = odd ? 0x03020706u : 0x05040100u;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const __bf16 two[2] = {(__bf16)acc[i][j][e], (__bf16)acc[i][j][e + 1]};
        const uint32_t own = __builtin_bit_cast(uint32_t, two);
        const uint32_t other = __builtin_amdgcn_update_dpp(own, own, 0xB1, 0xF, 0xF, false);
        const int t = 16 * i + 4 * lq + e + odd;
        const int r = 16 * (wave * NJ + j) + (lr & ~1);
        *(uint32_t*)(smem + t * YROW + 2 * r) = __builtin_amdgcn_perm(other, own, sel);
      }
  lds_barrier();
  constexpr int LPR = BR / 8;                          // lanes of a row
  __bf16* const y = (__bf16*)a.y;
  const bool whole = (a.ldy * 2) % 16 == 0 && (uintptr_t)a.y % 16 == 0;
  for (int t = tid / LPR; t < BT; t += NT / LPR) {
    const int r = r0 + 8 * (tid % LPR);
    if (t0 + t >= a.ntok || r >= a.m) continue;
    const char* src = smem + t * YROW + 16 * (tid % LPR);
    __bf16* dst = y + (t0 + t) * a.ldy + r;
    if (whole && r + 8 <= a.m) {
      *(uint4*)dst = *(const uint4*)src;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (r + e < a.m) dst[e] = ((const __bf16*)src)[e];
    }
  }
}

// Fewer tokens: tiles of BT tokens x 128 rows that read the packed codes, in
// tiles of 128 columns.  NP: x steps of such a tile (8-bit 1, bf16 2, float32
// 6).  Everything comes by asynchronous copies two tiles ahead: x for the
// workgroup, 32 rows of weights (2 KB), their steps and zero points for the
// wave that spreads them and multiplies by them.  Lanes next to each other copy
// bytes next to each other; loads in the operands' layout, one cache lookup a
// lane, took 33 us for 32 bf16 tokens of up_proj, these 20.  With overflow
// entries (OVER) the codes become bytes in LDS first, where the entries' are
// added (25 us; written to memory spread, 57).  What bounds it: latency with few
// columns a split, then the vector unit's spreading; up_proj 64 8-bit tokens
// 20 us, 1.6 TB/s.
constexpr int kSpreadRow = 128 + 16;                  // bytes of a spread row (OVER)
constexpr int batch_lds(int np, int bt, int sc, bool asym, bool over) {
  return 3 * np * bt * KB + 12 * (2048 + sc * (asym ? 512 : 256) + (over ? 512 : 0)) +
         (over ? 4 * 32 * kSpreadRow : 0);
}
constexpr int batch_steps(bool i8, int mode) {       // copies of 64 steps of a tile
  return mode == 0 ? 0 : (!i8 && mode == 2 ? 2 : 1);
}
template <bool I8, int NP, int BT, int MODE, bool ASYM, bool OVER>
__global__ __launch_bounds__(
    256, batch_lds(NP, BT, batch_steps(I8, MODE), ASYM, OVER) <= 80 * 1024 ? 2 : 1)
void batch_tiles(const PromptArgs a) {
  constexpr int BR = 128, NI = BT / 16, NJ = 2;
  constexpr int SUB = I8 ? 1 : 2, REPS = NP / SUB;      // blocks of a tile, x parts
  constexpr int NS = MODE == 2 ? 2 : 1;                 // steps of a block
  constexpr int SC = batch_steps(I8, MODE);             // SUB NS groups of 32 rows
  constexpr int XS = NP * BT * KB, NC = BT / 32;        // x of a tile; copies of an x step
  constexpr int ES = 2048 + SC * 256 * (ASYM ? 2 : 1);  // overflow entries, of the wave's part
  constexpr int WS = ES + (OVER ? 512 : 0);             // of a tile
  constexpr int COPIES = NP * NC + 2 + SC * (ASYM ? 2 : 1) + (OVER ? 2 : 0);
  constexpr int LDS = batch_lds(NP, BT, SC, ASYM, OVER);
  static_assert(3 * XS + 12 * WS <= LDS && kYBytes<BT, BR> <= LDS, "what is used");
  using acc_t = sum_t<I8>;
  __shared__ __attribute__((aligned(16))) char smem[LDS];
  const uint32_t lbase = (uint32_t)(uintptr_t)(lds_char*)smem;
  int t0, r0;
  if (!tile_of(a, BT, BR, t0, r0)) return;
  const int split = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int across = (a.n + 127) / 128;
  const int k0 = split * a.per, k1 = min(across, k0 + a.per), last = k1 - 1;

  // copies
  uint32_t xoff[NC], woff[2], wcol[2];
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    const int u = 256 * h + tid, r = u >> 3, c = (u & 7) ^ ((r >> 1) & 7);
    xoff[h] = (uint32_t)((min(t0 + r, a.ntok - 1) - t0) * a.xrow + 16 * c);
  }
  const int wr0 = r0 + 32 * wave;                       // the wave's rows
  const int rbase = min(wr0, a.m - 1), rows = min(a.m - rbase, 32);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = lane >> 2, c = (lane & 3) ^ (r >> 2);
    woff[h] = (uint32_t)(min(16 * h + r, rows - 1) * (int)a.ldq);
    wcol[h] = 16u * c;
  }
  const uint32_t srow = (uint32_t)(min(lane & 31, rows - 1) * a.ng);
  const char* const xbase = a.x + (int64_t)t0 * a.xrow;
  const uint8_t* const qbase = a.qweight + (int64_t)rbase * a.ldq;
  const float* const sbase = a.scales + (int64_t)rbase * a.ng;
  const uint8_t* const zbase = ASYM ? a.zeros + (int64_t)rbase * a.ng : nullptr;
  const uint32_t own = 3 * XS + wave * 3 * WS;
  // the overflow list's range for strip j of the wave (nothing past the last)
  const int strips = (a.m + 15) / 16;
  auto range = [&](int kt, int j, int& e0, int& e1) {
    const int st = min(wr0 / 16 + j, strips - 1);
    const const_int* const off = (const const_int*)(a.off + (int64_t)st * across + kt);
    e0 = max(off[0], 0);
    e1 = wr0 / 16 + j < strips ? min(off[1], a.n_out) : e0;
  };
  auto ask = [&](int kt, int slot) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int h = 0; h < NC; ++h)
        copy16(xoff[h], xbase + (int64_t)min(kt * NP + p, a.steps - 1) * KB,
               lbase + slot * XS + p * BT * KB + 4096u * h + 1024u * wave);
    const uint32_t dst = lbase + own + slot * WS;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = 64u * kt + wcol[h];
      copy16(woff[h] + (o < a.ldq ? o : 0), qbase, dst + 1024u * h);
    }
#pragma unroll
    for (int h = 0; h < SC; ++h) {
      // groups 2 h and 2 h + 1 of the tile, 32 rows each
      const uint32_t half = (I8 ? 2 : 4) * kt + (2 / NS) * (2 * h + (lane >> 5));
      const uint32_t at = srow + min((int)__umulhi(2 * half, a.per_group), a.ng - 1);
      copy4(4 * at, sbase, dst + 2048u + 256u * h);
      if constexpr (ASYM) copy1(at, zbase, dst + 2048u + 256u * (SC + h));
    }
    if constexpr (OVER) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        int e0, e1;
        range(kt, j, e0, e1);
        e0 = min(e0, a.n_out - 1);
        copy4(4u * min(lane, a.n_out - 1 - e0), a.outliers + e0, dst + ES + 256u * j);
      }
    }
  };

  float acc[NI][NJ][4];
  acc_t dir[MODE == 0 ? NI : 1][MODE == 0 ? NJ : 1];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
      if constexpr (MODE == 0) dir[i][j] = acc_t{0, 0, 0, 0};
    }
  float s_row[NJ];                                      // MODE 0
  int z_row[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    s_row[j] = MODE == 0 ? sbase[min(16 * j + lr, rows - 1)] : 0.0f;
    z_row[j] = MODE == 0 && ASYM ? zbase[min(16 * j + lr, rows - 1)] : 8;
  }

  // OVER: a row of 64 columns of a lane, its zero point (MODE 0)
  char* const spread = smem + 3 * XS + 12 * WS + wave * 32 * kSpreadRow;
  const int sr = lane >> 1, sh = lane & 1;
  const int z_lane = OVER && MODE == 0 && ASYM ? zbase[min(sr, rows - 1)] : 8;

  // 16-byte unit of an x row that lane group lq of half h works on: both
  // halves' codes next to each other, unless a half has a step of its own
  constexpr bool PAIRED = MODE != 2;
  auto unit = [&](int h) { return PAIRED ? 2 * lq + h : 4 * h + lq; };
  constexpr int PB = I8 ? 8 : 4;                        // packed bytes of a lane's half
  constexpr uint32_t flip = ASYM ? 0u : 0x88888888u, bias = ASYM ? kUnsignedHalves : kSignedHalves;

  ask(k0, 0);
  ask(min(k0 + 1, last), 1);
  for (int kt = k0, slot = 0; kt < k1; ++kt, slot = slot == 2 ? 0 : slot + 1) {
    // All but the next tile's copies have landed; past the barrier every wave's
    // have, and the slot before this one is free.
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(COPIES) : "memory");
    lds_barrier();
    ask(min(kt + 2, last), slot == 0 ? 2 : slot - 1);
    const char* const ws = smem + own + slot * WS;
    const float* const steps = (const float*)(ws + 2048);
    const int* const zeros = (const int*)(ws + 2048 + 256 * SC);
    if constexpr (OVER) {
      // the wave's integers as bytes, by rows, and the list's added to them
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int unit = (2 * sh + q) ^ ((sr & 15) >> 2);
        const uint4 p = *(const uint4*)(ws + 1024 * (sr >> 4) + 64 * (sr & 15) + 16 * unit);
        const int slot_z = (2 * sh + q) * SUB * NS / 4;
        const int z = MODE != 0 && ASYM ? zeros[32 * slot_z + sr] : z_lane;
        const uint32_t z4 = (uint32_t)z * 0x01010101u;
        const uint2 p0 = steps_i8(p.x ^ flip, z4), p1 = steps_i8(p.y ^ flip, z4);
        const uint2 p2 = steps_i8(p.z ^ flip, z4), p3 = steps_i8(p.w ^ flip, z4);
        char* const d = spread + sr * kSpreadRow + 64 * sh + 32 * q;
        *(uint4*)d = make_uint4(p0.x, p0.y, p1.x, p1.y);
        *(uint4*)(d + 16) = make_uint4(p2.x, p2.y, p3.x, p3.y);
      }
      // (a wave's LDS accesses are in order)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        int e0, e1;
        range(kt, j, e0, e1);
        for (int e = e0 + lane; e < e1; e += 64) {
          const int v = e - e0 < 64 ? *(const int*)(ws + ES + 256 * j + 4 * lane) : a.outliers[e];
          int8_t* const d = (int8_t*)(spread + (16 * j + ((v >> 7) & 15)) * kSpreadRow + (v & 127));
          *d = (int8_t)(*d + (v >> 16));
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
      if (SUB * kt + sub >= a.blocks) break;
      i32x4_t w[NJ][2];
      float sc[NJ][NS];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int o = 32 * sub + (PAIRED ? 2 * PB * lq + PB * h : 4 * PB * h + PB * lq);
          uint32_t p[PB / 4];
          __builtin_memcpy(p, ws + 1024 * j + 64 * lr + (((o >> 4) ^ (lr >> 2)) << 4) + (o & 15),
                           PB);
          const int at = 32 * (sub * NS + (NS == 2 ? h : 0)) + 16 * j + lr;
          if (MODE != 0 && h < NS) sc[j][h] = steps[at];
          if constexpr (OVER) {
            const char* const c = spread + (16 * j + lr) * kSpreadRow + 2 * o;
            if constexpr (I8) {
              w[j][h] = *(const i32x4_t*)c;
            } else {
              int8_t v[8];
              __builtin_memcpy(v, c, 8);
#pragma unroll
              for (int i = 0; i < 4; ++i)            // (small integers: exact in bf16)
                w[j][h][i] = (int)__builtin_amdgcn_perm(__float_as_uint((float)v[2 * i + 1]),
                                                        __float_as_uint((float)v[2 * i]),
                                                        0x07060302u);
            }
            continue;
          }
          const int z = MODE != 0 && ASYM ? zeros[at] : z_row[j];
          if constexpr (I8) {
            const uint32_t z4 = (uint32_t)z * 0x01010101u;
            const uint2 lo = steps_i8(p[0] ^ flip, z4), hi = steps_i8(p[1] ^ flip, z4);
            w[j][h] = i32x4_t{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
          } else {
            w[j][h] = __builtin_bit_cast(i32x4_t, steps_bf16(p[0], bias, z));
          }
        }
      }
      acc_t c[NI][NJ][NS];
#pragma unroll
      for (int part = 0; part < REPS; ++part) {
        const char* const xs = smem + slot * XS + (sub * REPS + part) * BT * KB;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          i32x4_t x[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x[h] = *(const i32x4_t*)(xs + unit_at(16 * i + lr, unit(h)));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              if constexpr (MODE == 0) {
                dir[i][j] = mma<I8>(x[h], w[j][h], dir[i][j]);
              } else {
                acc_t& o = c[i][j][NS == 2 ? h : 0];
                const bool first = part == 0 && (NS == 2 || h == 0);
                o = mma<I8>(x[h], w[j][h], first ? sum_start<I8>() : o);
              }
            }
        }
      }
      if constexpr (MODE != 0)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int h = 0; h < NS; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                acc[i][j][e] = fmaf(sc[j][h], sum_value(c[i][j][h], e), acc[i][j][e]);
                pin(acc[i][j][e]);
              }
    }
  }
  // nothing is in flight to LDS, and no wave reads it, at the end
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();
  if constexpr (MODE == 0) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = s_row[j] * (float)dir[i][j][e];
  }
  store_tile<BT, BR, 256>(a, acc, smem, t0, r0, split);
}

// MODE: how often sums are multiplied by their step.  0: one step per row,
// at the end; 1: every step (G a multiple of its columns); 2: twice a step.
template <bool I8, int BT, int BR, int WR, int MODE>
__global__ __launch_bounds__(64 * WR, 2) void prompt_tiles(const PromptArgs a) {
  constexpr int NT = 64 * WR;
  constexpr int NI = BT / 16, NJ = BR / WR / 16;
  constexpr int COLS = I8 ? 128 : 64;         // columns of a step
  constexpr int XB = BT * KB;
  constexpr int NC = XB / (16 * NT);          // copies of a wave per step
  constexpr int LDS = 3 * XB > kYBytes<BT, BR> ? 3 * XB : kYBytes<BT, BR>;
  static_assert(NC * 16 * NT == XB, "tile and threads fit");
  using acc_t = sum_t<I8>;
  __shared__ __attribute__((aligned(16))) char smem[LDS];
  lds_char* L = (lds_char*)smem;
  const uint32_t lbase = (uint32_t)(uintptr_t)L;

  int t0, r0;
  if (!tile_of(a, BT, BR, t0, r0)) return;
  const int split = blockIdx.y;
  const int s0 = split * a.per, s1 = min(a.steps, s0 + a.per);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // x copies: copy h of this lane fills unit 64 (NT / 64 h + wave) + lane
  uint32_t xoff[NC];
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    const int u = NT * h + 64 * wave + lane, r = u >> 3, c = (u & 7) ^ ((r >> 1) & 7);
    xoff[h] = (uint32_t)((min(t0 + r, a.ntok - 1) - t0) * a.xrow + 16 * c);
  }
  const char* xbase = a.x + (int64_t)t0 * a.xrow;
  auto copy_x = [&](int s, int slot) {
    const uint32_t dst = lbase + (uint32_t)slot * XB + 1024u * wave;
#pragma unroll
    for (int h = 0; h < NC; ++h) copy16(xoff[h], xbase + (int64_t)s * KB, dst + 16u * NT * h);
  };

  // weights: block j of this wave is strip r0 / 16 + wave NJ + j (the last one
  // again past the end); wave-uniform bases, the lane's offset is the same
  const int lr = lane & 15, lq = lane >> 4;
  auto strip = [&](int j) {
    return min(r0 / 16 + wave * NJ + j, (int)(a.rows16 / 16) - 1);
  };
  constexpr int NS = MODE == 2 ? 2 : 1;
  constexpr int NX = 4;                       // operands of x, read three ahead
  struct Weights {
    i32x4_t w[NJ][2];
    float s[NJ][NS];
  };
  auto block_of = [&](int s) { return a.reps == 1 ? s : s / 3; };
  auto load_w = [&](Weights& b, int s) {
    const int blk = block_of(s);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b.w[j][h] =
            (a.spread + ((int64_t)strip(j) * a.blocks + blk) * 128 + 64 * h)[(uint32_t)lane];
  };
  auto load_s = [&](Weights& b, int s) {
    if constexpr (MODE == 0) return;
    const int blk = block_of(s);
#pragma unroll
    for (int h = 0; h < NS; ++h) {
      const int g = min((int)__umulhi(4 * blk + 2 * h, a.per_group), a.ng - 1);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        b.s[j][h] = (a.steps_t + g * a.rows16 + 16 * strip(j))[(uint32_t)lr];
    }
  };
  // the compiler waits for the weights' registers here
  auto arrived = [&](Weights& b) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      asm volatile("" : "+v"(b.w[j][0]), "+v"(b.w[j][1])::"memory");
  };

  float acc[NI][NJ][4];
  acc_t dir[MODE == 0 ? NI : 1][MODE == 0 ? NJ : 1];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
      if constexpr (MODE == 0) dir[i][j] = acc_t{0, 0, 0, 0};
    }

  const acc_t zero = sum_start<I8>();
  // prologue: steps s0 and s0 + 1 on their way
  const int last = s1 - 1;
  Weights b[3];
  auto ask = [&](int s, int slot, Weights& b) {
    load_s(b, s);
    copy_x(s, slot);
    load_w(b, s);
  };
  ask(s0, 0, b[0]);
  ask(min(s0 + 1, last), 1, b[1]);

  auto step = [&](int s, int slot, Weights& b, Weights& bn) {
    // This step's x and weights, asked for two steps ago, have arrived: the
    // weights came last and loads return in order, so that the wait for the
    // weights' registers covers the x of this wave.  Past the barrier every
    // wave's part of this step's x is there, and the slot before it is free.
    arrived(b);
    lds_barrier();
    ask(min(s + 2, last), (slot + 2) % 3, bn);
    const char* xs = smem + slot * XB;
    i32x4_t x[NX][2];
    i32x4_t(&w)[NJ][2] = b.w;
    float(&sc)[NJ][NS] = b.s;
    auto read_x = [&](int i) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[i % NX][h] = *(const i32x4_t*)(xs + unit_at(16 * i + lr, 4 * h + lq));
    };
#pragma unroll
    for (int i = 0; i < NX - 1; ++i) read_x(i);
    if constexpr (MODE == 0) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (i + NX - 1 < NI) read_x(i + NX - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NJ; ++j) dir[i][j] = mma<I8>(x[i % NX][h], w[j][h], dir[i][j]);
      }
    } else {
      // Blocks of 16 x 16 in turn: one starts, the one before gets its second
      // half (MODE 1), the third before is multiplied by its step, so that
      // neither waits for a matrix instruction's result.
      constexpr int NU = NI * NJ * NS;
      acc_t c[4];
      auto scale = [&](auto uu, int e0) {
        constexpr int u = decltype(uu)::value;
        constexpr int i = u / NS / NJ, j = u / NS % NJ, h = u % NS;
#pragma unroll
        for (int e = e0; e < e0 + 2; ++e) {
          acc[i][j][e] = fmaf(sc[j][h], sum_value(c[u & 3], e), acc[i][j][e]);
          pin(acc[i][j][e]);       // here: not moved behind the other products
        }
      };
      static_for_up<NU + 3>([&](auto uu) {
        constexpr int u = decltype(uu)::value;
        constexpr int i = u / NS / NJ, j = u / NS % NJ, h = u % NS;
        if constexpr (u < NU) {
          c[u & 3] = mma<I8>(x[i % NX][h], w[j][h], zero);
          if constexpr (j == 1 && h == 0 && i + NX - 1 < NI) read_x(i + NX - 1);
        }
        if constexpr (u >= 3) scale(std::integral_constant<int, u - 3>{}, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE == 1 && u > 0 && u <= NU) {
          constexpr int v = u - 1, iv = v / NJ, jv = v % NJ;
          c[v & 3] = mma<I8>(x[iv % NX][1], w[jv][1], c[v & 3]);
        }
        if constexpr (u >= 3) scale(std::integral_constant<int, u - 3>{}, 2);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  };
  int s = s0;
  for (; s + 2 < s1; s += 3) {
    step(s, 0, b[0], b[2]);
    step(s + 1, 1, b[1], b[0]);
    step(s + 2, 2, b[2], b[1]);
  }
  if (s < s1) step(s, 0, b[0], b[2]);
  if (s + 1 < s1) step(s + 1, 1, b[1], b[0]);
  // nothing is in flight to LDS, and no wave reads it, at the end
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();
  if constexpr (MODE == 0) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float sj = a.steps_t[16 * strip(j) + lr];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = sj * (float)dir[i][j][e];
    }
  }

  store_tile<BT, BR, NT>(a, acc, smem, t0, r0, split);
}

// Sum of the splits in their order: a token and 1024 columns per workgroup,
// four a thread (VEC: rows of whole 16-byte units).
template <bool VEC>
__global__ __launch_bounds__(256) void prompt_join(const float* __restrict__ partial, int splits,
                                                   int64_t ntok, int64_t m,
                                                   const float* __restrict__ x_scales, void* y,
                                                   int ydtype, int64_t ldy) {
  const int64_t t = block_index(), r = (int64_t)blockIdx.z * 1024 + 4 * threadIdx.x;
  if (t >= ntok || r >= m) return;
  const int count = (int)min(m - r, (int64_t)4);
  auto load = [&](int s) {
    const float* p = partial + ((int64_t)s * ntok + t) * m + r;
    if constexpr (VEC) return *(const f32x4_t*)p;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < count) v[e] = p[e];
    return v;
  };
  f32x4_t v = load(0);
#pragma unroll 4
  for (int s = 1; s < splits; ++s) v += load(s);
  if (x_scales) v *= x_scales[t];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < count) {
      if (ydtype == PWQ_F32) ((float*)y)[t * ldy + r + e] = v[e];
      else ((__bf16*)y)[t * ldy + r + e] = (__bf16)v[e];
    }
}

// x to the rows prompt_tiles reads: padded with zeros to whole steps, in
// 8 bits (I8 kept), in bf16, or as three bf16 parts of float32 (64 columns of
// each part in turn; truncated, so the parts are exact and cannot overflow).
template <typename T, bool KEEP8>
__global__ __launch_bounds__(256) void stage_x(const T* __restrict__ x, int64_t ntok, int64_t n,
                                               int64_t ldx, char* __restrict__ out,
                                               int64_t units) {
  const int64_t i = block_index() * 256 + threadIdx.x;         // 8 columns each
  if (i >= ntok * units) return;
  const int64_t t = i / units, u = i % units, k0 = 8 * u;
  T v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = k0 + e < n ? x[t * ldx + k0 + e] : T(0);
  if constexpr (KEEP8) {
    uint2 o;
    __builtin_memcpy(&o, v, 8);
    *(uint2*)(out + i * 8) = o;
  } else if constexpr (std::is_same_v<T, uint16_t>) {
    uint4 o;
    __builtin_memcpy(&o, v, 16);
    *(uint4*)(out + i * 16) = o;
  } else if constexpr (std::is_same_v<T, int8_t>) {
    uint16_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (uint16_t)(__float_as_uint((float)v[e]) >> 16);
    uint4 p;
    __builtin_memcpy(&p, o, 16);
    *(uint4*)(out + i * 16) = p;
  } else {
    char* row = out + (t * units + u / 8 * 8) * 48 + u % 8 * 16;
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      uint16_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(v[e]) & 0xffff0000u;
        o[e] = (uint16_t)(b >> 16);
        v[e] -= __uint_as_float(b);
      }
      uint4 p;
      __builtin_memcpy(&p, o, 16);
      *(uint4*)(row + part * 128) = p;
    }
  }
}

dim3 tile_grid(const PromptArgs& p, int splits) {
  return dim3((unsigned)((p.tiles_t * p.tiles_r + 7) / 8 * 8), (unsigned)splits);
}

template <bool I8, int BT, int BR, int WR>
void launch_tiles(const PromptArgs& p, int mode, int splits, hipStream_t st) {
  const dim3 grid = tile_grid(p, splits);
  if (mode == 0) prompt_tiles<I8, BT, BR, WR, 0><<<grid, 64 * WR, 0, st>>>(p);
  else if (mode == 1) prompt_tiles<I8, BT, BR, WR, 1><<<grid, 64 * WR, 0, st>>>(p);
  else prompt_tiles<I8, BT, BR, WR, 2><<<grid, 64 * WR, 0, st>>>(p);
}

template <bool I8, int NP, int BT, bool ASYM, bool OVER>
void launch_batch_mode(const PromptArgs& p, int mode, int splits, hipStream_t st) {
  const dim3 grid = tile_grid(p, splits);
  if (mode == 0) batch_tiles<I8, NP, BT, 0, ASYM, OVER><<<grid, 256, 0, st>>>(p);
  else if (mode == 1) batch_tiles<I8, NP, BT, 1, ASYM, OVER><<<grid, 256, 0, st>>>(p);
  else batch_tiles<I8, NP, BT, 2, ASYM, OVER><<<grid, 256, 0, st>>>(p);
}

template <bool I8, int NP, int BT>
void launch_batch(const PromptArgs& p, int mode, int splits, hipStream_t st) {
  if (p.n_out > 0)
    return p.zeros ? launch_batch_mode<I8, NP, BT, true, true>(p, mode, splits, st)
                   : launch_batch_mode<I8, NP, BT, false, true>(p, mode, splits, st);
  p.zeros ? launch_batch_mode<I8, NP, BT, true, false>(p, mode, splits, st)
          : launch_batch_mode<I8, NP, BT, false, false>(p, mode, splits, st);
}

}  // namespace

// What prompt_tiles makes of a product: 8-bit or bf16 operands, steps, tile,
// splits and workspace.
PromptPlan prompt_plan(const void* x, int32_t xdtype, int64_t ntok, int64_t ldx, int64_t m,
                       int64_t n, int32_t G, int64_t n_out) {
  PromptPlan p{};
  const bool row = G == n;
  // (128 rows of x within 32-bit offsets, three parts each; what is joined
  // within the extents of a launch)
  p.ok = (row || G % 32 == 0) && ntok > 0 && m > 0 && n < (1 << 21) && ntok < (1 << 26) &&
         m < (1 << 26);
  if (!p.ok) return p;
  // 8-bit operands: a group's sum is an int32, of at most 128 columns unless
  // the whole row is one group (2^17 products of 128 x 127 fit)
  p.i8 = xdtype == PWQ_I8 && (row ? n <= (1 << 17) : G % 64 == 0);
  const int cols = p.i8 ? 128 : 64;
  p.mode = row ? 0 : (G % cols == 0 ? 1 : 2);
  p.reps = xdtype == PWQ_F32 ? 3 : 1;
  p.steps = (n + cols - 1) / cols * p.reps;
  p.staged_row = p.steps * KB;
  // Tile and column splits by their estimated time: steps of a workgroup of 128
  // x 128 that has its CU alone, of two that share it, and of one of 128 x 256
  // (from 256 to 8192 tokens of q_proj, up_proj and down_proj; twice as many
  // columns and sums in 8 bits, twice a step the most).  The splits' float32
  // sums are written and read at about 8.5 TB/s, in the last-level cache, and
  // joined by a launch of its own (3 us).  Where the two tiles differ most: 2048
  // bf16 tokens of 4096 x 14336 take 266 us in wide ones and 298 in narrow
  // ones, 700 8-bit tokens of 14336 x 4096 94 and 86; splits: 512 8-bit tokens
  // of 4096 x 4096 take 28, 26, 28, 27 and 35 us (joined) in 1, 2, 3, 4 and 8.
  const int kind = !p.i8 ? 0 : (p.mode == 2 ? 2 : 1);
  const double us_one[] = {0.70, 0.78, 0.95}, us_two[] = {1.2, 1.37, 1.65};
  const double us_wide[] = {1.05, 1.3, 1.6};
  auto join_us = [&](int64_t splits) {
    return splits > 1 ? 3.0 + 2.0 * splits * ntok * m * 4 / 8.5e6 : 0.0;
  };
  double best = 0;
  // batch_tiles as long as its spreading of the codes for every tile of tokens
  // costs less than spread_weights and its traffic: 256 8-bit tokens of
  // 14336 x 4096 38 us against 52, 512 65 both (q_proj 26 against 33); 256 bf16
  // tokens 56 against 79, 384 83 against 100 (down_proj 88 against 93), 512 103
  // against 96; with overflow entries 128 bf16 tokens 69 both, 256 119 against
  // 81; float32 128 tokens 91 against 90, 129 122 against 109.
  p.fused = ntok <= (n_out > 0 || p.reps == 3 ? 128 : (p.i8 ? 512 : 320));
  if (p.fused) {
    // 32 x 128 or 64 x 128 tiles and column splits by their estimated time, as
    // above: microseconds of a tile's 128 columns for one workgroup on a CU and
    // for two, the first ones' arrival as one and a half of them.  (64 bf16
    // tokens of 14336 x 4096: 26 us in 4 splits, 29 in 2; 8-bit ones 22 and 20;
    // 128 8-bit tokens of 4096 x 4096 17 us in 4 splits, 20 in 8; splits of
    // fewer than 512 columns gained nothing.)
    p.token_tile = ntok <= 32 || p.reps == 3 ? 32 : 64;
    const int of = p.reps == 3 ? 2 : (p.i8 ? 0 : 1);
    const double one[2][3] = {{0.58, 1.05, 1.5}, {0.85, 1.45}};
    const double two[2][3] = {{1.2, 1.6, 3.0}, {1.75, 2.2}};
    p.tiles_t = (ntok + p.token_tile - 1) / p.token_tile;
    p.tiles_r = (m + 127) / 128;
    const int64_t across = (n + 127) / 128, most = std::max<int64_t>(1, across / 4);
    for (int64_t k = 1; k <= most; ++k) {
      const int64_t per = (across + k - 1) / k, splits = (across + per - 1) / per;
      if (splits != k) continue;
      const int64_t groups = p.tiles_t * p.tiles_r * splits, left = groups % 512;
      const int b = p.token_tile == 64;
      double us = (double)(groups / 512) * two[b][of] +
                  (left == 0 ? 0.0 : (left <= 256 ? one[b][of] : two[b][of]));
      us = us * (per + 1.5) + join_us(splits);
      if (best == 0 || us < best) {
        best = us;
        p.per = per;
        p.splits = splits;
      }
    }
  }
  for (int wide = 0; wide < 2 && !p.fused; ++wide) {
    const int64_t tt = (ntok + 127) / 128, edge = wide ? 256 : 128, tr = (m + edge - 1) / edge;
    const int64_t most = std::min<int64_t>(16, std::max<int64_t>(1, p.steps / 4));
    for (int64_t k = 1; k <= most; ++k) {
      const int64_t per = (p.steps + k - 1) / k, splits = (p.steps + per - 1) / per;
      if (splits != k) continue;
      const int64_t groups = tt * tr * splits, left = groups % 512;
      double us = wide ? (double)((groups + 255) / 256) * us_wide[kind]
                       : (double)(groups / 512) * us_two[kind] +
                             (left == 0 ? 0.0 : (left <= 256 ? us_one[kind] : us_two[kind]));
      us *= per;
      us += join_us(splits);
      if (best == 0 || us < best) {
        best = us;
        p.wide = wide;
        p.tiles_t = tt;
        p.tiles_r = tr;
        p.per = per;
        p.splits = splits;
      }
    }
  }
  // tiles of 512 threads within the x extent of a launch
  if (p.tiles_t * p.tiles_r >= (1 << 22)) return PromptPlan{};
  // with the spreading: a launch and its bytes at 5 TB/s
  p.us = best + (p.fused ? 0.0 : 3.0 + (double)m * n * (p.i8 ? 1.5 : 2.5) / 5e6);
  p.rows16 = (m + 15) / 16 * 16;
  p.spread_bytes = p.fused ? 0 : (size_t)(p.rows16 * (p.steps / p.reps) * KB);
  p.steps_bytes = p.fused ? 0 : (size_t)(p.rows16 * (n / G) * 4);
  p.partial_bytes = p.splits > 1 ? (size_t)p.splits * ntok * m * 4 : 0;
  // read in place: whole steps, aligned rows, and 256 of them within 32 bits
  const int64_t es = xdtype == PWQ_I8 ? 1 : (xdtype == PWQ_BF16 ? 2 : 4), xrow = ldx * es;
  p.direct = p.reps == 1 && (xdtype == PWQ_I8) == p.i8 && p.staged_row == n * es &&
             xrow % 16 == 0 && (uintptr_t)x % 16 == 0 && xrow < (int64_t(1) << 23);
  p.staged_bytes = p.direct ? 0 : (size_t)ntok * p.staged_row;
  return p;
}

// staged / partial: workspace of the plan's sizes.
hipError_t launch_prompt(const PackedLinearLaunch& a, const PromptPlan& pl, const PromptWs& w,
                         hipStream_t st) {
  PromptArgs p{};
  const int64_t es = a.xdtype == PWQ_I8 ? 1 : (a.xdtype == PWQ_BF16 ? 2 : 4);
  const int64_t xrow = a.ldx * es;
  if (pl.direct) {
    p.x = (const char*)a.x;
    p.xrow = xrow;
  } else {
    const int64_t units = pl.staged_row / pl.reps / (pl.i8 ? 8 : 16);
    const dim3 grid = block_grid((a.ntok * units + 255) / 256);
    char* o = (char*)w.staged;
    if (a.xdtype == PWQ_I8 && pl.i8)
      stage_x<int8_t, true><<<grid, 256, 0, st>>>((const int8_t*)a.x, a.ntok, a.n, a.ldx, o, units);
    else if (a.xdtype == PWQ_I8)
      stage_x<int8_t, false><<<grid, 256, 0, st>>>((const int8_t*)a.x, a.ntok, a.n, a.ldx, o,
                                                   units);
    else if (a.xdtype == PWQ_BF16)
      stage_x<uint16_t, false><<<grid, 256, 0, st>>>((const uint16_t*)a.x, a.ntok, a.n, a.ldx, o,
                                                     units);
    else
      stage_x<float, false><<<grid, 256, 0, st>>>((const float*)a.x, a.ntok, a.n, a.ldx, o, units);
    p.x = o;
    p.xrow = pl.staged_row;
  }
  p.steps = (int)pl.steps;
  p.reps = pl.reps;
  p.per = (int)pl.per;
  p.tiles_t = (int)pl.tiles_t;
  p.tiles_r = (int)pl.tiles_r;
  p.x_scales = a.x_scales;
  p.qweight = a.qweight;
  p.ldq = a.ldq;
  p.scales = a.scales;
  p.zeros = a.zeros;
  p.off = a.outlier_off;
  p.outliers = a.outliers;
  p.n_out = a.outlier_off ? (int)a.n_out : 0;
  p.spread = (const i32x4_t*)w.spread;
  p.blocks = (int)(pl.steps / pl.reps);
  p.steps_t = w.steps;
  p.rows16 = pl.rows16;
  p.ntok = (int)a.ntok;
  p.m = (int)a.m;
  p.n = (int)a.n;
  p.ng = (int)(a.n / a.G);
  if (pl.mode != 0) {
    const uint32_t halves = (uint32_t)a.G / (pl.i8 ? 64 : 32);
    p.per_group = (uint32_t)(((int64_t(1) << 31) + halves - 1) / halves);
  }
  p.y = a.y;
  p.ydtype = a.ydtype;
  p.ldy = a.ldy;
  p.partial = pl.splits > 1 ? (float*)w.partial : nullptr;
  if (!pl.fused) {
    const int across = (int)((a.n + 127) / 128);
    const int64_t tiles = pl.rows16 / 16 * across;
    const dim3 grid = block_grid((tiles + 3) / 4);
    if (pl.i8)
      spread_weights<true><<<grid, 256, 0, st>>>(
          a.qweight, a.ldq, a.scales, a.zeros, a.outlier_off, a.outliers, p.n_out, a.m, (int)a.n,
          a.G, p.ng, across, tiles, (i32x4_t*)w.spread, p.blocks, w.steps, pl.rows16);
    else
      spread_weights<false><<<grid, 256, 0, st>>>(
          a.qweight, a.ldq, a.scales, a.zeros, a.outlier_off, a.outliers, p.n_out, a.m, (int)a.n,
          a.G, p.ng, across, tiles, (i32x4_t*)w.spread, p.blocks, w.steps, pl.rows16);
  }
  const int mode = pl.mode, k = (int)pl.splits;
  if (pl.fused) {
    const bool few = pl.token_tile == 32;
    if (pl.i8) (few ? launch_batch<true, 1, 32> : launch_batch<true, 1, 64>)(p, mode, k, st);
    else if (pl.reps == 3) launch_batch<false, 6, 32>(p, mode, k, st);
    else (few ? launch_batch<false, 2, 32> : launch_batch<false, 2, 64>)(p, mode, k, st);
  } else if (pl.wide) {
    if (pl.i8) launch_tiles<true, 128, 256, 8>(p, mode, k, st);
    else launch_tiles<false, 128, 256, 8>(p, mode, k, st);
  } else {
    if (pl.i8) launch_tiles<true, 128, 128, 4>(p, mode, k, st);
    else launch_tiles<false, 128, 128, 4>(p, mode, k, st);
  }
  if (p.partial) {
    dim3 grid = block_grid(a.ntok);
    grid.z = (unsigned)((a.m + 1023) / 1024);
    (a.m % 4 == 0 ? prompt_join<true> : prompt_join<false>)<<<grid, 256, 0, st>>>(
        p.partial, (int)pl.splits, a.ntok, a.m, a.x_scales, a.y, a.ydtype, a.ldy);
  }
  return hipGetLastError();
}

}  // namespace pwq
