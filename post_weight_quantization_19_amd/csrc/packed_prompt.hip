// y = x W^^T of a packed layer for many tokens: tiles of BT tokens x BR rows
// on the matrix cores.
//
//   y[t, r] = x_scale[t] * sum_g s[r, g] * sum_{k in g} x[t, k] (c - z)[r, k]
//
// The inner sum runs over integers c - z: v_mfma_i32_16x16x64_i8 for 8-bit x
// (exact int32 sums), v_mfma_f32_16x16x32_bf16 otherwise (c - z is exact in
// bf16, products are exact in float32).  A float32 x is the sum of three bf16
// parts (the top, middle and last 8 bits of its significand), each of which
// runs over the same weights.
//
// A step covers 128 bytes of every x row (128 8-bit or 64 bf16 columns).  x
// goes HBM -> LDS by asynchronous copies one step ahead through three slots;
// the packed weights go through registers, where they are spread to the type
// of x, into one of two slots.  LDS rows are 128 bytes; their 16-byte units
// are permuted by the row so that 16 rows' reads of one column block cover
// every bank.
#include "pwq_internal.h"

#include <algorithm>

namespace pwq {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;
typedef __attribute__((address_space(3))) char lds_char;

constexpr int KB = 128;            // bytes of an x row per step

// Asynchronous copy of 16 bytes per lane, sbase + voff of each lane to
// lds + 16 lane (lds and sbase wave-uniform).  M0 is restored.
__device__ __forceinline__ void copy16(uint32_t voff, const void* sbase, uint32_t lds) {
  uint32_t keep;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(keep)
      : "v"(voff), "s"(sbase), "s"(lds)
      : "memory");
}

// Byte of 16-byte unit c of LDS row r.
__device__ __forceinline__ uint32_t unit_at(int r, int c) {
  return (uint32_t)(r * KB + ((c ^ ((r >> 1) & 7)) << 4));
}

// Eight 4-bit steps of a dword to bytes: w has the codes 0 .. 15, z4 the zero
// point in every byte (z <= 127: no borrow passes a byte, as every byte is at
// least 128 before the subtraction).
__device__ __forceinline__ uint2 steps_i8(uint32_t w, uint32_t z4) {
  const uint32_t even = (((w & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
  const uint32_t odd = ((((w >> 4) & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
  return make_uint2(__builtin_amdgcn_perm(odd, even, 0x05010400u),
                    __builtin_amdgcn_perm(odd, even, 0x07030602u));
}

// Eight signed 4-bit codes to bytes of 16 times their value.
__device__ __forceinline__ uint2 signed16_i8(uint32_t w) {
  const uint32_t even = (w << 4) & 0xf0f0f0f0u, odd = w & 0xf0f0f0f0u;
  return make_uint2(__builtin_amdgcn_perm(odd, even, 0x05010400u),
                    __builtin_amdgcn_perm(odd, even, 0x07030602u));
}

// ... to bf16: a code's four bits are put at the top of the mantissa of 16,
// and 16 + z is subtracted in float32, whose upper half holds the difference
// exactly (no conversion instruction: those run at a quarter of the rate).
// zb = 16 + z, or 24 with `bias` 0x41c0 for signed halves (it flips their top
// bit; 0x4180 otherwise).
__device__ __forceinline__ uint4 steps_bf16(uint32_t w, uint32_t bias, float zb) {
  constexpr uint32_t M = 0x00780078u;
  const uint32_t c[4] = {((w << 3) & M) ^ bias, ((w >> 1) & M) ^ bias, ((w >> 5) & M) ^ bias,
                         ((w >> 9) & M) ^ bias};            // columns i and i + 4
  float lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = __uint_as_float(c[i] << 16) - zb;
    hi[i] = __uint_as_float(c[i] & 0xffff0000u) - zb;
  }
  auto two = [](float x, float y) {
    return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
  };
  return make_uint4(two(lo[0], lo[1]), two(lo[2], lo[3]), two(hi[0], hi[1]), two(hi[2], hi[3]));
}

// 1.5 2^23 as an integer: int32 sums below 2^22 that start here read as
// 1.5 2^23 + sum when taken for a float32.
constexpr int kMagic = 0x4b400000;

struct PromptArgs {
  const char* x;          // rows of `steps` * 128 bytes, 16-byte aligned
  int64_t xrow;           // bytes between x rows
  int steps;              // steps over the whole row
  int reps;               // steps per weight block (3 for float32 parts)
  int per;                // steps per split
  int tiles_t, tiles_r;
  const float* x_scales;
  const uint8_t* qweight;
  int64_t ldq;
  const float* scales;
  const uint8_t* zeros;
  const int32_t* off;
  const int32_t* outliers;
  int n_out;
  int ntok, m, n, G, ng;
  void* y;
  int ydtype;
  int64_t ldy;
  float* partial;         // splits x ntok x m, or NULL
};

// MODE: how often sums are multiplied by their step.  0: one step per row,
// at the end; 1: every step (G a multiple of its columns); 2: twice a step.
// PLAIN: signed codes without overflow entries (8-bit operands are then 16
// times the code, which takes fewer instructions to spread).
template <bool I8, int BT, int BR, int WT, int WR, int MODE, bool PLAIN>
__global__ __launch_bounds__(64 * WT * WR) void prompt_tiles(const PromptArgs a) {
  constexpr int NT = 64 * WT * WR;
  constexpr int NI = BT / WT / 16, NJ = BR / WR / 16;
  constexpr int COLS = I8 ? 128 : 64;         // columns of a step
  constexpr int WB = COLS / 2;                // packed bytes of a row per step
  constexpr int PER = BR * WB / NT;           // packed bytes of a thread per step
  constexpr int XB = BT * KB, WBUF = BR * KB;
  constexpr int NC = XB / (16 * NT);          // copies of a wave per step
  static_assert(PER == (I8 ? 32 : 16) && NC * 16 * NT == XB, "tile and threads fit");
  using acc_t = std::conditional_t<I8, i32x4_t, f32x4_t>;
  __shared__ __attribute__((aligned(16))) char smem[3 * XB + 2 * WBUF];
  lds_char* L = (lds_char*)smem;
  const uint32_t lbase = (uint32_t)(uintptr_t)L;

  // tile of this workgroup: XCD b % 8 owns a contiguous range of tiles,
  // tokens fastest, so that its L2 holds the weights of a few row tiles
  const int tiles = a.tiles_t * a.tiles_r;
  const int split = blockIdx.y;
  int tile;
  {
    const int b = blockIdx.x, x = b & 7, q = tiles / 8, r = tiles % 8;
    tile = x * q + min(x, r) + (b >> 3);
    if ((b >> 3) >= q + (x < r ? 1 : 0)) return;
  }
  const int t0 = tile % a.tiles_t * BT, r0 = tile / a.tiles_t * BR;
  const int s0 = split * a.per, s1 = min(a.steps, s0 + a.per);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WR, wr = wave % WR;

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

  // weights: thread -> row and part of the row's bytes
  constexpr int TPR = WB / PER;               // threads per row
  const int wrow = tid / TPR, wpart = tid % TPR;
  const int grow = min(r0 + wrow, a.m - 1);
  const uint8_t* const wbase = a.qweight + r0 * a.ldq;
  const uint32_t wsrc = (uint32_t)((grow - r0) * a.ldq + wpart * PER);
  const int wleft = (int)a.ldq - wpart * PER;   // bytes from wsrc to the row's end
  const uint32_t flip = a.zeros ? 0u : 0x88888888u;
  // (SYM reads the steps' bytes in the zero points' place and uses 8)
  const uint8_t* zsrc = a.zeros ? a.zeros + (int64_t)grow * a.ng
                                : (const uint8_t*)(a.scales + (int64_t)grow * a.ng);
  uint4 wreg[PER / 16];
  int zreg = 8;
  auto load_w = [&](int s) {
    const int o = s / a.reps * WB;
#pragma unroll
    for (int i = 0; i < PER / 16; ++i)
      wreg[i] = *(const uint4*)(wbase + (wsrc + (uint32_t)(o + 16 * i < wleft ? o + 16 * i : 0)));
    if constexpr (!PLAIN)
      zreg = zsrc[MODE == 0 ? 0 : min((o + wpart * PER) * 2, a.n - 1) / a.G];
  };
  // overflow entries of the thread's strip of 16 rows
  const int across = (a.n + kPackCols - 1) / kPackCols;
  const int strip = min(r0 / kPackRows + wrow / kPackRows,
                        (a.m + kPackRows - 1) / kPackRows - 1);
  auto put_w = [&](int s, int slot) {
    const uint32_t dst = (uint32_t)(3 * XB + slot * WBUF);
    const int z = PLAIN || !a.zeros ? 8 : zreg;
    if constexpr (I8 && PLAIN) {
#pragma unroll
      for (int i = 0; i < PER / 16; ++i) {
        const uint2 p0 = signed16_i8(wreg[i].x), p1 = signed16_i8(wreg[i].y);
        const uint2 p2 = signed16_i8(wreg[i].z), p3 = signed16_i8(wreg[i].w);
        const int c = (wpart * PER + 16 * i) / 8;
        *(uint4*)(smem + dst + unit_at(wrow, c)) = make_uint4(p0.x, p0.y, p1.x, p1.y);
        *(uint4*)(smem + dst + unit_at(wrow, c + 1)) = make_uint4(p2.x, p2.y, p3.x, p3.y);
      }
    } else if constexpr (I8) {
      const uint32_t z4 = (uint32_t)z * 0x01010101u;
#pragma unroll
      for (int i = 0; i < PER / 16; ++i) {
        const uint2 p0 = steps_i8(wreg[i].x ^ flip, z4), p1 = steps_i8(wreg[i].y ^ flip, z4);
        const uint2 p2 = steps_i8(wreg[i].z ^ flip, z4), p3 = steps_i8(wreg[i].w ^ flip, z4);
        const int c = (wpart * PER + 16 * i) / 8;
        *(uint4*)(smem + dst + unit_at(wrow, c)) = make_uint4(p0.x, p0.y, p1.x, p1.y);
        *(uint4*)(smem + dst + unit_at(wrow, c + 1)) = make_uint4(p2.x, p2.y, p3.x, p3.y);
      }
    } else {
      const float zb = 16.0f + (float)z;
      const uint32_t bias = !PLAIN && a.zeros ? 0x41804180u : 0x41c041c0u;
      const int c = wpart * PER / 4;
      *(uint4*)(smem + dst + unit_at(wrow, c)) = steps_bf16(wreg[0].x, bias, zb);
      *(uint4*)(smem + dst + unit_at(wrow, c + 1)) = steps_bf16(wreg[0].y, bias, zb);
      *(uint4*)(smem + dst + unit_at(wrow, c + 2)) = steps_bf16(wreg[0].z, bias, zb);
      *(uint4*)(smem + dst + unit_at(wrow, c + 3)) = steps_bf16(wreg[0].w, bias, zb);
    }
    if constexpr (!PLAIN) if (a.n_out > 0) {
      // codes beyond 4 bits: the thread adds the entries of its own part of
      // its own row (its writes above are in order with these)
      const int k0 = s / a.reps * COLS;
      const int tl = strip * across + min(k0 / kPackCols, across - 1);
      const int e0 = max(a.off[tl], 0), e1 = min(a.off[tl + 1], a.n_out);
      const int first = k0 % kPackCols + 2 * wpart * PER;
      for (int e = e0; e < e1; ++e) {
        const int v = a.outliers[e], k = (v & 127) - first;
        if (((v >> 7) & 15) == (wrow & 15) && k >= 0 && k < 2 * PER) {
          const int at = 2 * wpart * PER + k;
          if constexpr (I8) {
            char* p = smem + dst + unit_at(wrow, at >> 4) + (at & 15);
            *(int8_t*)p = (int8_t)(*(int8_t*)p + (v >> 16));
          } else {
            char* p = smem + dst + unit_at(wrow, at >> 3) + 2 * (at & 7);
            const float f = bf16_to_f32(*(uint16_t*)p) + (float)(v >> 16);
            *(uint16_t*)p = (uint16_t)(__float_as_uint(f) >> 16);
          }
        }
      }
    }
  };

  // Steps (scales): lane l loads that of row l of the wave's 64, and lane
  // l % 16 + 16 j hands it on for block j (a load in the operands' layout
  // would look up each row four times).
  static_assert(NJ == 4, "a lane per row of the wave");
  const float* const sbase = a.scales + (int64_t)r0 * a.ng;
  const uint32_t sp = (uint32_t)((min(r0 + 64 * wr + lane, a.m - 1) - r0) * a.ng);
  constexpr int NS = MODE == 2 ? 2 : 1;
  float sc[NJ][NS], sn[NS];
  auto load_s = [&](int s) {
    const int k0 = s / a.reps * COLS;
#pragma unroll
    for (int h = 0; h < NS; ++h) {
      const int g = MODE == 0 ? 0 : min((k0 + h * (COLS / 2)) / a.G, a.ng - 1);
      sn[h] = sbase[sp + g] * (I8 && PLAIN ? 0.0625f : 1.0f);
    }
  };
  auto spread_s = [&]() {
#pragma unroll
    for (int h = 0; h < NS; ++h)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        sc[j][h] = __int_as_float(__builtin_amdgcn_ds_bpermute(4 * (16 * j + (lane & 15)),
                                                               __float_as_int(sn[h])));
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

  auto mma = [&](const i32x4_t& x, const i32x4_t& w, const acc_t& c) -> acc_t {
    if constexpr (I8) return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, w, c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x),
                                                     __builtin_bit_cast(bf16x8_t, w), c, 0, 0, 0);
  };
  const int lr = lane & 15, lq = lane >> 4;
  // what a block's sum starts from, and its value
  acc_t zero = {0, 0, 0, 0};
  if constexpr (I8) zero = acc_t{kMagic, kMagic, kMagic, kMagic};
  auto value = [](const acc_t& c, int e) {
    if constexpr (I8) return __int_as_float(c[e]) - 12582912.0f;
    else return c[e];
  };

  // prologue: step s0 in LDS, step s0 + 1 on its way
  const int last = s1 - 1;
  load_w(s0);
  copy_x(s0, s0 % 3);
  put_w(s0, s0 & 1);
  load_s(s0);
  load_w(min(s0 + 1, last));
  copy_x(min(s0 + 1, last), (s0 + 1) % 3);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();

  // The two waves of a SIMD spread the next step's weights at different
  // times, one at the start of a step and one at its end, so that the matrix
  // unit has work from the other.  (Past the last step they spread and
  // load it again, without branches.)
  const bool early = wave < WT * WR / 2;
  auto next = [&](int s) {
    // the last step's loads: weights of step s + 1 in registers, its x in LDS
    // (every wave's, once the barrier at the end of this step is passed)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    put_w(min(s + 1, last), (s + 1) & 1);
    if constexpr (MODE != 0) load_s(min(s + 1, last));
    load_w(min(s + 2, last));
    copy_x(min(s + 2, last), (s + 2) % 3);
  };
  for (int s = s0; s < s1; ++s) {
    if constexpr (MODE != 0) spread_s();
    if (early) next(s);
    const char* xs = smem + s % 3 * XB;
    const char* ws = smem + 3 * XB + (s & 1) * WBUF;
    i32x4_t w[NJ][2], x[2][2];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[j][h] = *(const i32x4_t*)(ws + unit_at(16 * (wr * NJ + j) + lr, 4 * h + lq));
    auto read_x = [&](int i) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[i & 1][h] = *(const i32x4_t*)(xs + unit_at(16 * (wt * NI + i) + lr, 4 * h + lq));
    };
    read_x(0);
    if constexpr (MODE == 0) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (i + 1 < NI) read_x(i + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NJ; ++j) dir[i][j] = mma(x[i & 1][h], w[j][h], dir[i][j]);
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
          acc[i][j][e] = fmaf(sc[j][h], value(c[u & 3], e), acc[i][j][e]);
          pin(acc[i][j][e]);       // here: not moved behind the other products
        }
      };
      static_for_up<NU + 3>([&](auto uu) {
        constexpr int u = decltype(uu)::value;
        constexpr int i = u / NS / NJ, j = u / NS % NJ, h = u % NS;
        if constexpr (u < NU) {
          c[u & 3] = mma(x[i & 1][h], w[j][h], zero);
          if constexpr (j == 1 && h == 0 && i + 1 < NI) read_x(i + 1);
        }
        if constexpr (u >= 3) scale(std::integral_constant<int, u - 3>{}, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE == 1 && u > 0 && u <= NU) {
          constexpr int v = u - 1, iv = v / NJ, jv = v % NJ;
          c[v & 3] = mma(x[iv & 1][1], w[jv][1], c[v & 3]);
        }
        if constexpr (u >= 3) scale(std::integral_constant<int, u - 3>{}, 2);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    if (!early) next(s);
    lds_barrier();
  }
  // nothing is in flight to LDS, and no wave reads it, at the end
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();
  if constexpr (MODE == 0) {
    spread_s();
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = sc[j][0] * (float)dir[i][j][e];
  }

  // lane l holds tokens 4 (l / 16) + e, row l % 16 of every block
  const bool split_sum = a.partial != nullptr;
  if (a.x_scales && !split_sum) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float xsc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        xsc[e] = a.x_scales[min(t0 + 16 * (wt * NI + i) + 4 * lq + e, a.ntok - 1)];
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
        const int t = t0 + 16 * (wt * NI + i) + 4 * lq + e;
        if (t < a.ntok)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int r = r0 + 16 * (wr * NJ + j) + lr;
            if (r < a.m) y[t * ld + r] = acc[i][j][e];
          }
      }
    return;
  }
  // bf16: through LDS, so that rows of y are written 16 bytes a lane.  Two
  // neighbouring lanes trade halves: the even one packs both their rows of
  // token e, the odd one of token e + 1.
  constexpr int YROW = 2 * BR + 32;                    // bytes of a token's row in LDS
  static_assert(BT * YROW <= 3 * XB + 2 * WBUF, "the tile fits");
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
        const int t = 16 * (wt * NI + i) + 4 * lq + e + odd;
        const int r = 16 * (wr * NJ + j) + (lr & ~1);
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

// Sum of the splits in their order.
__global__ __launch_bounds__(256) void prompt_join(const float* __restrict__ partial, int splits,
                                                   int64_t ntok, int64_t m,
                                                   const float* __restrict__ x_scales, void* y,
                                                   int ydtype, int64_t ldy) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= ntok * m) return;
  const int64_t t = i / m, r = i % m;
  float v = partial[i];
  for (int s = 1; s < splits; ++s) v += partial[(int64_t)s * ntok * m + i];
  if (x_scales) v *= x_scales[t];
  if (ydtype == PWQ_F32) ((float*)y)[t * ldy + r] = v;
  else ((__bf16*)y)[t * ldy + r] = (__bf16)v;
}

// x to the rows prompt_tiles reads: padded with zeros to whole steps, in
// 8 bits (I8 kept), in bf16, or as three bf16 parts of float32 (64 columns of
// each part in turn; truncated, so the parts are exact and cannot overflow).
template <typename T, bool KEEP8>
__global__ __launch_bounds__(256) void stage_x(const T* __restrict__ x, int64_t ntok, int64_t n,
                                               int64_t ldx, char* __restrict__ out,
                                               int64_t units) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // 8 columns each
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

template <bool I8, int BT, int BR, int WT, int WR, bool PLAIN>
void launch_mode(const PromptArgs& p, int mode, int splits, hipStream_t st) {
  const dim3 grid((unsigned)((p.tiles_t * p.tiles_r + 7) / 8 * 8), (unsigned)splits);
  const int nt = 64 * WT * WR;
  if (mode == 0) prompt_tiles<I8, BT, BR, WT, WR, 0, PLAIN><<<grid, nt, 0, st>>>(p);
  else if (mode == 1) prompt_tiles<I8, BT, BR, WT, WR, 1, PLAIN><<<grid, nt, 0, st>>>(p);
  else prompt_tiles<I8, BT, BR, WT, WR, 2, PLAIN><<<grid, nt, 0, st>>>(p);
}

template <bool I8, int BT, int BR, int WT, int WR>
void launch_tiles(const PromptArgs& p, int mode, int splits, hipStream_t st) {
  if (!p.zeros && p.n_out == 0) launch_mode<I8, BT, BR, WT, WR, true>(p, mode, splits, st);
  else launch_mode<I8, BT, BR, WT, WR, false>(p, mode, splits, st);
}

}  // namespace

// What prompt_tiles makes of a product: 8-bit or bf16 operands, steps, tile,
// splits and workspace.
PromptPlan prompt_plan(const void* x, int32_t xdtype, int64_t ntok, int64_t ldx, int64_t m,
                       int64_t n, int32_t G) {
  PromptPlan p{};
  const bool row = G == n;
  p.ok = (row || G % 32 == 0) && ntok > 0 && m > 0;
  if (!p.ok) return p;
  p.i8 = xdtype == PWQ_I8 && (row || G % 64 == 0);
  const int cols = p.i8 ? 128 : 64;
  p.mode = row ? 0 : (G % cols == 0 ? 1 : 2);
  p.reps = xdtype == PWQ_F32 ? 3 : 1;
  p.steps = (n + cols - 1) / cols * p.reps;
  p.staged_row = p.steps * KB;
  p.big = ntok > 128 && m > 128 && ((ntok + 255) / 256) * ((m + 255) / 256) >= 192;
  const int64_t edge = p.big ? 256 : 128;
  p.tiles_t = (ntok + edge - 1) / edge;
  p.tiles_r = (m + edge - 1) / edge;
  // too few tiles for 256 CUs (512 workgroups of the small tile): split the
  // columns, at least 4 steps a split
  const int64_t tiles = p.tiles_t * p.tiles_r;
  p.splits = 1;
  if (!p.big && tiles < 256)
    p.splits = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, p.steps / 8));
  p.per = (p.steps + p.splits - 1) / p.splits;
  p.splits = (p.steps + p.per - 1) / p.per;
  p.partial_bytes = p.splits > 1 ? (size_t)p.splits * ntok * m * 4 : 0;
  // read in place: whole steps, aligned rows, and 256 of them within 32 bits
  const int64_t es = xdtype == PWQ_I8 ? 1 : (xdtype == PWQ_BF16 ? 2 : 4), xrow = ldx * es;
  p.direct = p.reps == 1 && (xdtype == PWQ_I8) == p.i8 && p.staged_row == n * es &&
             xrow % 16 == 0 && (uintptr_t)x % 16 == 0 && xrow < (int64_t(1) << 23);
  p.staged_bytes = p.direct ? 0 : (size_t)ntok * p.staged_row;
  return p;
}

// staged / partial: workspace of the plan's sizes.
hipError_t launch_prompt(const PackedLinearLaunch& a, const PromptPlan& pl, void* staged,
                         void* partial, hipStream_t st) {
  PromptArgs p{};
  const int64_t es = a.xdtype == PWQ_I8 ? 1 : (a.xdtype == PWQ_BF16 ? 2 : 4);
  const int64_t xrow = a.ldx * es;
  if (pl.direct) {
    p.x = (const char*)a.x;
    p.xrow = xrow;
  } else {
    const int64_t units = pl.staged_row / pl.reps / (pl.i8 ? 8 : 16);
    const dim3 grid((unsigned)((a.ntok * units + 255) / 256));
    char* o = (char*)staged;
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
  p.ntok = (int)a.ntok;
  p.m = (int)a.m;
  p.n = (int)a.n;
  p.G = a.G;
  p.ng = (int)(a.n / a.G);
  p.y = a.y;
  p.ydtype = a.ydtype;
  p.ldy = a.ldy;
  p.partial = pl.splits > 1 ? (float*)partial : nullptr;
  if (pl.big) {
    if (pl.i8) launch_tiles<true, 256, 256, 2, 4>(p, pl.mode, (int)pl.splits, st);
    else launch_tiles<false, 256, 256, 2, 4>(p, pl.mode, (int)pl.splits, st);
  } else {
    if (pl.i8) launch_tiles<true, 128, 128, 2, 2>(p, pl.mode, (int)pl.splits, st);
    else launch_tiles<false, 128, 128, 2, 2>(p, pl.mode, (int)pl.splits, st);
  }
  if (p.partial)
    prompt_join<<<dim3((unsigned)((a.ntok * a.m + 255) / 256)), 256, 0, st>>>(
        p.partial, (int)pl.splits, a.ntok, a.m, a.x_scales, a.y, a.ydtype, a.ldy);
  return hipGetLastError();
}

}  // namespace pwq
