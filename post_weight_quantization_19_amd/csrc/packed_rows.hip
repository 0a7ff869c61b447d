// y = x W^^T of a packed layer for few tokens (up to 64): every weight is
// read once, spread in registers, and multiplied on the matrix cores.
//
// A workgroup owns a strip of 16 rows; its waves split the columns in tiles of
// 128 and their partial sums are joined in LDS in wave order.  In a tile the
// operands are x (16 tokens) and the integer steps c - z of 16 rows: lane l
// holds token l % 16 and row l % 16, and the GB / 4 columns GB h +
// (GB / 4)(l / 16) .. of block h, GB <= G, so that the four lane groups of a
// matrix instruction stay within one group of the steps.  The sum of a block
// (int32 for 8-bit x, float32 for exact products of bf16 otherwise) is
// multiplied by the step of the lane's row and added in float32.
//
// Codes beyond 4 bits enter as further columns: up to 32 (64 for 8-bit x)
// entries of a tile at a time, x gathered at their columns, the entry's value
// in its own row and 0 in the others.
#include "pwq_internal.h"

#include <algorithm>

namespace pwq {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;
struct __attribute__((packed, aligned(1))) vec16 { uint4 v; };
struct __attribute__((packed, aligned(1))) vec8 { uint2 v; };

enum { X_BF16 = 0, X_I8 = 1, X_F32 = 2, X_I8_BF16 = 3 };
template <int XK> struct XType { using T = uint16_t; };
template <> struct XType<X_I8> { using T = int8_t; };
template <> struct XType<X_I8_BF16> { using T = int8_t; };
template <> struct XType<X_F32> { using T = float; };

template <int N, typename T>
struct Cols { T v[N]; };

// N consecutive elements (any alignment); those at or past `left` are 0.
template <int N, typename T>
__device__ __forceinline__ Cols<N, T> load_cols(const T* p, int left) {
  Cols<N, T> c;
  if (left >= N) {
    constexpr int B = N * sizeof(T);
    if constexpr (B % 16 == 0) {
#pragma unroll
      for (int i = 0; i < B / 16; ++i) {
        const uint4 u = ((const vec16*)p)[i].v;
        __builtin_memcpy((char*)&c + 16 * i, &u, 16);
      }
    } else {
      static_assert(B == 8);
      const uint2 u = ((const vec8*)p)->v;
      __builtin_memcpy(&c, &u, 8);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) c.v[e] = e < left ? p[e] : T(0);
  }
  return c;
}

__device__ __forceinline__ uint32_t pack_hi(float a, float b) {   // exact for small integers
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Eight 4-bit steps of a dword (codes 0 .. 15) minus z, to bf16 or bytes.
__device__ __forceinline__ bf16x8_t steps_bf16(uint32_t w, float z) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  uint4 o;
  uint32_t* q = (uint32_t*)&o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = pack_hi((float)((even >> (8 * i)) & 0xffu) - z, (float)((odd >> (8 * i)) & 0xffu) - z);
  return __builtin_bit_cast(bf16x8_t, o);
}
__device__ __forceinline__ uint2 steps_i8(uint32_t w, uint32_t z4) {
  const uint32_t even = (((w & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
  const uint32_t odd = ((((w >> 4) & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
  return make_uint2(__builtin_amdgcn_perm(odd, even, 0x05010400u),
                    __builtin_amdgcn_perm(odd, even, 0x07030602u));
}

// Part `part` (0, 1, 2) of eight float32 in bf16, truncated: exact, and the
// remainders are left in v.
__device__ __forceinline__ bf16x8_t f32_part(float* v) {
  uint4 o;
  uint32_t* q = (uint32_t*)&o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = pack_hi(v[2 * i], v[2 * i + 1]);
    v[2 * i] -= __uint_as_float(__float_as_uint(v[2 * i]) & 0xffff0000u);
    v[2 * i + 1] -= __uint_as_float(__float_as_uint(v[2 * i + 1]) & 0xffff0000u);
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

__device__ __forceinline__ f32x4_t mma(bf16x8_t x, bf16x8_t w, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

// Eight columns of x (from `p`, its own type) against eight bf16 steps.
template <int XK>
__device__ __forceinline__ f32x4_t mma_x(const typename XType<XK>::T* p, bf16x8_t w, f32x4_t c) {
  if constexpr (XK == X_F32) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e];
#pragma unroll
    for (int part = 0; part < 3; ++part) c = mma(f32_part(v), w, c);
    return c;
  } else if constexpr (XK == X_BF16) {
    bf16x8_t x;
    __builtin_memcpy(&x, p, 16);
    return mma(x, w, c);
  } else {
    uint4 o;
    uint32_t* q = (uint32_t*)&o;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack_hi((float)p[2 * i], (float)p[2 * i + 1]);
    return mma(__builtin_bit_cast(bf16x8_t, o), w, c);
  }
}

// NT blocks of 16 tokens from 16 NT blockIdx.y on; GB columns per block; U
// tiles loaded at a time; OVER: with overflow entries.
template <int XK, int NT, int GB, int U, bool OVER>
__global__ __launch_bounds__(1024) void packed_rows(const PackedLinearLaunch a) {
  using T = typename XType<XK>::T;
  using acc_t = std::conditional_t<XK == X_I8, i32x4_t, f32x4_t>;
  constexpr int NB = 128 / GB, NC = GB / 4;     // blocks of a tile, columns of a lane in one
  constexpr int NW = NC / 8;                    // dwords of a lane per block
  extern __shared__ float joined[];             // [wave][NT][4][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t strip = blockIdx.x, t0 = (int64_t)blockIdx.y * 16 * NT;
  const int64_t row = min(strip * kPackRows + lr, a.m - 1);
  const int64_t ng = a.n / a.G;
  const int n = (int)a.n, G = a.G;
  const int across = (n + 127) >> 7, per = (across + waves - 1) / waves;
  const int k0 = wave * per, k1 = min(across, k0 + per);
  const uint8_t* q = a.qweight + row * a.ldq;
  const float* sp = a.scales + row * ng;
  // SYM: the zero point is 8 once the signs are flipped (what is read in its
  // place, the row's steps, is not used)
  const bool asym = a.zeros != nullptr;
  const uint8_t* zp = asym ? a.zeros + row * ng : (const uint8_t*)sp;
  const uint32_t flip = asym ? 0u : 0x88888888u;
  const T* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    xp[i] = (const T*)a.x + min(t0 + 16 * i + lr, a.ntok - 1) * a.ldx;

  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // group of the next block, kept without divisions
  int g = 128 * k0 / G, in_g = 128 * k0 % G;

  // `count` <= UU tiles from kt on.  Every load is issued before the first is
  // used, without branches: tiles past `count` load the last one again.
  auto tiles = [&](auto uu, auto ragged, int kt, int count) {
    constexpr int UU = decltype(uu)::value;
    constexpr bool RAGGED = decltype(ragged)::value;
    uint32_t w[UU][NB][NW];
    float s[UU][NB];
    int z[UU][NB];
    Cols<NC, T> x[UU][NB][NT];
#pragma unroll
    for (int u = 0; u < UU; ++u)
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        const int k = 128 * (kt + min(u, count - 1)) + GB * h + NC * lq;
        const uint8_t* p = q + (!RAGGED || k / 2 < a.ldq ? k / 2 : 0);
        if constexpr (NW == 4) {
          const uint4 v = *(const uint4*)p;
          w[u][h][0] = v.x, w[u][h][1] = v.y, w[u][h][2] = v.z, w[u][h][3] = v.w;
        } else if constexpr (NW == 2) {
          const uint2 v = *(const uint2*)p;
          w[u][h][0] = v.x, w[u][h][1] = v.y;
        } else {
          w[u][h][0] = *(const uint32_t*)p;
        }
        const int gi = min(g, (int)ng - 1);
        s[u][h] = sp[gi];
        z[u][h] = zp[gi];
        in_g += GB;
        const bool next = in_g >= G;
        g += next, in_g -= next ? G : 0;
      }
#pragma unroll
    for (int u = 0; u < UU; ++u)
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        const int k = 128 * (kt + min(u, count - 1)) + GB * h + NC * lq;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          x[u][h][i] = load_cols<NC>(xp[i] + k, RAGGED ? n - k : NC);
      }
    asm volatile("" ::: "memory");             // the loads stay in front of the sums
#pragma unroll
    for (int u = 0; u < UU; ++u) {
      if (u >= count) break;
      int e0 = 0, e1 = 0;
      if constexpr (OVER) {
        const int64_t tile = strip * across + kt + u;
        e0 = max(a.outlier_off[tile], 0);
        e1 = (int)min((int64_t)a.outlier_off[tile + 1], a.n_out);
      }
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        const int zi = asym ? z[u][h] : 8;
        acc_t c[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) c[i] = acc_t{0, 0, 0, 0};
        if constexpr (XK == X_I8) {
          const uint32_t z4 = (uint32_t)zi * 0x01010101u;
#pragma unroll
          for (int j = 0; j < NW; j += 2) {
            const uint2 lo = steps_i8(w[u][h][j] ^ flip, z4);
            const uint2 hi = steps_i8(w[u][h][j + 1] ^ flip, z4);
            const i32x4_t b = {(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              i32x4_t v;
              __builtin_memcpy(&v, x[u][h][i].v + 8 * j, 16);
              c[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, b, c[i], 0, 0, 0);
            }
          }
        } else {
          const float zf = (float)zi;
#pragma unroll
          for (int j = 0; j < NW; ++j) {
            const bf16x8_t b = steps_bf16(w[u][h][j] ^ flip, zf);
#pragma unroll
            for (int i = 0; i < NT; ++i) c[i] = mma_x<XK>(x[u][h][i].v + 8 * j, b, c[i]);
          }
        }
        constexpr int PE = XK == X_I8 ? 16 : 8;          // entries of a lane at a time
        if constexpr (OVER) for (int e = e0; e < e1; e += 4 * PE) {
          int ent[PE];
#pragma unroll
          for (int i = 0; i < PE; ++i) {
            const int at = e + PE * lq + i;
            ent[i] = at < e1 ? a.outliers[at] : 0;       // 0: value 0 at column 0
            if ((ent[i] & 127) / GB != h) ent[i] = 0;    // another block's
            if (128 * (kt + u) + (ent[i] & 127) >= n) ent[i] = 0;
          }
          Cols<PE, T> xe[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < PE; ++i)
              xe[t].v[i] = ent[i] ? xp[t][128 * (kt + u) + (ent[i] & 127)] : T(0);
          if constexpr (XK == X_I8) {
            i32x4_t b = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < PE; ++i)
              if (((ent[i] >> 7) & 15) == lr) b[i / 4] |= ((ent[i] >> 16) & 255) << (8 * (i % 4));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              i32x4_t v;
              __builtin_memcpy(&v, xe[t].v, 16);
              c[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, b, c[t], 0, 0, 0);
            }
          } else {
            float d[PE];
#pragma unroll
            for (int i = 0; i < PE; ++i)
              d[i] = ((ent[i] >> 7) & 15) == lr ? (float)(ent[i] >> 16) : 0.0f;
            uint4 o = make_uint4(pack_hi(d[0], d[1]), pack_hi(d[2], d[3]), pack_hi(d[4], d[5]),
                                 pack_hi(d[6], d[7]));
#pragma unroll
            for (int t = 0; t < NT; ++t)
              c[t] = mma_x<XK>(xe[t].v, __builtin_bit_cast(bf16x8_t, o), c[t]);
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(s[u][h], (float)c[i][e], acc[i][e]);
      }
    }
  };
  const int kf = max(k0, min(k1, n >> 7));     // the first tile that is not whole
  for (int kt = k0; kt < kf; kt += U)
    tiles(std::integral_constant<int, U>{}, std::false_type{}, kt, min(U, kf - kt));
  if (kf < k1) {
    g = 128 * kf / G, in_g = 128 * kf % G;
    tiles(std::integral_constant<int, 1>{}, std::true_type{}, kf, 1);
  }

  // join the waves' sums in their order; lane l: tokens 4 (l / 16) + e, row l % 16
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) joined[((wave * NT + i) * 4 + e) * 64 + lane] = acc[i][e];
  __syncthreads();
  for (int v = threadIdx.x; v < NT * 256; v += blockDim.x) {
    const int i = v >> 8, e = (v >> 6) & 3, l = v & 63;
    const int64_t t = t0 + 16 * i + 4 * (l >> 4) + e, r = strip * kPackRows + (l & 15);
    if (t >= a.ntok || r >= a.m) continue;
    float sum = joined[v];
    for (int o = 1; o < waves; ++o) sum += joined[o * NT * 256 + v];
    if (a.x_scales) sum *= a.x_scales[t];
    if (a.ydtype == PWQ_F32) ((float*)a.y)[t * a.ldy + r] = sum;
    else ((__bf16*)a.y)[t * a.ldy + r] = (__bf16)sum;
  }
}

template <int XK, int NT, int GB, int U>
void launch_u(const PackedLinearLaunch& a, int waves, hipStream_t st) {
  const dim3 grid((unsigned)((a.m + kPackRows - 1) / kPackRows),
                  (unsigned)((a.ntok + 16 * NT - 1) / (16 * NT)));
  if constexpr (NT <= 2 && U == 1) if (a.outlier_off) {
    packed_rows<XK, NT, GB, 1, true><<<grid, 64 * waves, waves * NT * 1024, st>>>(a);
    return;
  }
  packed_rows<XK, NT, GB, U, false><<<grid, 64 * waves, waves * NT * 1024, st>>>(a);
}

template <int XK, int NT, int GB>
void launch_nt(const PackedLinearLaunch& a, hipStream_t st) {
  // tiles in flight that the registers hold
  constexpr int MOST = XK == X_F32 || GB == 32 ? 1 : std::max(1, 4 / NT);
  const int64_t strips = (a.m + kPackRows - 1) / kPackRows, across = (a.n + 127) / 128;
  // about 16 waves per CU over the whole launch
  int waves = 1;
  while (waves < 16 && strips * waves < 4096 && waves < across) waves *= 2;
  const int64_t per = (across + waves - 1) / waves;
  if constexpr (MOST >= 4) if (per > 2 && !a.outlier_off) return launch_u<XK, NT, GB, 4>(a, waves, st);
  if constexpr (MOST >= 2) if (per > 1 && !a.outlier_off) return launch_u<XK, NT, GB, 2>(a, waves, st);
  launch_u<XK, NT, GB, 1>(a, waves, st);
}

template <int XK, int NT>
void launch_gb(const PackedLinearLaunch& a, int gb, hipStream_t st) {
  if constexpr (XK == X_I8_BF16) {
    launch_nt<XK, NT, 32>(a, st);
  } else {
    if (gb == 128) launch_nt<XK, NT, 128>(a, st);
    else if (gb == 64) launch_nt<XK, NT, 64>(a, st);
    else if constexpr (XK != X_I8) launch_nt<XK, NT, 32>(a, st);
  }
}

template <int XK>
void launch_x(const PackedLinearLaunch& a, int gb, hipStream_t st) {
  // 64 tokens at once need more registers than float32 x or entries leave
  if (a.ntok <= 16) return launch_gb<XK, 1>(a, gb, st);
  if constexpr (XK == X_BF16 || XK == X_I8)
    if (a.ntok > 32 && !a.outlier_off) return launch_gb<XK, 4>(a, gb, st);
  launch_gb<XK, 2>(a, gb, st);
}

}  // namespace

bool rows_ok(int64_t ntok, int64_t n, int32_t G) {
  return ntok <= kRowsTokens && (G == n || G % 32 == 0);
}

hipError_t launch_rows(const PackedLinearLaunch& a, hipStream_t st) {
  const int gb = a.G == a.n || a.G % 128 == 0 ? 128 : (a.G % 64 == 0 ? 64 : 32);
  if (a.xdtype == PWQ_BF16) launch_x<X_BF16>(a, gb, st);
  else if (a.xdtype == PWQ_F32) launch_x<X_F32>(a, gb, st);
  else if (gb == 32) launch_x<X_I8_BF16>(a, gb, st);
  else launch_x<X_I8>(a, gb, st);
  return hipGetLastError();
}

}  // namespace pwq
