// y = x W^^T of a packed layer for up to 16 tokens: every weight is read once,
// spread in registers, and multiplied on the matrix cores.
//
// A workgroup owns a strip of 16 rows; its waves split the columns in tiles of
// 128 and their partial sums are joined in LDS in wave order.  A wave copies
// its tiles (16 rows x 64 bytes of weights, and the tokens' x) to LDS of its
// own by asynchronous copies, `depth` tiles ahead: lanes next to each other
// read bytes next to each other, which the operand layout of the matrix
// instructions does not.  (Loads straight into that layout cost a cache lookup
// per lane and bound the kernel: 16 us for up_proj's 29 MB and one 8-bit token.)
// Every tile issues the same number of copies, so that the waits are constants;
// waits chosen at run time and copies under branches took 11.2 us where these
// take 8.8, and 19.5 against 13.4 for 16 bf16 tokens.
//
// What bounds it: with one token the weights' bytes, from a last-level cache
// that holds the layer (up_proj one 8-bit token 8.8 us, 3.6 TB/s; 10.0 from HBM; a
// kernel that only reads those bytes takes 5.4 to 6.3), or a launch and the first
// bytes' way (q_proj 4.6 us; a launch alone 2.7).  bf16 x spends the vector unit on
// spreading (11.4 us), 16 tokens read 128 KB of x for every 16 rows (13.9 us).
//
// Operands: x (16 tokens) and the codes of 16 rows.  Lane l holds token l % 16
// and row l % 16, and of block h of GB columns, GB <= G, the GB / 4 from
// GB h + (GB / 4)(l / 16) on, so that a matrix instruction stays within one
// group of the steps.  The sum of a block (int32 for 8-bit x, float32 for
// exact products of bf16 otherwise) is multiplied by the step of the lane's
// row and added in float32.
//
// Codes beyond 4 bits enter as further columns: up to 32 (64 for 8-bit x)
// entries of a tile at a time, x gathered at their columns, the entry's value
// in its own row and 0 in the others.  A wave holds 256 entries in LDS; they are
// copied like the weights (q_proj one bf16 token with 0.2% of such codes 6.9
// us, 5.1 without; read by ordinary loads, which wait for the copies, 7.7).
#include "pwq_internal.h"

#include <algorithm>

namespace pwq {
namespace {

enum { X_BF16 = 0, X_I8 = 1, X_F32 = 2, X_I8_BF16 = 3 };
template <int XK> struct XType { using T = uint16_t; };
template <> struct XType<X_I8> { using T = int8_t; };
template <> struct XType<X_I8_BF16> { using T = int8_t; };
template <> struct XType<X_F32> { using T = float; };

// Eight signed halves to bytes of 16 times the code, its four bits at the top.
__device__ __forceinline__ uint2 signed16_i8(uint32_t w) {
  const uint32_t even = (w << 4) & 0xf0f0f0f0u, odd = w & 0xf0f0f0f0u;
  return make_uint2(__builtin_amdgcn_perm(odd, even, 0x05010400u),
                    __builtin_amdgcn_perm(odd, even, 0x07030602u));
}

__device__ __forceinline__ f32x4_t mma(bf16x8_t x, bf16x8_t w, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

// Eight columns of x as bf16 operands; float32 x as three bf16 parts that add up
// to it: the top, middle and last 8 bits of the significand (truncated: exact,
// and no overflow).
template <int XK> constexpr int kParts = XK == X_F32 ? 3 : 1;
template <int XK>
__device__ __forceinline__ void x_parts(const typename XType<XK>::T* p,
                                        bf16x8_t (&out)[kParts<XK>]) {
  uint4 o;
  uint32_t* q = (uint32_t*)&o;
  if constexpr (XK == X_BF16) {
    __builtin_memcpy(&o, p, 16);
    out[0] = __builtin_bit_cast(bf16x8_t, o);
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)p[e];
#pragma unroll
    for (int part = 0; part < kParts<XK>; ++part) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& lo = v[2 * i];
        float& hi = v[2 * i + 1];
        q[i] = pack_hi(lo, hi);
        if (part + 1 < kParts<XK>) {
          lo -= __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
          hi -= __uint_as_float(__float_as_uint(hi) & 0xffff0000u);
        }
      }
      out[part] = __builtin_bit_cast(bf16x8_t, o);
    }
  }
}

// LDS of a wave: slots of tiles on their way (weights 1 KB, NX KB of x), the
// steps and zero points of 16 rows x `sg` groups (4, 8 or 16), overflow
// entries.  As many tiles ahead as leave about 16 waves' worth on a CU (two
// more or two less made no difference).
constexpr int kEntries = 256, kOffsets = 64;
constexpr int depth_of(int nx) { return nx == 1 ? 4 : (nx == 2 ? 3 : 2); }
constexpr int wave_bytes(int nx, int sg, bool over) {
  return depth_of(nx) * 1024 * (1 + nx) + 2 * 16 * sg * 4 + (over ? 4 * (kEntries + kOffsets) : 0);
}

// NX: copies of x per tile, 1 KB each; ASYM: read for 8-bit x only (the other
// kinds go by the pointer).
template <int XK, int GB, int NX, bool ASYM, bool OVER>
__global__ __launch_bounds__(1024) void packed_rows(const PackedLinearLaunch a) {
  using T = typename XType<XK>::T;
  using acc_t = std::conditional_t<XK == X_I8, i32x4_t, f32x4_t>;
  constexpr int ES = sizeof(T);
  constexpr int NB = 128 / GB, NC = GB / 4;     // blocks of a tile, columns of a lane in one
  constexpr int NW = NC / 8;                    // dwords of a lane per block
  constexpr int XROW = 128 * ES, UNITS = XROW / 16, RPC = 64 / UNITS;   // x rows per copy
  constexpr int CH = 16 / NB;                   // tiles of a chunk: at most 16 groups
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t strip = blockIdx.x;
  const int tok = (int)a.ntok, n = (int)a.n, G = a.G, ng = a.ng, ldq = (int)a.ldq;
  const int xcols = (int)a.xcols;
  const int across = (n + 127) >> 7, per = a.per, sg = a.sg;
  constexpr int depth = depth_of(NX), slot_bytes = 1024 * (1 + NX);
  const int k0 = wave * per, k1 = min(across, k0 + per);
  const int rows = (int)min(a.m - strip * kPackRows, (int64_t)kPackRows);
  const bool asym = XK == X_I8 ? ASYM : a.zeros != nullptr;
  const int own = wave * wave_bytes(NX, sg, OVER);
  char* const L = smem + own;
  const uint32_t lbase = (uint32_t)(uintptr_t)(lds_char*)smem + own;
  const float* const steps = (float*)(L + depth * slot_bytes);
  const int* const zs = (int*)(steps + 16 * sg);
  const int* const ents = (const int*)(L + wave_bytes(NX, sg, false));
  const int* const offs = ents + kEntries;

  // copies: lane -> 16-byte unit.  Units of a row are permuted by the row so
  // that the operand reads below spread over the banks.
  const int wr = lane >> 2, wc = (lane & 3) ^ (wr >> 2);
  const uint32_t woff = (uint32_t)(min(wr, rows - 1) * ldq + 16 * wc);
  const uint8_t* const wbase = a.qweight + strip * kPackRows * a.ldq;
  const int xr = lane / UNITS;
  const uint32_t ldxb = (uint32_t)(a.ldx * ES);
  auto swz = [](int t) { return ES == 1 ? (t >> 1) & 7 : t & 15; };
  const bool ragged = xcols % 128 != 0;
  auto copy_tile = [&](int kt, int slot) {
    const uint32_t dst = lbase + (uint32_t)(slot * slot_bytes);
    const int wo = 64 * kt;
    copy16(woff + (wo + 16 * wc < ldq ? (uint32_t)wo : 0u - 16u * wc), wbase, dst);
    const char* const xt = (const char*)a.x + (int64_t)kt * XROW;
    if (!ragged || kt + 1 < across) {
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        const int t = j * RPC + xr, c = (lane % UNITS) ^ swz(t);
        if (NX > 1 || t < tok)
          copy16(min(t, tok - 1) * ldxb + 16u * c, xt, dst + 1024u + 1024u * j);
      }
    } else {
      // the last tile, past the row: zeros (waited for with everything else)
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        const int t = j * RPC + xr, c = (lane % UNITS) ^ swz(t);
        if (kt * XROW + 16 * c < xcols * ES)
          copy16(min(t, tok - 1) * ldxb + 16u * c, xt, dst + 1024u + 1024u * j);
        else
          *(uint4*)(L + slot * slot_bytes + 1024 + 1024 * j + 16 * lane) = make_uint4(0, 0, 0, 0);
      }
    }
  };
  const int tr = min(lr, tok - 1);                    // the lane's x row
  auto x_unit = [&](const char* xs, int c) { return xs + tr * XROW + ((c ^ swz(tr)) << 4); };

  // the kEntries overflow entries from ebase on, in LDS
  int ebase = 0;
  auto hold_entries = [&](int from) {
    ebase = from;
    const int count = (int)min(a.n_out - from, (int64_t)kEntries);
#pragma unroll
    for (int i = 0; i < kEntries / 64; ++i)
      if (64 * i + lane < count)
        copy4(4u * (64 * i + lane), a.outliers + from,
              lbase + wave_bytes(NX, sg, false) + 256u * i);
  };

  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};

  // chunks of tiles whose steps fit LDS (one, unless a wave has many tiles)
  for (int c0 = k0; c0 < k1; c0 += CH) {
    const int c1 = min(k1, c0 + CH);
    const int g0 = 128 * c0 / G;
    // steps and zero points, ahead of the tiles (a load into registers would
    // be waited for together with every copy in flight)
    for (int i = 0; i < sg / 4; ++i) {
      const int at = 64 * i + lane, r = min(at / sg, rows - 1), g = min(g0 + at % sg, ng - 1);
      const uint32_t dst = lbase + (uint32_t)(depth * slot_bytes + 256 * i);
      copy4(4u * (r * ng + g), a.scales + strip * kPackRows * ng, dst);
      if (asym) copy1(r * ng + g, a.zeros + strip * kPackRows * ng, dst + 64u * sg);
    }
    if constexpr (OVER) {
      const int* const off = a.outlier_off + strip * across + c0;
      copy4(4u * min(lane, c1 - c0), off, lbase + wave_bytes(NX, sg, false) + 4 * kEntries);
    }
#pragma unroll
    for (int d = 0; d < depth; ++d)
      if (c0 + d < c1) copy_tile(c0 + d, d);
    if constexpr (OVER) {
      // the list's place by a scalar load, which waits for no copy
      const const_int* const off = (const const_int*)(a.outlier_off + strip * across);
      hold_entries(max(off[c0], 0));
    }
    // group of the next block, without divisions
    int g = 0, in_g = 128 * c0 - g0 * G;
    int slot = 0;
    for (int kt = c0; kt < c1; ++kt) {
      // this tile's copies have landed: all but those of depth - 1 more tiles,
      // each of which issued every one of its copies (the list's entries came
      // after the first tiles)
      if (kt + depth <= c1 && !(OVER && kt == c0))
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((depth - 1) * (1 + NX)) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const char* ws = L + slot * slot_bytes;
      const char* xs = ws + 1024;
      int e0 = 0, e1 = 0;
      if constexpr (OVER) {
        e0 = max(__builtin_amdgcn_readfirstlane(offs[kt - c0]), 0);
        e1 = (int)min((int64_t)__builtin_amdgcn_readfirstlane(offs[kt - c0 + 1]), a.n_out);
      }
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        const float s = steps[lr * sg + g] * (XK == X_I8 && !asym ? 0.0625f : 1.0f);
        const int zv = zs[lr * sg + g], z = asym ? zv : 8;
        in_g += GB;
        if (in_g >= G) in_g -= G, ++g;
        uint32_t w[NW];
        {
          const int o = (GB * h + NC * lq) / 2;
          __builtin_memcpy(w, ws + lr * 64 + (((o >> 4) ^ (lr >> 2)) << 4) + (o & 15), 4 * NW);
        }
        acc_t c = {0, 0, 0, 0};
        if constexpr (XK == X_I8) {
          const uint32_t z4 = (uint32_t)z * 0x01010101u;
#pragma unroll
          for (int j = 0; j < NW; j += 2) {
            uint2 lo, hi;
            if (asym) lo = steps_i8(w[j], z4), hi = steps_i8(w[j + 1], z4);
            else lo = signed16_i8(w[j]), hi = signed16_i8(w[j + 1]);
            const i32x4_t f = {(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
            const i32x4_t v = *(const i32x4_t*)x_unit(xs, (GB * h + NC * lq + 8 * j) / 16);
            c = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, f, c, 0, 0, 0);
          }
        } else {
          const uint32_t bias = asym ? kUnsignedHalves : kSignedHalves;
#pragma unroll
          for (int j = 0; j < NW; ++j) {
            const bf16x8_t f = __builtin_bit_cast(bf16x8_t, steps_bf16(w[j], bias, z));
            const int col = GB * h + NC * lq + 8 * j;
            T xv[8];
            if constexpr (XK == X_BF16) {
              __builtin_memcpy(xv, x_unit(xs, col / 8), 16);
            } else if constexpr (XK == X_F32) {
              __builtin_memcpy(xv, x_unit(xs, col / 4), 16);
              __builtin_memcpy(xv + 4, x_unit(xs, col / 4 + 1), 16);
            } else {
              __builtin_memcpy(xv, x_unit(xs, col / 16) + col % 16, 8);
            }
            bf16x8_t v[kParts<XK>];
            x_parts<XK>(xv, v);
#pragma unroll
            for (int part = 0; part < kParts<XK>; ++part) c = mma(v[part], f, c);
          }
        }
        acc_t ce = {0, 0, 0, 0};
        constexpr int PE = XK == X_I8 ? 16 : 8;          // entries of a lane at a time
        if constexpr (OVER) for (int e = e0; e < e1; e += 4 * PE) {
          // the lane's entries e + 4 i + l / 16; most tiles have few, so by twos
          int val[PE] = {}, most = 0;
          T xe[PE] = {};
          if (e < ebase || min(e + 4 * PE, e1) > ebase + kEntries) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            hold_entries(e);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          }
#pragma unroll
          for (int i = 0; i < PE; i += 2) {
            if (e + 4 * i >= e1) break;
#pragma unroll
            for (int k = i; k < i + 2; ++k) {
              const int ent = ents[min(e + 4 * k + lq, e1 - 1) - ebase];
              const int col = ent & 127;                 // (columns past n hold zeros)
              xe[k] = *(const T*)(x_unit(xs, col * ES / 16) + col * ES % 16);
              val[k] = e + 4 * k + lq < e1 && col / GB == h && ((ent >> 7) & 15) == lr ? ent >> 16
                                                                                      : 0;
              if constexpr (XK == X_I8 && ASYM) most = max(most, val[k]);
            }
          }
          if constexpr (XK == X_I8) {
            i32x4_t v;
            __builtin_memcpy(&v, xe, 16);
            auto multiply = [&](auto of) {
              i32x4_t f = {0, 0, 0, 0};
#pragma unroll
              for (int i = 0; i < PE; ++i) f[i / 4] |= (of(val[i]) & 255) << (8 * (i % 4));
              ce = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, f, ce, 0, 0, 0);
            };
            // an entry beside a zero point above 15 goes to 239: what a signed
            // byte does not hold is multiplied on its own
            if (ASYM && __any(most > 127)) {
              multiply([](int e) { return min(e, 127); });
              multiply([](int e) { return max(e - 127, 0); });
            } else {
              multiply([](int e) { return e; });
            }
          } else {
            float d[PE];
#pragma unroll
            for (int i = 0; i < PE; ++i) d[i] = (float)val[i];
            const uint4 o = make_uint4(pack_hi(d[0], d[1]), pack_hi(d[2], d[3]),
                                       pack_hi(d[4], d[5]), pack_hi(d[6], d[7]));
            bf16x8_t v[kParts<XK>];
            x_parts<XK>(xe, v);
#pragma unroll
            for (int part = 0; part < kParts<XK>; ++part)
              ce = mma(v[part], __builtin_bit_cast(bf16x8_t, o), ce);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (XK == X_I8) {
            int v = c[e];
            if constexpr (OVER) v += asym ? ce[e] : 16 * ce[e];
            acc[e] = fmaf(s, (float)v, acc[e]);
          } else {
            float v = c[e];
            if constexpr (OVER) v += ce[e];
            acc[e] = fmaf(s, v, acc[e]);
          }
        }
      }
      if (kt + depth < c1) {
        // the slot's reads are done before it is filled again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy_tile(kt + depth, slot);
      }
      if (++slot == depth) slot = 0;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // join the waves' sums in their order; lane l: tokens 4 (l / 16) + e, row l % 16
  float* const joined = (float*)smem;
  const int stride = wave_bytes(NX, sg, OVER) / 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) joined[wave * stride + e * 64 + lane] = acc[e];
  __syncthreads();
  for (int v = threadIdx.x; v < 256; v += blockDim.x) {
    const int e = v >> 6, l = v & 63;
    const int64_t t = 4 * (l >> 4) + e, r = strip * kPackRows + (l & 15);
    if (t >= tok || r >= a.m) continue;
    float sum = joined[v];
#pragma unroll 4
    for (int o = 1; o < waves; ++o) sum += joined[o * stride + v];
    if (a.x_scales) sum *= a.x_scales[t];
    if (a.ydtype == PWQ_F32) ((float*)a.y)[t * a.ldy + r] = sum;
    else ((__bf16*)a.y)[t * a.ldy + r] = (__bf16)sum;
  }
}

// x to rows of `wide` columns, zeros past n.
template <typename T>
__global__ __launch_bounds__(256) void pad_rows(const T* __restrict__ x, int64_t ntok, int64_t n,
                                                int64_t ldx, T* __restrict__ out, int64_t wide) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= ntok * wide) return;
  const int64_t t = i / wide, k = i % wide;
  out[i] = k < n ? x[t * ldx + k] : T(0);
}

constexpr int kLdsBytes = 160 * 1024;

template <int XK, int GB, int NX, bool ASYM, bool OVER>
void launch_waves(PackedLinearLaunch a, hipStream_t st) {
  // about 16 waves per CU over the whole launch, as far as LDS goes (up_proj
  // one bf16 token 10.9 us with 4096 waves, 13.2 with 6144; down_proj 11.0 with
  // workgroups of up to 16 waves, 12.2 with 12)
  const int64_t strips = (a.m + kPackRows - 1) / kPackRows, across = (a.n + 127) / 128;
  int most = (int)std::clamp<int64_t>(4096 / strips, 1, 16), bytes;
  for (;; --most) {
    a.per = (int)((across + most - 1) / most);
    a.sg = 4;
    while (a.sg < std::min(16, a.per * (128 / GB))) a.sg *= 2;
    bytes = wave_bytes(NX, a.sg, OVER);
    if (most * bytes <= kLdsBytes) break;
  }
  a.ng = (int)(a.n / a.G);
  const int waves = (int)((across + a.per - 1) / a.per);
  packed_rows<XK, GB, NX, ASYM, OVER>
      <<<dim3((unsigned)strips), 64 * waves, waves * bytes, st>>>(a);
}

template <int XK, int GB, int NX>
void launch_nx(const PackedLinearLaunch& a, hipStream_t st) {
  const bool over = a.outlier_off != nullptr;
  if constexpr (XK == X_I8) if (a.zeros)
    return over ? launch_waves<XK, GB, NX, true, true>(a, st)
                : launch_waves<XK, GB, NX, true, false>(a, st);
  over ? launch_waves<XK, GB, NX, false, true>(a, st)
       : launch_waves<XK, GB, NX, false, false>(a, st);
}

// Copies of x per tile: 1 KB holds 4 tokens of bf16, 8 of 8 bits, 2 of float32.
template <int XK, int GB>
void launch_gb(const PackedLinearLaunch& a, hipStream_t st) {
  if constexpr (XK == X_BF16) {
    if (a.ntok <= 4) return launch_nx<XK, GB, 1>(a, st);
    a.ntok <= 8 ? launch_nx<XK, GB, 2>(a, st) : launch_nx<XK, GB, 4>(a, st);
  } else if constexpr (XK == X_F32) {
    if (a.ntok <= 4) return launch_nx<XK, GB, 2>(a, st);
    a.ntok <= 8 ? launch_nx<XK, GB, 4>(a, st) : launch_nx<XK, GB, 8>(a, st);
  } else {
    a.ntok <= 8 ? launch_nx<XK, GB, 1>(a, st) : launch_nx<XK, GB, 2>(a, st);
  }
}

template <int XK>
void launch_x(const PackedLinearLaunch& a, int gb, hipStream_t st) {
  if constexpr (XK != X_I8_BF16) {
    if (gb == 128) return launch_gb<XK, 128>(a, st);
    if (gb == 64) return launch_gb<XK, 64>(a, st);
  }
  if constexpr (XK != X_I8) launch_gb<XK, 32>(a, st);
}

}  // namespace

// Up to 16 tokens, what a matrix operand holds (as batch_tiles, 16 bf16 tokens
// of q_proj, up_proj and down_proj take 11.5, 20.1 and 21.1 us instead of 6.3, 16.3
// and 17.1, 8-bit ones 9.9, 15.3 and 16.2 instead of 5.2, 12.5 and 13.3); steps
// per 32 columns or more (or per row); offsets and the launch's 4 m threads
// within 32 bits.
bool rows_ok(int64_t ntok, int64_t m, int64_t n, int32_t G) {
  return ntok <= kRowsTokens && (G == n || G % 32 == 0) && n < (1 << 24) && m < (1 << 29);
}

// Bytes of the padded copy of x; 0 where its rows can be copied in 16-byte
// units as they are.
size_t rows_staged_bytes(const void* x, int32_t xdtype, int64_t ntok, int64_t n, int64_t ldx) {
  const int64_t es = xdtype == PWQ_I8 ? 1 : (xdtype == PWQ_BF16 ? 2 : 4);
  const bool direct = ldx < (1 << 24) && ldx * es % 16 == 0 && n * es % 16 == 0 &&
                      (uintptr_t)x % 16 == 0;
  return direct ? 0 : (size_t)(ntok * ((n + 15) / 16 * 16) * es);
}

hipError_t launch_rows(PackedLinearLaunch a, void* staged, hipStream_t st) {
  if (staged) {
    const int64_t wide = (a.n + 15) / 16 * 16;
    const dim3 grid((unsigned)((a.ntok * wide + 255) / 256));
    if (a.xdtype == PWQ_I8)
      pad_rows<<<grid, 256, 0, st>>>((const uint8_t*)a.x, a.ntok, a.n, a.ldx, (uint8_t*)staged,
                                     wide);
    else if (a.xdtype == PWQ_BF16)
      pad_rows<<<grid, 256, 0, st>>>((const uint16_t*)a.x, a.ntok, a.n, a.ldx, (uint16_t*)staged,
                                     wide);
    else
      pad_rows<<<grid, 256, 0, st>>>((const uint32_t*)a.x, a.ntok, a.n, a.ldx, (uint32_t*)staged,
                                     wide);
    a.x = staged;
    a.ldx = wide;
  }
  a.xcols = staged ? a.ldx : a.n;
  const int gb = a.G == a.n || a.G % 128 == 0 ? 128 : (a.G % 64 == 0 ? 64 : 32);
  if (a.xdtype == PWQ_BF16) launch_x<X_BF16>(a, gb, st);
  else if (a.xdtype == PWQ_F32) launch_x<X_F32>(a, gb, st);
  else if (gb == 32) launch_x<X_I8_BF16>(a, gb, st);
  else launch_x<X_I8>(a, gb, st);
  return hipGetLastError();
}

}  // namespace pwq
