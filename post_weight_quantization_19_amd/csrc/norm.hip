// Root-mean-square norm with the residual's addition and an 8-bit output:
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w,
//   8 bits: step = max|y| / 127 (1 if that is 0), q = rint(y / step).
//
// rms_norm_regs keeps a token's row in registers: x and residual are read
// once, the sum and y written once (7 bytes an element for bf16 in, 8 bits
// out), with two reductions in between.  TPR threads share a row, 8
// consecutive elements each NV times over; a workgroup keeps the weight of
// its columns in registers and walks over tokens.  Rows longer than the
// registers hold take rms_norm_rows, which reads them three times.
//
// What bounds it: HBM for many tokens (8192 x 4096 bf16 with residual to 8 bits
// 49 us, 4.8 TB/s; 2048 x 14336 bf16 27.4 us, 4.3 TB/s; a large copy reaches
// 5.1), a launch and two reductions for few (one token of 4096 4.4 us).  Rows
// that are not 16-byte aligned read in smaller pieces (2047 x 4099 23 us, 2.5
// TB/s).
#include "pwq_internal.h"

#include <algorithm>

namespace pwq {
namespace {

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += red[i];
  return s;
}

// Maximum in which a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

// The code of a rounded quotient; 0 in a token whose maximum (or step) is not
// finite.  A step of a few units of the smallest float32 is rounded by up to a
// half, so that quotients go to 190: they are cut at 127.
__device__ __forceinline__ float code_of(float q, float mx) {
  return mx <= __FLT_MAX__ ? fminf(fmaxf(q, -127.0f), 127.0f) : 0.0f;
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor(v, o, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
  for (int i = 1; i < (int)(blockDim.x >> 6); ++i) s = max_nan(s, red[i]);
  return s;
}

struct __attribute__((packed, aligned(1))) pack16 { uint32_t v[4]; };
struct __attribute__((packed, aligned(1))) pack8 { uint32_t v[2]; };

// Eight consecutive elements as they are in memory (any alignment).
template <typename T> struct Raw { pack16 v[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Raw<T> raw8(const T* p) { return *(const Raw<T>*)p; }
__device__ __forceinline__ void widen(const Raw<float>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.v[e / 4].v[e % 4]);
}
__device__ __forceinline__ void widen(const Raw<uint16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(r.v[0].v[e] << 16);
    v[2 * e + 1] = __uint_as_float(r.v[0].v[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  const __bf16 x[2] = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, x);
}

// Elements lo .. 7 to p .. p + 7.
template <typename T>
__device__ __forceinline__ void store8(T* p, int lo, const float (&v)[8]) {
  if (lo == 0) {
    if constexpr (std::is_same_v<T, float>) {
      pack16 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) a.v[e] = __float_as_uint(v[e]), b.v[e] = __float_as_uint(v[4 + e]);
      ((pack16*)p)[0] = a, ((pack16*)p)[1] = b;
    } else if constexpr (std::is_same_v<T, uint16_t>) {
      pack16 a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a.v[e] = two_bf16(v[2 * e], v[2 * e + 1]);
      *(pack16*)p = a;
    } else {
      pack8 a;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a.v[h] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) a.v[h] |= ((uint32_t)(int)v[4 * h + e] & 255u) << (8 * e);
      }
      *(pack8*)p = a;
    }
  } else {
#pragma unroll
    for (int e = 1; e < 8; ++e)
      if (e >= lo) {
        if constexpr (std::is_same_v<T, float>) p[e] = v[e];
        else if constexpr (std::is_same_v<T, uint16_t>) p[e] = (uint16_t)two_bf16(v[e], 0.0f);
        else p[e] = (T)(int)v[e];
      }
  }
}

// Sum or maximum over the TPR threads of a row (the workgroup, or a wave).
template <int TPR, typename Op>
__device__ __forceinline__ float row_reduce(float v, float* red, Op op) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = op(v, __shfl_xor(v, o, 64));
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v = op(v, red[i]);
  }
  return v;
}

// The vector of a thread at or past the row's end starts 8 before the end
// instead, and its first `lo` elements, a neighbour's, count as 0.
template <typename T, int TPR, int NV, bool RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_norm_regs(const RmsNormLaunch a) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;       // rows of a workgroup at a time
  __shared__ float red[2][2][16];                      // [token parity][sum, maximum]
  const int in = threadIdx.x % TPR, n = (int)a.n;
  const bool ragged = n < 8 * TPR * NV;
  int at[NV], lo[NV];
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = 8 * (in + TPR * i);
    at[i] = min(k, n - 8);
    lo[i] = min(k - at[i], 8);
    if (a.wdtype == PWQ_F32) widen(raw8((const float*)a.weight + at[i]), w[i]);
    else widen(raw8((const uint16_t*)a.weight + at[i]), w[i]);
  }
  const float inv_n = 1.0f / (float)n;
  const int64_t step_t = (int64_t)gridDim.x * RPB;
  int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (t >= a.ntok) return;
  Raw<T> x[NV], q[RES ? NV : 1];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = raw8((const T*)a.x + row * a.ldx + at[i]);
    if constexpr (RES)
#pragma unroll
      for (int i = 0; i < NV; ++i) q[i] = raw8((const T*)a.residual + row * a.ldr + at[i]);
  };
  load(t);
  for (int parity = 0; t < a.ntok; t += step_t, parity ^= 1) {
    float h[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      widen(x[i], h[i]);
      if constexpr (RES) {
        float v[8];
        widen(q[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += v[e];
      }
      if (ragged)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = e >= lo[i] ? h[i][e] : 0.0f;
    }
    if (t + step_t < a.ntok) load(t + step_t);           // the next token's, behind this one
    if (a.sum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) store8((T*)a.sum + t * a.lds + at[i], lo[i], h[i]);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    ss = row_reduce<TPR>(ss, red[parity][0], [](float p, float q) { return p + q; });
    const float r = rsqrtf(fmaf(ss, inv_n, a.eps));
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] = h[i][e] * r * w[i][e];
        mx = max_nan(mx, fabsf(h[i][e]));
      }
    if (a.ydtype == PWQ_I8) {
      mx = row_reduce<TPR>(mx, red[parity][1], max_nan);
      float step = mx / 127.0f;
      if (step == 0.0f) step = 1.0f;
      if (in == 0) a.scales[t] = step;
      // rint(h / step).  The product with the reciprocal is within 2^-16 of the
      // quotient (1.5 units of the last place of 127), so that it rounds alike
      // unless it lies that near a tie; there, and where the maximum or the
      // reciprocal may not be finite, divide.  (Always dividing: one token of
      // 14336 6.0 us instead of 5.2, 2048 of them 59.5 instead of 56.5.)
      const float inv = 1.0f / step;
      const float near = mx > 1e-30f && mx <= __FLT_MAX__ ? 0.5f - 0x1p-15f : -1.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float c[8], off = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = h[i][e] * inv;
          c[e] = __builtin_rintf(v);
          off = fmaxf(off, fabsf(v - c[e]));
        }
        if (off > near)
#pragma unroll
          for (int e = 0; e < 8; ++e) c[e] = code_of(__builtin_rintf(h[i][e] / step), mx);
        store8((int8_t*)a.y + t * a.ldy + at[i], lo[i], c);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (a.ydtype == PWQ_F32) store8((float*)a.y + t * a.ldy + at[i], lo[i], h[i]);
        else store8((uint16_t*)a.y + t * a.ldy + at[i], lo[i], h[i]);
      }
    }
  }
}

// One workgroup per token, three passes over its row.
template <typename T>
__global__ __launch_bounds__(256) void rms_norm_rows(
    const void* x, int64_t ntok, int64_t n, int64_t ldx, const void* residual, int64_t ldr,
    const void* weight, int wf32, float eps, void* sum, int64_t lds, void* y, int ydtype, int64_t ldy, float* scales) {
  __shared__ float red[4];
  const int64_t t = block_index();
  if (t >= ntok) return;
  auto h_at = [&](int64_t k) {
    float h = load1<T>(x, t * ldx + k);
    if (residual) h += load1<T>(residual, t * ldr + k);
    return h;
  };
  auto w_at = [&](int64_t k) {
    return wf32 ? ((const float*)weight)[k] : bf16_to_f32(((const uint16_t*)weight)[k]);
  };
  float ss = 0.0f;
  for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
    const float h = h_at(k);
    ss = fmaf(h, h, ss);
  }
  const float r = rsqrtf(block_sum(ss, red) / (float)n + eps);
  float step = 1.0f;
  if (ydtype == PWQ_I8) {
    float mx = 0.0f;
    for (int64_t k = threadIdx.x; k < n; k += blockDim.x)
      mx = max_nan(mx, fabsf(h_at(k) * r * w_at(k)));
    mx = block_max(mx, red);
    step = mx / 127.0f;
    if (step == 0.0f) step = 1.0f;
    if (threadIdx.x == 0) scales[t] = step;
  }
  for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
    const float h = h_at(k);
    const float v = h * r * w_at(k);
    if (sum) {
      if constexpr (std::is_same_v<T, float>) ((float*)sum)[t * lds + k] = h;
      else ((__bf16*)sum)[t * lds + k] = (__bf16)h;
    }
    if (ydtype == PWQ_F32) ((float*)y)[t * ldy + k] = v;
    else if (ydtype == PWQ_BF16) ((__bf16*)y)[t * ldy + k] = (__bf16)v;
    else {
      ((int8_t*)y)[t * ldy + k] = (int8_t)(int)code_of(__builtin_rintf(v / step), step);
    }
  }
}

template <typename T, int TPR, int NV>
void launch_regs(const RmsNormLaunch& a, hipStream_t st) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  // workgroups that run at once, 1536 threads a CU: the rest of the tokens are
  // walked over (1024 and 2048 threads: 8192 x 8192 96 and 91 us instead of 89;
  // 8192 x 4096 47.0 and 47.4 instead of 48.7; 8192 x 14336 169 and 173, 172)
  const int64_t blocks = std::min<int64_t>(
      (a.ntok + RPB - 1) / RPB, 256 * (1536 / std::max(TPR, 256) + (TPR == 1024)));
  const dim3 grid((unsigned)blocks), block(TPR < 256 ? 256 : TPR);
  if (a.residual) rms_norm_regs<T, TPR, NV, true><<<grid, block, 0, st>>>(a);
  else rms_norm_regs<T, TPR, NV, false><<<grid, block, 0, st>>>(a);
}

template <typename T>
void launch_loop(const RmsNormLaunch& a, hipStream_t st) {
  rms_norm_rows<T><<<block_grid(a.ntok), 256, 0, st>>>(
      a.x, a.ntok, a.n, a.ldx, a.residual, a.ldr, a.weight, a.wdtype == PWQ_F32, a.eps, a.sum,
      a.lds, a.y, a.ydtype, a.ldy, a.scales);
}

template <typename T>
void launch_type(const RmsNormLaunch& a, hipStream_t st) {
  const int64_t n = a.n;
  // Each form's width is what its registers hold.  Up to 2048 columns a wave a
  // row, without barriers; above, few tokens: more threads a row, for latency;
  // many: fewer, for fewer barriers.  us, bf16 with residual to 8 bits, this form
  // and the other (1024 threads up to 256 tokens, 256 or 512 above):
  //    columns   1 token     256 tokens   512 tokens   4096 tokens
  //        512   2.5, 4.3    -            3.2, 3.7     6.0, 9.7
  //       2048   4.1, 4.3    -            5.4, 4.4     15.9, 15.7
  //       4096   4.4, 3.5    5.4, 4.8     6.6, 9.6     27, 45
  //       8192   4.3, 4.5    6.8, 7.3     10.8, 12.2   48, 55
  //      14336   5.8, 6.1    10.4, 10.9   19.0, 18.6   94, 90
  if (n < 8) return launch_loop<T>(a, st);
  if (n <= 512) return launch_regs<T, 64, 1>(a, st);
  if (n <= 1024) return launch_regs<T, 64, 2>(a, st);
  if (n <= 2048) return launch_regs<T, 64, 4>(a, st);
  if (a.ntok >= 512) {
    if (n <= 4096) return launch_regs<T, 256, 2>(a, st);
    if (n <= 8192) return launch_regs<T, 256, 4>(a, st);
    if (n <= 16384) return launch_regs<T, 512, 4>(a, st);
  }
  if (n <= 8192) return launch_regs<T, 1024, 1>(a, st);
  if (n <= 16384) return launch_regs<T, 1024, 2>(a, st);
  if (n <= 32768) return launch_regs<T, 1024, 4>(a, st);
  launch_loop<T>(a, st);
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormLaunch& a, hipStream_t st) {
  if (a.ntok == 0) return hipSuccess;
  if (a.xdtype == PWQ_F32) launch_type<float>(a, st);
  else launch_type<uint16_t>(a, st);
  return hipGetLastError();
}

}  // namespace pwq
