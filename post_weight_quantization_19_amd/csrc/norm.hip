// Root-mean-square norm with the residual's addition and an 8-bit output:
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w,
//   8 bits: step = max|y| / 127 (1 if 0), q = rint(y / step).
#include "pwq_internal.h"

namespace pwq {
namespace {

template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (std::is_same_v<T, float>) return ((const float*)p)[i];
  else return bf16_to_f32(((const uint16_t*)p)[i]);
}

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

// One workgroup per token, three passes over its row.
template <typename T>
__global__ __launch_bounds__(256) void rms_norm_rows(
    const void* x, int64_t n, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
    int wf32, float eps, void* sum, int64_t lds, void* y, int ydtype, int64_t ldy, float* scales) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x;
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
    step = mx == 0.0f ? 1.0f : mx / 127.0f;
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
      const float q = __builtin_rintf(v / step);
      ((int8_t*)y)[t * ldy + k] = q == q ? (int8_t)(int)q : (int8_t)0;
    }
  }
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormLaunch& a, hipStream_t st) {
  if (a.ntok == 0) return hipSuccess;
  const dim3 grid((unsigned)a.ntok), block(256);
  const int wf32 = a.wdtype == PWQ_F32;
  if (a.xdtype == PWQ_F32)
    rms_norm_rows<float><<<grid, block, 0, st>>>(a.x, a.n, a.ldx, a.residual, a.ldr, a.weight,
                                                 wf32, a.eps, a.sum, a.lds, a.y, a.ydtype, a.ldy,
                                                 a.scales);
  else
    rms_norm_rows<uint16_t><<<grid, block, 0, st>>>(a.x, a.n, a.ldx, a.residual, a.ldr, a.weight,
                                                    wf32, a.eps, a.sum, a.lds, a.y, a.ydtype,
                                                    a.ldy, a.scales);
  return hipGetLastError();
}

}  // namespace pwq
