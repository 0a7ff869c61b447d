// Packing integer codes into 4 bits with an overflow list (once per layer), and
// the product of the packed layer with tokens for what the other kernels leave:
// groups that are no multiple of 32 columns, and the longest rows (a wave per row).
#include "pwq_internal.h"

#include <algorithm>

namespace pwq {
namespace {

__device__ __forceinline__ int clip_code(int c, bool asym) {
  return asym ? min(max(c, 0), 15) : min(max(c, -8), 7);
}

// One wave per tile (16 rows x 128 columns): lane l packs columns 2l, 2l + 1
// of every row and counts the codes that do not fit.
__global__ __launch_bounds__(64) void pack_tiles(const int32_t* __restrict__ codes, int64_t m,
                                                 int64_t n, int64_t ldc, int asym,
                                                 const int32_t* __restrict__ zeros, int G,
                                                 int64_t ng, uint8_t* __restrict__ qweight,
                                                 int64_t ldq, int64_t across, int64_t tiles,
                                                 int32_t* __restrict__ counts,
                                                 int32_t* __restrict__ info) {
  const int64_t tile = block_index();
  if (tile >= tiles) return;
  const int64_t r0 = tile / across * kPackRows, c0 = tile % across * kPackCols;
  const int lane = threadIdx.x;
  int over = 0, bad = 0;
  for (int i = 0; i < kPackRows; ++i) {
    const int64_t r = r0 + i;
    if (r >= m) break;
    int half[2] = {0, 0};
    bool any = false;
    for (int j = 0; j < 2; ++j) {
      const int64_t k = c0 + 2 * lane + j;
      bool out = false, wide = false;
      if (k < n) {
        const int c = codes[r * ldc + k];
        const int cc = clip_code(c, asym);
        const int64_t step = (int64_t)c - (asym ? zeros[r * ng + k / G] : 0);
        half[j] = cc & 15;
        out = c != cc;
        wide = step < -127 || step > 127;
        any = true;
      }
      over += __popcll(__ballot(out));
      bad += __popcll(__ballot(wide));
    }
    const int64_t b = c0 / 2 + lane;
    if (b < ldq) qweight[r * ldq + b] = (uint8_t)(any ? half[0] | half[1] << 4 : 0);
  }
  if (lane == 0) {
    counts[tile] = over;
    if (bad) atomicAdd(&info[0], bad);
  }
}

// Zero points to 8 bits.
__global__ __launch_bounds__(256) void pack_zeros(const int32_t* __restrict__ zeros, int64_t count,
                                                  uint8_t* __restrict__ zeros8,
                                                  int32_t* __restrict__ info) {
  const int64_t i = block_index() * 256 + threadIdx.x;
  bool bad = false;
  if (i < count) {
    const int z = zeros[i];
    bad = z < 0 || z > 127;
    zeros8[i] = (uint8_t)(bad ? 0 : z);
  }
  const int k = __popcll(__ballot(bad));
  if (k && (threadIdx.x & 63) == 0) atomicAdd(&info[1], k);
}

// Counts to first entries, in place; off[tiles] = their number (one
// workgroup, 1024 tiles a round).
__global__ __launch_bounds__(1024) void pack_scan(int32_t* __restrict__ off, int64_t tiles,
                                                  int32_t* __restrict__ info) {
  __shared__ int64_t wave_total[16];
  __shared__ int64_t base;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (threadIdx.x == 0) base = 0;
  for (int64_t i0 = 0; i0 < tiles; i0 += 1024) {
    const int64_t i = i0 + threadIdx.x;
    const int64_t c = i < tiles ? off[i] : 0;
    int64_t s = c;
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t u = __shfl_up(s, o, 64);
      if (lane >= o) s += u;
    }
    if (lane == 63) wave_total[w] = s;
    __syncthreads();
    int64_t before = base;
    for (int j = 0; j < w; ++j) before += wave_total[j];
    if (i < tiles) off[i] = (int32_t)min(before + s - c, (int64_t)INT32_MAX);
    __syncthreads();
    if (threadIdx.x == 1023) base = before + s;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    off[tiles] = (int32_t)min(base, (int64_t)INT32_MAX);
    if (base > INT32_MAX) info[0] = INT32_MAX;
  }
}

__global__ __launch_bounds__(64) void pack_entries(const int32_t* __restrict__ codes, int64_t m,
                                                   int64_t n, int64_t ldc, int asym,
                                                   int64_t across, int64_t tiles,
                                                   const int32_t* __restrict__ off,
                                                   int32_t* __restrict__ outliers,
                                                   int64_t max_out) {
  const int64_t tile = block_index();
  if (tile >= tiles) return;
  int64_t e = off[tile];
  if (off[tile + 1] == e) return;
  const int64_t r0 = tile / across * kPackRows, c0 = tile % across * kPackCols;
  const int lane = threadIdx.x;
  const unsigned long long lower = (1ull << lane) - 1;
  for (int i = 0; i < kPackRows; ++i) {
    const int64_t r = r0 + i;
    if (r >= m) break;
    for (int j = 0; j < 2; ++j) {
      const int64_t k = c0 + 64 * j + lane;
      int beyond = 0;
      if (k < n) {
        const int c = codes[r * ldc + k];
        beyond = c - clip_code(c, asym);
      }
      const unsigned long long b = __ballot(beyond != 0);
      const int64_t at = e + __popcll(b & lower);
      if (beyond && at < max_out)
        outliers[at] = (int32_t)((uint32_t)beyond << 16) | (i * kPackCols + 64 * j + lane);
      e += __popcll(b);
    }
  }
}

__global__ void clear_info(int32_t* info) { info[threadIdx.x] = 0; }

// ---- the product, any shape: one wave per row and up to TT tokens
constexpr int TT = 4;

template <typename T>
__global__ __launch_bounds__(256) void linear_any(const PackedLinearLaunch a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = block_index() * 4 + (threadIdx.x >> 6);
  if (r >= a.m) return;
  const int64_t ng = a.n / a.G;
  const float* s = a.scales + r * ng;
  const uint8_t* z = a.zeros ? a.zeros + r * ng : nullptr;
  const uint8_t* q = a.qweight + r * a.ldq;
  const int64_t across = (a.n + kPackCols - 1) / kPackCols;
  for (int64_t t0 = (int64_t)blockIdx.z * TT; t0 < a.ntok; t0 += (int64_t)gridDim.z * TT) {
    float acc[TT] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](int64_t k, float step) {
      const float sk = s[k / a.G];
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const int64_t t = t0 + i < a.ntok ? t0 + i : a.ntok - 1;
        acc[i] = fmaf(sk, step * load1<T>(a.x, t * a.ldx + k), acc[i]);
      }
    };
    for (int64_t b = lane; 2 * b < a.n; b += 64) {
      const int v = q[b];
      for (int j = 0; j < 2 && 2 * b + j < a.n; ++j) {
        const int64_t k = 2 * b + j;
        const int h = (v >> (4 * j)) & 15;
        add(k, (float)(z ? h - z[k / a.G] : (h ^ 8) - 8));
      }
    }
    if (a.outlier_off)
      for (int64_t c = 0; c < across; ++c) {
        const int64_t tile = r / kPackRows * across + c;
        const int64_t e1 = min((int64_t)a.outlier_off[tile + 1], a.n_out);
        for (int64_t e = max(a.outlier_off[tile], 0) + lane; e < e1; e += 64) {
          const int v = a.outliers[e];
          const int64_t k = c * kPackCols + (v & 127);
          if (((v >> 7) & 15) == r % kPackRows && k < a.n) add(k, (float)(v >> 16));
        }
      }
    for (int i = 0; i < TT && t0 + i < a.ntok; ++i) {
      float v = acc[i];
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
      if (lane == 0) {
        if (a.x_scales) v *= a.x_scales[t0 + i];
        if (a.ydtype == PWQ_F32) ((float*)a.y)[(t0 + i) * a.ldy + r] = v;
        else ((__bf16*)a.y)[(t0 + i) * a.ldy + r] = (__bf16)v;
      }
    }
  }
}

}  // namespace

hipError_t launch_pack_codes(const int32_t* codes, int64_t m, int64_t n, int64_t ldc, bool asym,
                             const int32_t* zeros, int G, uint8_t* qweight, uint8_t* zeros8,
                             int32_t* off, int32_t* info, hipStream_t st) {
  const int64_t across = (n + kPackCols - 1) / kPackCols, ng = n / G;
  const int64_t tiles = (m + kPackRows - 1) / kPackRows * across;
  clear_info<<<1, 2, 0, st>>>(info);
  if (tiles > 0)
    pack_tiles<<<block_grid(tiles), 64, 0, st>>>(codes, m, n, ldc, asym, zeros, G, ng, qweight,
                                                 packed_row_bytes(n), across, tiles, off, info);
  pack_scan<<<1, 1024, 0, st>>>(off, tiles, info);
  if (asym && m > 0)
    pack_zeros<<<block_grid((m * ng + 255) / 256), 256, 0, st>>>(zeros, m * ng, zeros8, info);
  return hipGetLastError();
}

hipError_t launch_pack_overflow(const int32_t* codes, int64_t m, int64_t n, int64_t ldc, bool asym,
                                const int32_t* off, int32_t* outliers, int64_t max_out,
                                hipStream_t st) {
  const int64_t across = (n + kPackCols - 1) / kPackCols;
  const int64_t tiles = (m + kPackRows - 1) / kPackRows * across;
  if (tiles == 0) return hipSuccess;
  pack_entries<<<block_grid(tiles), 64, 0, st>>>(codes, m, n, ldc, asym, across, tiles, off,
                                                 outliers, max_out);
  return hipGetLastError();
}

hipError_t launch_linear_any(const PackedLinearLaunch& a, hipStream_t st) {
  if (a.ntok == 0 || a.m == 0) return hipSuccess;
  dim3 grid = block_grid((a.m + 3) / 4);
  grid.z = (unsigned)std::min<int64_t>((a.ntok + TT - 1) / TT, 65535);
  if (a.xdtype == PWQ_F32) linear_any<float><<<grid, 256, 0, st>>>(a);
  else if (a.xdtype == PWQ_BF16) linear_any<uint16_t><<<grid, 256, 0, st>>>(a);
  else linear_any<int8_t><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace pwq
