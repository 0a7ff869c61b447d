// Device-side helpers shared by the libpwq kernels (gfx950 / CDNA4 only).
//
// MFMA operand layouts used below (wave64):
//   v_mfma_f32_32x32x16_bf16 : A lane l holds A[l%32][8*(l/32) + e], e=0..7;
//                              B lane l holds B[8*(l/32) + e][l%32].
//   v_mfma_f32_32x32x2f32    : A lane l holds A[l%32][l/32]; B [l/32][l%32].
//   v_mfma_f64_16x16x4f64    : A lane l holds A[l%16][l/16]; B [l/16][l%16].
//   32x32 results: lane l, register r -> C[8*(r/4) + 4*(l/32) + r%4][l%32].
//   16x16 f32 results: lane l, register r -> C[4*(l/16) + r][l%16].
//   16x16 f64 results: lane l, register r -> C[4*r + l/16][l%16].
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace pwq {

typedef __attribute__((__vector_size__(8 * sizeof(short)))) short bf16x8_t;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef __attribute__((__vector_size__(4 * sizeof(double)))) double f64x4_t;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) {
  return __uint_as_float(((uint32_t)b) << 16);
}

// Element loads from W (bf16 bits or float) widened to the working type.
template <typename T>
__device__ __forceinline__ T load_w(const void* W, int32_t wdtype, int64_t idx) {
  if (wdtype == 1) return (T)bf16_to_f32(((const uint16_t*)W)[idx]);
  return (T)(((const float*)W)[idx]);
}

// Broadcast lane q of every 16-lane row to the whole row (DPP row_newbcast).
// Every lane is written (all rows and banks enabled), so the "old" operand
// is the value itself: no separate register has to be cleared first.
template <int Q>
__device__ __forceinline__ float row_bcast(float v) {
  const int b = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, 0x150 + Q, 0xF, 0xF, false));
}
template <int Q>
__device__ __forceinline__ double row_bcast(double v) {
  long long b = __builtin_bit_cast(long long, v);
  const int l0 = (int)(b & 0xffffffffll), h0 = (int)(b >> 32);
  int lo = __builtin_amdgcn_update_dpp(l0, l0, 0x150 + Q, 0xF, 0xF, false);
  int hi = __builtin_amdgcn_update_dpp(h0, h0, 0x150 + Q, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (long long)(((unsigned long long)(unsigned)hi << 32) |
                                                (unsigned long long)(unsigned)lo));
}

// Straight-line "loop" I = N-1, N-2, ..., 0 with I a compile-time constant in
// the body (register arrays stay registers; DPP controls stay immediates).
template <int I, typename F>
__device__ __forceinline__ void static_for_down(F&& f) {
  if constexpr (I >= 0) {
    f(std::integral_constant<int, I>{});
    static_for_down<I - 1>(f);
  }
}

// Global -> LDS copy of a ROWS x COLS tile by NT threads: every load is issued
// before the first LDS store, so the tile costs one memory latency, not one
// per loop iteration.  get(r, c) returns the (masked) source element.
template <typename T, int ROWS, int COLS, int NT, int LDD, typename Get>
__device__ __forceinline__ void tile_to_lds(T* __restrict__ dst, int tid, Get&& get) {
  constexpr int PER = (ROWS * COLS + NT - 1) / NT;
  T v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid + NT * i;
    v[i] = (e < ROWS * COLS) ? get(e / COLS, e % COLS) : (T)0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid + NT * i;
    if (e < ROWS * COLS) dst[(e / COLS) * LDD + e % COLS] = v[i];
  }
}

// Workgroup barrier for LDS traffic only: waits for this wave's LDS
// operations (lgkmcnt(0)) and meets the other waves, without the release
// fence of __syncthreads(), whose vmcnt(0) would drain global loads that are
// deliberately still in flight.  The signal fences stop the compiler from
// moving memory accesses across it.
__device__ __forceinline__ void lds_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // vmcnt(63) expcnt(7) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Empty register constraint: the value must exist in a VGPR at this point.
__device__ __forceinline__ void pin(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void pin(double& v) { asm volatile("" : "+v"(v)); }

// Straight-line "loop" I = 0 .. N-1 with I a compile-time constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for_up(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for_up<N, I + 1>(f);
  }
}

__device__ __forceinline__ float rint_t(float x) { return __builtin_rintf(x); }
__device__ __forceinline__ double rint_t(double x) { return __builtin_rint(x); }

// Deterministic wave64 sum (butterfly; the same order on every run).
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ float wave_min(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fminf(v, __shfl_xor(v, o, 64));
  return v;
}

// Kernel status flags kept in the workspace: [0] = first failing column + 1.
struct DevFlags {
  int32_t info;
  int32_t pad[63];
};

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(4))) int const_int;

// Asynchronous copies of 16 bytes, 4 bytes, or one byte (to a dword) per active
// lane: sbase + voff of each lane to lds + 16 lane, or lds + 4 lane (lds and
// sbase wave-uniform).  M0 is restored.
#define PWQ_COPY(NAME, OP)                                                                    \
  __device__ __forceinline__ void NAME(uint32_t voff, const void* sbase, uint32_t lds) {     \
    uint32_t keep;                                                                           \
    asm volatile(                                                                            \
        "s_mov_b32 %0, m0\n\t"                                                               \
        "s_mov_b32 m0, %3\n\t" OP                                                            \
        " %1, %2\n\t"                                                                        \
        "s_mov_b32 m0, %0"                                                                   \
        : "=&s"(keep)                                                                        \
        : "v"(voff), "s"(sbase), "s"(lds)                                                    \
        : "memory");                                                                         \
  }
PWQ_COPY(copy16, "global_load_lds_dwordx4")
PWQ_COPY(copy4, "global_load_lds_dword")
PWQ_COPY(copy1, "global_load_lds_ubyte")
#undef PWQ_COPY

// Index of a workgroup in a launch of block_grid workgroups.
constexpr int kGridShift = 21;
__device__ __forceinline__ int64_t block_index() {
  return (int64_t)blockIdx.y << kGridShift | blockIdx.x;
}

// An element of x in float32 (uint16_t: bf16).
template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (std::is_same_v<T, float>) return ((const float*)p)[i];
  else if constexpr (std::is_same_v<T, int8_t>) return (float)((const int8_t*)p)[i];
  else return bf16_to_f32(((const uint16_t*)p)[i]);
}

// The upper halves of two float32 (exact for small integers).
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Eight 4-bit steps of a dword to bf16, z the zero point (8 for signed halves).  A
// code, bits 0 .. 3 of a float16 64 + u / 16 (`bias` in every half; signed halves
// get their top bit flipped), becomes 1024 + u - (1024 + z) in one multiplication
// and addition; the upper half of that float32 holds the difference exactly.
// (Codes as 16 + u in bf16, corrected by 16 + z times the sum of x, made one to
// 16 tokens 1 to 3% faster, but lost three bits of a small result and all of
// one whose x is above 2^123.)
constexpr uint32_t kUnsignedHalves = 0x54005400u, kSignedHalves = 0x54085408u;
__device__ __forceinline__ uint4 steps_bf16(uint32_t w, uint32_t bias, int z) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  constexpr uint32_t M = 0x000f000fu;
  const float zb = 1024.0f + (float)z;
  float lo[4], hi[4];                                  // columns i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2_t h = __builtin_bit_cast(f16x2_t, ((w >> (4 * i)) & M) ^ bias);
    lo[i] = fmaf((float)h[0], 16.0f, -zb);
    hi[i] = fmaf((float)h[1], 16.0f, -zb);
  }
  return make_uint4(pack_hi(lo[0], lo[1]), pack_hi(lo[2], lo[3]), pack_hi(hi[0], hi[1]),
                    pack_hi(hi[2], hi[3]));
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

}  // namespace pwq
