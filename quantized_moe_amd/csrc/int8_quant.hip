// Activations to int8 with one scale per row.
//
// Bound by memory: a row is read once and stays in the registers of one wave
// (up to 1024 inputs) or of one block of four while its maximum is taken.
#include "blockscale.hpp"

namespace qmoe {

// The scale of a row whose largest magnitude has the bits `amax`.
__device__ __forceinline__ float i8_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(amax), 0x1p-100f) / 127.0f;
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t a) {
  a = dpp_umax<0xb1>(a);   // quad_perm [1,0,3,2]
  a = dpp_umax<0x4e>(a);   // quad_perm [2,3,0,1]
  a = dpp_umax<0x141>(a);  // row_half_mirror: the other quad of 8
  a = dpp_umax<0x140>(a);  // row_mirror: the other 8 of 16
  a = max(a, (uint32_t)__shfl_xor((int)a, 16, 64));
  return max(a, (uint32_t)__shfl_xor((int)a, 32, 64));
}

// |v| <= 127 (+ rounding) as a byte: in v + 1.5 2^23 the last bit stands for 1,
// so the sum is rounded to whole numbers, halves to even, and its low byte is the
// two's complement.
__device__ __forceinline__ uint32_t i8_bits(float v) { return __float_as_uint(v + 0x1.8p23f); }
__device__ __forceinline__ uint32_t i8x4(float a, float b, float c, float d) {
  const uint32_t lo = __builtin_amdgcn_perm(i8_bits(b), i8_bits(a), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(i8_bits(d), i8_bits(c), 0x04000c0cu);
  return lo | hi;
}

// WAVES waves own a row, NV pieces of 16 bytes of it in every lane.
template <int XDT, int WAVES, int NV>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const void* __restrict__ x, int64_t ldx, int M, int K,
                                                          int8_t* __restrict__ q, int64_t ldq, float* __restrict__ s) {
  constexpr int PER = XDT == X_BF16 ? 8 : 4, LANES = 64 * WAVES;  // values of a piece
  __shared__ uint32_t wave_max[4];
  const int64_t m = WAVES == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (m >= M) return;
  const int l = threadIdx.x & (LANES - 1);
  const char* row = static_cast<const char*>(x) + m * ldx * (16 / PER);
  u32x4_t v[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int c = i * LANES + l;
    v[i] = c * PER < K ? *reinterpret_cast<const u32x4_t*>(row + (int64_t)c * 16) : u32x4_t{0, 0, 0, 0};
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int w = 0; w < 4; w++) {
      if constexpr (XDT == X_BF16) {
        a = max(a, v[i][w] << 16 & 0x7fffffffu);
        a = max(a, v[i][w] & 0x7fff0000u);
      } else {
        a = max(a, v[i][w] & 0x7fffffffu);
      }
    }
  a = wave_umax(a);
  if constexpr (WAVES > 1) {
    if ((l & 63) == 0) wave_max[l >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; w++) a = max(a, wave_max[w]);
  }
  const float sc = i8_scale(a);
  const bool number = a < 0x7f800000u;  // (else the scale is NaN and the codes 0)
  const bool normal = sc >= 0x1p-80f;
  const float r = 1.0f / sc;
  int8_t* out = q + m * ldq;
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int c = i * LANES + l;
    float u[PER];
#pragma unroll
    for (int w = 0; w < 4; w++) {
      if constexpr (XDT == X_BF16) {
        u[2 * w] = bf16_bits_to_float(v[i][w]);
        u[2 * w + 1] = __uint_as_float(v[i][w] & 0xffff0000u);
      } else {
        u[w] = __uint_as_float(v[i][w]);
      }
    }
#pragma unroll
    for (int e = 0; e < PER; e++) u[e] = normal ? divide_exact(u[e], sc, r) : u[e] / sc;
    if (c * PER >= K) continue;
    if constexpr (XDT == X_BF16) {
      const uint32_t w0 = number ? i8x4(u[0], u[1], u[2], u[3]) : 0, w1 = number ? i8x4(u[4], u[5], u[6], u[7]) : 0;
      *reinterpret_cast<uint2*>(out + c * 8) = make_uint2(w0, w1);
    } else {
      *reinterpret_cast<uint32_t*>(out + c * 4) = number ? i8x4(u[0], u[1], u[2], u[3]) : 0;
    }
  }
  if (l == 0) s[m] = sc;
}

template <int XDT, int WAVES, int NV>
static hipError_t launch(const void* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq, float* s, hipStream_t st) {
  auto* k = i8_quantize_kernel<XDT, WAVES, NV>;
  QMOE_LAUNCH(k, dim3((unsigned)(WAVES == 1 ? (M + 3) / 4 : M)), dim3(256), 0, st, x, ldx, M, K, q, ldq, s);
  return hipGetLastError();
}

// A wave for a row of up to four pieces a lane, a block for a longer one.
template <int XDT>
static hipError_t launch_rows(const void* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq, float* s, hipStream_t st) {
  const int pieces = K / (XDT == X_BF16 ? 8 : 4);  // at most 2048, 4096
  if (pieces <= 64) return launch<XDT, 1, 1>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 128) return launch<XDT, 1, 2>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 256) return launch<XDT, 1, 4>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 512) return launch<XDT, 4, 2>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 1024) return launch<XDT, 4, 4>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 2048) return launch<XDT, 4, 8>(x, ldx, M, K, q, ldq, s, st);
  if constexpr (XDT == X_F32) return launch<XDT, 4, 16>(x, ldx, M, K, q, ldq, s, st);
  return hipErrorInvalidValue;
}

hipError_t launch_i8_quantize(const void* x, int x_dtype, int64_t ldx, int M, int K, int8_t* q, int64_t ldq, float* s,
                              hipStream_t st) {
  return x_dtype == X_BF16 ? launch_rows<X_BF16>(x, ldx, M, K, q, ldq, s, st)
                           : launch_rows<X_F32>(x, ldx, M, K, q, ldq, s, st);
}

}  // namespace qmoe
