// Activations to int8 with one scale per row.
//
// Bound by memory: a row is read once and stays in the registers of half a wave, of
// one or of a block of four (by its length) while its maximum is taken.  Loads go
// past the caches (16384 x 8192 fp32 125 -> 118 us), stores only where there are more
// codes than stay there for the product that follows (118 -> 115, 5.8 TB/s; 1024 x 4096
// fp32 5.1 us with stores into them and 5.6 without, 16384 x 4096 52.5 and 55).
#include "blockscale.hpp"

namespace qmoe {

// The scale of a row whose largest magnitude has the bits `amax`.
__device__ __forceinline__ float i8_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(amax), 0x1p-100f) / 127.0f;
}

// Over 32 or all 64 lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_umax(uint32_t a) {
  a = dpp_umax<0xb1>(a);   // quad_perm [1,0,3,2]
  a = dpp_umax<0x4e>(a);   // quad_perm [2,3,0,1]
  a = dpp_umax<0x141>(a);  // row_half_mirror: the other quad of 8
  a = dpp_umax<0x140>(a);  // row_mirror: the other 8 of 16
  a = max(a, (uint32_t)__shfl_xor((int)a, 16, 64));
  return LANES == 32 ? a : max(a, (uint32_t)__shfl_xor((int)a, 32, 64));
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

// LANES lanes (32, 64 or the block) own a row, NV pieces of 16 bytes of it each.
template <int XDT, int LANES, int NV>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const void* __restrict__ x, int64_t ldx, int M, int K,
                                                          int8_t* __restrict__ q, int64_t ldq, float* __restrict__ s, bool past) {
  constexpr int PER = XDT == X_BF16 ? 8 : 4;  // values of a piece
  __shared__ uint32_t wave_max[4];
  const int64_t m = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (m >= M) return;
  const int l = threadIdx.x & (LANES - 1);
  const char* row = static_cast<const char*>(x) + m * ldx * (16 / PER);
  u32x4_t v[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int c = i * LANES + l;
    v[i] = c * PER < K ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row + (int64_t)c * 16)) : u32x4_t{0, 0, 0, 0};
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
  a = lanes_umax<LANES>(a);
  if constexpr (LANES == 256) {
    if ((l & 63) == 0) wave_max[l >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; w++) a = max(a, wave_max[w]);
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
      if (past)
        __builtin_nontemporal_store(u32x2_t{w0, w1}, reinterpret_cast<u32x2_t*>(out + c * 8));
      else
        *reinterpret_cast<u32x2_t*>(out + c * 8) = u32x2_t{w0, w1};
    } else {
      const uint32_t w = number ? i8x4(u[0], u[1], u[2], u[3]) : 0;
      if (past)
        __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(out + c * 4));
      else
        *reinterpret_cast<uint32_t*>(out + c * 4) = w;
    }
  }
  if (l == 0) s[m] = sc;
}

constexpr int64_t PAST_CACHES = 100 * 1000 * 1000;

template <int XDT, int LANES, int NV>
static hipError_t launch(const void* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq, float* s, hipStream_t st) {
  auto* k = i8_quantize_kernel<XDT, LANES, NV>;
  constexpr int ROWS = 256 / LANES;
  QMOE_LAUNCH(k, dim3((unsigned)(((int64_t)M + ROWS - 1) / ROWS)), dim3(256), 0, st, x, ldx, M, K, q, ldq, s, (int64_t)M * K > PAST_CACHES);
  return hipGetLastError();
}

// Half a wave or a wave for a row of up to four pieces a lane, a block for a longer one.
template <int XDT>
static hipError_t launch_rows(const void* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq, float* s, hipStream_t st) {
  const int pieces = K / (XDT == X_BF16 ? 8 : 4);  // at most 2048, 4096
  if (pieces <= 32) return launch<XDT, 32, 1>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 64) return launch<XDT, 32, 2>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 128) return launch<XDT, 32, 4>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 256) return launch<XDT, 64, 4>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 512) return launch<XDT, 256, 2>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 1024) return launch<XDT, 256, 4>(x, ldx, M, K, q, ldq, s, st);
  if (pieces <= 2048) return launch<XDT, 256, 8>(x, ldx, M, K, q, ldq, s, st);
  if constexpr (XDT == X_F32) return launch<XDT, 256, 16>(x, ldx, M, K, q, ldq, s, st);
  return hipErrorInvalidValue;
}

hipError_t launch_i8_quantize(const void* x, int x_dtype, int64_t ldx, int M, int K, int8_t* q, int64_t ldq, float* s,
                              hipStream_t st) {
  return x_dtype == X_BF16 ? launch_rows<X_BF16>(x, ldx, M, K, q, ldq, s, st)
                           : launch_rows<X_F32>(x, ldx, M, K, q, ldq, s, st);
}

}  // namespace qmoe
