// Activations to E4M3 with one scale per row and 128 inputs.
//
// Bound by memory: every value is read once and written once as a byte.  A
// half wave (32 lanes) owns a group, 4 values per lane.
#include "blockscale.hpp"

namespace qmoe {

template <int XDT>
__global__ __launch_bounds__(256) void bs_quantize_kernel(const void* __restrict__ x, int64_t ldx, int64_t groups,
                                                          int KB, int K, uint8_t* __restrict__ q, int64_t ldq,
                                                          float* __restrict__ s) {
  const int64_t g = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (g >= groups) return;
  const int lane = threadIdx.x & 31;
  const int64_t m = g / KB;
  const int c = (int)(g - m * KB) * BS + 4 * lane;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < K) {
    if constexpr (XDT == X_BF16) {
      const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + m * ldx + c);
      v[0] = bf16_bits_to_float(b.x);
      v[1] = __uint_as_float(b.x & 0xffff0000u);
      v[2] = bf16_bits_to_float(b.y);
      v[3] = __uint_as_float(b.y & 0xffff0000u);
    } else {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + m * ldx + c);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) a = max(a, abs_bits(v[i]));
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, i, 64));
  const float sc = bs_scale(a);
  const bool bad = a >= 0x7f800000u;
  if (c < K)
    *reinterpret_cast<uint32_t*>(q + m * ldq + c) = bad ? 0u : e4m3x4(v[0] / sc, v[1] / sc, v[2] / sc, v[3] / sc);
  if (lane == 0) s[g] = sc;
}

hipError_t launch_bs_quantize(const void* x, int x_dtype, int64_t ldx, int M, int K, uint8_t* q, int64_t ldq, float* s,
                              hipStream_t st) {
  const int KB = bs_blocks(K);
  const int64_t groups = (int64_t)M * KB;
  const dim3 grid((unsigned)((groups + 7) / 8));
  if (x_dtype == X_BF16)
    QMOE_LAUNCH(bs_quantize_kernel<X_BF16>, grid, dim3(256), 0, st, x, ldx, groups, KB, K, q, ldq, s);
  else
    QMOE_LAUNCH(bs_quantize_kernel<X_F32>, grid, dim3(256), 0, st, x, ldx, groups, KB, K, q, ldq, s);
  return hipGetLastError();
}

}  // namespace qmoe
