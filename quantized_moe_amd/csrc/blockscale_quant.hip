// Activations to E4M3 with one scale per row and 128 inputs.
//
// Bound by memory: every value is read once and leaves as a byte.  16 lanes own
// a group, 8 values per lane (16-byte loads, and for fp32 two pieces half a
// group apart so that each load instruction reads whole lines), so a block of
// 256 threads has 16 groups in flight and its maximum is four DPP steps.
// Measured: 16384 x 8192 fp32 in 111 us (6.1 TB/s; a large copy reaches 4.8),
// 1024 x 4096 bf16 in 4.6 us.
#include "blockscale.hpp"

namespace qmoe {

template <int XDT>
__global__ __launch_bounds__(256) void bs_quantize_kernel(const void* __restrict__ x, int64_t ldx, int64_t groups,
                                                          int KB, int K, uint8_t* __restrict__ q, int64_t ldq,
                                                          float* __restrict__ s) {
  const int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (g >= groups) return;
  const int lane = threadIdx.x & 15;
  const int64_t m = g / KB;
  const int c0 = (int)(g - m * KB) * BS + (XDT == X_BF16 ? 8 : 4) * lane;
  const int c1 = c0 + (XDT == X_BF16 ? 4 : 64);  // the lane's two runs of 4 values
  const bool in0 = c0 < K, in1 = c1 < K;         // (K is a multiple of 16)
  float v[8] = {};
  if constexpr (XDT == X_BF16) {
    if (in0) {
      const uint4 b = ld16(static_cast<const uint16_t*>(x) + m * ldx + c0);
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16_bits_to_float(w[i]);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
    const float* row = static_cast<const float*>(x) + m * ldx;
    if (in0) *reinterpret_cast<f32x4_t*>(v) = *reinterpret_cast<const f32x4_t*>(row + c0);
    if (in1) *reinterpret_cast<f32x4_t*>(v + 4) = *reinterpret_cast<const f32x4_t*>(row + c1);
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) a = max(a, abs_bits(v[i]));
  a = dpp_umax<0xb1>(a);   // quad_perm [1,0,3,2]
  a = dpp_umax<0x4e>(a);   // quad_perm [2,3,0,1]
  a = dpp_umax<0x141>(a);  // row_half_mirror: the other quad of 8
  a = dpp_umax<0x140>(a);  // row_mirror: the other 8 of 16
  const float sc = bs_scale(a);
  uint32_t w0 = 0, w1 = 0;
  if (a < 0x7f800000u) {  // (else the scale is NaN and the codes 0)
    if (sc >= 0x1p-80f) {
      const float r = 1.0f / sc;
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = divide_exact(v[i], sc, r);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = v[i] / sc;
    }
    w0 = e4m3x4(v[0], v[1], v[2], v[3]);
    w1 = e4m3x4(v[4], v[5], v[6], v[7]);
  }
  uint8_t* out = q + m * ldq;
  if constexpr (XDT == X_BF16) {
    if (in0) *reinterpret_cast<uint2*>(out + c0) = make_uint2(w0, w1);
  } else {
    if (in0) *reinterpret_cast<uint32_t*>(out + c0) = w0;
    if (in1) *reinterpret_cast<uint32_t*>(out + c1) = w1;
  }
  if (lane == 0) s[g] = sc;
}

hipError_t launch_bs_quantize(const void* x, int x_dtype, int64_t ldx, int M, int K, uint8_t* q, int64_t ldq, float* s,
                              hipStream_t st) {
  const int KB = bs_blocks(K);
  const int64_t groups = (int64_t)M * KB;
  const dim3 grid((unsigned)((groups + 15) / 16));  // at most 2^23 blocks
  if (x_dtype == X_BF16)
    QMOE_LAUNCH(bs_quantize_kernel<X_BF16>, grid, dim3(256), 0, st, x, ldx, groups, KB, K, q, ldq, s);
  else
    QMOE_LAUNCH(bs_quantize_kernel<X_F32>, grid, dim3(256), 0, st, x, ldx, groups, KB, K, q, ldq, s);
  return hipGetLastError();
}

}  // namespace qmoe
