// Gate: scores, groups and top-k of given router logits (definition in
// include/moe.h).  Contraction is off in this file: the fp32 steps of the
// scores decide selections near a tie, so each is rounded on its own.
#include <math.h>

#include "common.hpp"
#include "kernels.hpp"
#include "topk.hpp"

#pragma clang fp contract(off)

namespace qmoe {

// e^t for t in [-80, 80]: the steps of sigmoid32 (include/moe.h).
__device__ __forceinline__ float exp32(float t) {
  const float kf = t * 0x1.715476p+0f;
  const float n = (kf + 0x1.8p+23f) - 0x1.8p+23f;
  const float r = (t - n * 0x1.62e400p-1f) - n * 0x1.7f7d1cp-20f;
  float p = 0x1.6c16c2p-10f;
  p = p * r + 0x1.111112p-7f;
  p = p * r + 0x1.555556p-5f;
  p = p * r + 0x1.555556p-3f;
  p = p * r + 0.5f;
  p = p * r + 1.0f;
  p = p * r + 1.0f;
  return p * __uint_as_float((uint32_t)((int)n + 127) << 23);
}

// Keys order as (value descending, index ascending); 0 is "out".  A value in
// (> -inf) has order bits above those of -inf, so its key is never 0.
__device__ __forceinline__ uint64_t rank_key(float v, int i) {
  return v > -INFINITY ? ((uint64_t)logit_order_bits(v) << 32) | (uint32_t)~i : 0ull;
}

// One wave per token, the experts' values in LDS.
template <int SLOTS>
__global__ __launch_bounds__(64) void gate_kernel(GateLaunch a) {
  __shared__ float sv[64 * SLOTS];
  const int lane = threadIdx.x, t = blockIdx.x;
  const int E = a.E, EG = E / a.n_groups;
  const bool pick_groups = a.top_groups < a.n_groups;
  float z[SLOTS], s[SLOTS];
  bool in[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; i++) {
    const int e = min(lane + 64 * i, E - 1);
    const int64_t at = (int64_t)t * a.z_stride + e;
    z[i] = a.z_dtype == X_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.z)[at])
                               : static_cast<const float*>(a.z)[at];
    in[i] = lane + 64 * i < E && z[i] > -0x1p127f;  // (false for NaN)
    z[i] = in[i] ? fminf(z[i], 3.402823466e38f) : -INFINITY;
  }
  if (a.score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < SLOTS; i++) s[i] = sigmoid32(z[i]);
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) m = fmaxf(m, z[i]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
    float p = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      s[i] = in[i] ? exp32(fmaxf(z[i] - m, -80.0f)) : 0.0f;
      p = p + s[i];
    }
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) p = p + __shfl_down(p, x, 64);
    p = __shfl(p, 0, 64);
#pragma unroll
    for (int i = 0; i < SLOTS; i++) s[i] = s[i] / p;
  }
  float v[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; i++) {
    const int e = min(lane + 64 * i, E - 1);
    v[i] = a.bias ? s[i] + a.bias[e] : (pick_groups && a.group_score == MOE_GROUP_TOP2_SUM ? s[i] : z[i]);
    if (!in[i] || !(v[i] > -INFINITY)) v[i] = -INFINITY;
  }
  if (pick_groups) {
#pragma unroll
    for (int i = 0; i < SLOTS; i++) sv[lane + 64 * i] = v[i];
    __syncthreads();
    float b1 = -INFINITY, b2 = -INFINITY;
    if (lane < a.n_groups)
      for (int i = 0; i < EG; i++) {
        const float x = sv[lane * EG + i];
        b2 = fmaxf(b2, fminf(b1, x));
        b1 = fmaxf(b1, x);
      }
    if (a.group_score == MOE_GROUP_TOP2_SUM && b2 > -INFINITY) b1 = b1 + b2;
    uint64_t key = rank_key(b1, lane), kept = 0;
    for (int r = 0; r < a.top_groups; r++) {
      const uint64_t best = wave_max_u64(key);
      if (best == 0) break;
      kept |= 1ull << (int)~(uint32_t)best;
      if (key == best) key = 0;
    }
#pragma unroll
    for (int i = 0; i < SLOTS; i++)
      if (!(kept >> ((lane + 64 * i) / EG) & 1)) v[i] = -INFINITY;
  }
  uint64_t key[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; i++) key[i] = rank_key(v[i], lane + 64 * i);
  int my_e = -1;
  float my_s = 0.0f, total = 0.0f;
  for (int r = 0; r < a.k; r++) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) best = key[i] > best ? key[i] : best;
    best = wave_max_u64(best);
    if (best == 0) break;
    const int e = (int)~(uint32_t)best;
    float se = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      if (key[i] == best) key[i] = 0;
      if (e >> 6 == i) se = s[i];
    }
    se = __shfl(se, e & 63, 64);
    total = total + se;
    if (lane == r) my_e = e, my_s = se;
  }
  if (lane < a.k) {
    const float w = a.renormalize ? (my_e >= 0 ? my_s / total : 0.0f) : my_s;
    a.idx[(int64_t)t * a.k + lane] = my_e;
    a.wt[(int64_t)t * a.k + lane] = w * a.scale;
  }
}

hipError_t launch_gate(const GateLaunch& a, hipStream_t s) {
  const dim3 grid((unsigned)a.T);
  if (a.E <= 256)
    QMOE_LAUNCH(gate_kernel<4>, grid, dim3(64), 0, s, a);
  else if (a.E <= 512)
    QMOE_LAUNCH(gate_kernel<8>, grid, dim3(64), 0, s, a);
  else
    QMOE_LAUNCH(gate_kernel<16>, grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe
