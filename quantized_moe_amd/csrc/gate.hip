// Gate: scores, groups and top-k of given router logits (definition in
// include/moe.h).  Contraction is off in this file: the fp32 steps of the
// scores decide selections near a tie, so each is rounded on its own.
#include <math.h>

#include <type_traits>

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

// 1 / x correctly rounded for x in [1, 2^117]: the hardware's reciprocal is off
// by one unit at most, and a Newton step with its residual from a fused
// multiply-add leaves the nearest fp32 number (checked for every significand).
// 5 instructions where the general IEEE division takes 10.
__device__ __forceinline__ float recip_exact(float x) {
  float r = __builtin_amdgcn_rcpf(x);
  r = __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
  return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

// The same bits as sigmoid32 (topk.hpp).
__device__ __forceinline__ float sigmoid_score(float z) {
  return recip_exact(1.0f + exp32(-fminf(fmaxf(z, -80.0f), 80.0f)));
}

// Maximum over the wave, the same in every lane.  Lanes that a step's shift
// gives no source keep their value.  (Written out: from the builtins the
// compiler makes a move and a maximum of each step.  A step reads other lanes'
// results of the one before, which takes two wait states.)
__device__ __forceinline__ float wave_fmax(float v) {
  asm("s_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_shr:1 row_mask:0xf bank_mask:0xf\n\ts_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_shr:2 row_mask:0xf bank_mask:0xf\n\ts_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_shr:4 row_mask:0xf bank_mask:0xf\n\ts_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_shr:8 row_mask:0xf bank_mask:0xf\n\ts_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_bcast:15 row_mask:0xa bank_mask:0xf\n\ts_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_bcast:31 row_mask:0xc bank_mask:0xf\n\ts_nop 1"
      : "+v"(v));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// A wave per token, four tokens per block; everything stays in registers.
//
// P = 2^LG lanes hold a group (all 64 the one group when no groups are chosen):
// lane g P + p has experts g EG + p + P i, i < SLOTS, EG = E / groups.  A
// group's two best are then a butterfly over its lanes, its rank a count over
// the groups' values, and an expert that is out is a -inf in its slot.  Each
// round of the top-k takes the wave maximum of the lanes' maxima (6 DPP steps)
// and finds who has it by comparing every slot with it: the comparisons' lane
// masks are scalars, so the lowest index (group, slot, lane) is found by the
// scalar unit beside other waves' vector work.  Only what orders the experts is
// computed for all of them; the chosen ones' scores are taken at the end.
//
// Bound by vector instructions: about 35 a score and 20 a round and token.
template <int SLOTS, int ZDT, int LG>  // LG < 0: any other number of lanes
__global__ __launch_bounds__(256) void gate_kernel(GateLaunch a, int lg_) {
  __shared__ float terms[4][64 * 16];  // softmax terms of grouped experts, for their sum's order
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(wave);
  if (t >= a.T) return;
  const int lg = LG < 0 ? lg_ : LG;
  const bool pick_groups = LG == 6 ? false : a.top_groups < a.n_groups;
  const int G = pick_groups ? a.n_groups : 1, EG = a.E / G, P = 1 << lg;
  const int g = lane >> lg, p = lane & (P - 1), e0 = g * EG + p;
  const bool top2 = pick_groups && a.group_score == MOE_GROUP_TOP2_SUM;

  // slots that exist: i < n_own (unsigned offsets from a uniform row pointer)
  const int n_own = g < G && p < EG ? (EG - p + P - 1) >> lg : 0;
  using Z = typename std::conditional<ZDT == X_BF16, uint16_t, float>::type;
  const Z* zrow = static_cast<const Z*>(a.z) + (int64_t)t * a.z_stride;
  const uint32_t at = n_own > 0 ? e0 : 0;
  float z[SLOTS], bias[SLOTS] = {};
#pragma unroll
  for (int i = 0; i < SLOTS; i++) {
    const Z v = zrow[i < n_own ? at + P * i : at];
    if constexpr (ZDT == X_BF16)
      z[i] = bf16_bits_to_float(v);
    else
      z[i] = v;
  }
  if (a.bias) {  // (requested with the logits: one wait)
#pragma unroll
    for (int i = 0; i < SLOTS; i++) bias[i] = a.bias[i < n_own ? at + P * i : at];
  }
#pragma unroll
  for (int i = 0; i < SLOTS; i++)  // (false for NaN)
    z[i] = i < n_own && z[i] > -0x1p127f ? fminf(z[i], 3.402823466e38f) : -INFINITY;

  float m = 0.0f, total = 1.0f;  // softmax: the largest logit, the sum of the terms
  if (a.score == MOE_SCORE_SOFTMAX) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) m = fmaxf(m, z[i]);
    m = wave_fmax(m);
  }
  // a masked expert's term is 0 and its -inf stays
  auto term = [&](float x) { return x > -INFINITY ? exp32(fmaxf(x - m, -80.0f)) : 0.0f; };
  float v[SLOTS];
  if (a.score == MOE_SCORE_SOFTMAX) {
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = term(z[i]);
    if (pick_groups) {  // partial e % 64 is another lane's
#pragma unroll
      for (int i = 0; i < SLOTS; i++)
        if (i < n_own) terms[wave][e0 + P * i] = v[i];
      __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations are in order)
      for (int e = lane; e < a.E; e += 64) part = part + terms[wave][e];
    } else {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) part = part + v[i];
    }
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) part = part + __shfl_xor(part, s, 64);
    total = part;
  }
  if (a.bias || top2) {
    if (a.score == MOE_SCORE_SIGMOID) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) v[i] = sigmoid_score(z[i]);
    } else {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) v[i] = v[i] / total;
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) v[i] = v[i] + bias[i];
    }
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = z[i] > -INFINITY && v[i] > -INFINITY ? v[i] : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = z[i];
  }

  if (pick_groups) {
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      b2 = fmaxf(b2, fminf(b1, v[i]));
      b1 = fmaxf(b1, v[i]);
    }
    for (int s = 1; s < P; s <<= 1) {
      const float c1 = __shfl_xor(b1, s, 64), c2 = __shfl_xor(b2, s, 64);
      b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
      b1 = fmaxf(b1, c1);
    }
    if (top2 && b2 > -INFINITY) b1 = b1 + b2;
    int before = 0;  // groups that come before this lane's
    for (int h = 0; h < G; h++) {
      const float c = read_lane(b1, h << lg);
      before += h < g ? c >= b1 : c > b1;
    }
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = before < a.top_groups ? v[i] : -INFINITY;
  }

  int my_e = -1;
  float my_z = -INFINITY;
  for (int r = 0; r < a.k; r++) {
    float b = v[0];
#pragma unroll
    for (int i = 1; i < SLOTS; i++) b = fmaxf(b, v[i]);
    b = wave_fmax(b);
    if (!(b > -INFINITY)) break;
    uint64_t has[SLOTS], any = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      has[i] = __ballot(v[i] == b);  // (-0 == +0)
      any |= has[i];
    }
    const int first = __builtin_ctzll(any) >> lg;  // the lowest group
    const uint64_t lanes = (lg == 6 ? ~0ull : (1ull << P) - 1) << (first << lg);
    int slot = 0;
    uint64_t in_slot = 0;
#pragma unroll
    for (int i = SLOTS - 1; i >= 0; i--)
      if (has[i] & lanes) {
        slot = i;
        in_slot = has[i] & lanes;
      }
    const int l = __builtin_ctzll(in_slot);
    const int e = first * EG + (l & (P - 1)) + P * slot;
    float ze = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; i++)
      if (slot == i) {
        ze = read_lane(z[i], l);
        v[i] = lane == l ? -INFINITY : v[i];
      }
    if (lane == r) {
      my_e = e;
      my_z = ze;
    }
  }
  const float chosen = a.score == MOE_SCORE_SIGMOID ? sigmoid_score(my_z) : term(my_z) / total;
  const float s = my_e >= 0 ? chosen : 0.0f;
  float sum = 0.0f;
  for (int r = 0; r < a.k; r++) sum = sum + read_lane(s, r);
  if (lane < a.k) {
    const float w = a.renormalize && my_e >= 0 ? s / sum : s;
    a.idx[(int64_t)t * a.k + lane] = my_e;
    a.wt[(int64_t)t * a.k + lane] = w * a.scale;
  }
}

template <int SLOTS, int LG>
static void launch_slots(const GateLaunch& a, int lg, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 3) / 4));
  if (a.z_dtype == X_BF16)
    QMOE_LAUNCH((gate_kernel<SLOTS, X_BF16, LG>), grid, dim3(256), 0, s, a, lg);
  else
    QMOE_LAUNCH((gate_kernel<SLOTS, X_F32, LG>), grid, dim3(256), 0, s, a, lg);
}

template <int LG>
static void launch_lanes(const GateLaunch& a, int lg, int slots, hipStream_t s) {
  if (slots <= 4) return launch_slots<4, LG>(a, lg, s);
  if (slots <= 6) return launch_slots<6, LG>(a, lg, s);
  if (slots <= 8) return launch_slots<8, LG>(a, lg, s);
  if (slots <= 16) return launch_slots<16, LG>(a, lg, s);
  if constexpr (LG < 0) launch_slots<32, LG>(a, lg, s);
}

hipError_t launch_gate(const GateLaunch& a, hipStream_t s) {
  const int G = a.top_groups < a.n_groups ? a.n_groups : 1;
  int lg = 6;
  while ((G << lg) > 64) lg--;
  const int slots = (a.E / G + (1 << lg) - 1) >> lg;  // at most 16 for powers of two, 32 for other G
  if (lg == 6)  // no groups: the lanes' offsets are constants
    launch_lanes<6>(a, lg, slots, s);
  else
    launch_lanes<-1>(a, lg, slots, s);
  return hipGetLastError();
}

}  // namespace qmoe
