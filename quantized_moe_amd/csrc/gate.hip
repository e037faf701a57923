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
  return __builtin_amdgcn_ldexpf(p, (int)n);  // p 2^n, a normal number
}

// Maxima and minima of numbers (the compiler, which must allow for signalling
// NaNs, puts a quieting instruction before each operand).
__device__ __forceinline__ float vmax(float a, float b) {
  float d;
  asm("v_max_f32 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
__device__ __forceinline__ float vmin(float a, float b) {
  float d;
  asm("v_min_f32 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
__device__ __forceinline__ float vmax3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
template <int N>
__device__ __forceinline__ float max_of(const float (&v)[N]) {
  float b = v[0];
  int i = 1;
#pragma unroll
  for (; i + 1 < N; i += 2) b = vmax3(b, v[i], v[i + 1]);
  return i < N ? vmax(b, v[N - 1]) : b;
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
  return recip_exact(1.0f + exp32(-__builtin_amdgcn_fmed3f(z, -80.0f, 80.0f)));
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
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int b = (int)__float_as_uint(v);
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(b, b, CTRL, 0xf, 0xf, false));
}
// The fold of 64 partials, p[l] = p[l] + p[l + s] for s = 32 .. 1, in every
// lane: additions commute, so lanes l and l ^ s may both take the step's sum,
// and once lanes equal modulo 2 s agree, a rotation by s within 16 serves.
__device__ __forceinline__ float fold64(float p) {
  const uint32_t b = __float_as_uint(p);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);  // lanes l & 31 and l | 32
  const uint32_t c = __float_as_uint(__uint_as_float(h[0]) + __uint_as_float(h[1]));
  const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  p = __uint_as_float(q[0]) + __uint_as_float(q[1]);
  p = p + dpp<0x128>(p);  // row_ror 8
  p = p + dpp<0x124>(p);  // row_ror 4
  p = p + dpp<0x122>(p);  // row_ror 2
  return p + dpp<0x121>(p);
}
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ bool in_lanes(uint64_t mask) { return __builtin_amdgcn_inverse_ballot_w64(mask); }

// A wave per token, four tokens per block; everything stays in registers.
//
// P = 2^LG lanes hold a group (all 64 the one group when no groups are chosen):
// lane g P + p has experts g EG + p + P i, i < SLOTS, EG = E / groups.  A
// group's two best are then a butterfly over its lanes, its rank a count over
// the groups' values, and an expert that is out is a -inf in its slot.  Each
// round of the top-k takes the wave maximum of the lanes' maxima (6 DPP steps)
// and compares every slot with it.  Nearly always one slot of one lane has it:
// the comparisons' lane masks, which are scalars, show that, clear the slot and
// name the lane; which slot it was, lane r finds for round r at the end, all
// rounds at once.  Equal values take the scalar search for the lowest index
// (group, slot, lane).  Only what orders the experts is computed for all of
// them; the chosen ones' scores are taken at the end.
//
// Bound by vector instructions: about 30 a score and 25 a round and token.
// Measured: 65536 tokens, 384 experts in 8 groups with a bias 59 us (100 MB of
// logits: 21 us at a large copy's rate), 1 token 4.6 us.
//
// FULL: every lane has an expert in every slot.
template <int SLOTS, int ZDT, int LG, bool FULL>  // LG < 0: any other number of lanes
__global__ __launch_bounds__(256) void gate_kernel(GateLaunch a, int lg_, int groups, int group_experts) {
  __shared__ float terms[4][64 * 16];  // softmax terms of grouped experts, for their sum's order
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  const int lg = LG < 0 ? lg_ : LG;
  const bool pick_groups = LG != 6;
  const int G = LG == 6 ? 1 : groups, EG = group_experts, P = 1 << lg;
  const int g = lane >> lg, p = lane & (P - 1), e0 = g * EG + p;
  const bool top2 = pick_groups && a.group_score == MOE_GROUP_TOP2_SUM;
  // slots that exist: i < n_own (unsigned offsets from a uniform row pointer)
  const int n_own = FULL ? SLOTS : g < G && p < EG ? (EG - p + P - 1) >> lg : 0;
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
    z[i] = i < n_own && z[i] > -0x1p127f ? vmin(z[i], 3.402823466e38f) : -INFINITY;

  float m = 0.0f, total = 1.0f;  // softmax: the largest logit, the sum of the terms
  // a masked expert's term is 0 and its -inf stays
  auto term = [&](float x) {
    const float e = exp32(vmax(x - m, -80.0f));  // (finite whatever x is)
    return x > -INFINITY ? e : 0.0f;
  };
  float v[SLOTS];
  if (a.score == MOE_SCORE_SOFTMAX) {
    m = wave_fmax(max_of(z));
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
    total = fold64(part);
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
      for (int i = 0; i < SLOTS; i++) v[i] = vmax(v[i] + bias[i], -INFINITY);  // (NaN to -inf)
    }
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = z[i] > -INFINITY ? v[i] : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = z[i];
  }

  if (pick_groups) {
    float b1 = v[0], b2 = -INFINITY;
#pragma unroll
    for (int i = 1; i < SLOTS; i++) {
      b2 = vmax(b2, vmin(b1, v[i]));
      b1 = vmax(b1, v[i]);
    }
    auto merge = [&](float c1, float c2) {  // with another lane's two best
      b2 = vmax3(b2, c2, vmin(b1, c1));
      b1 = vmax(b1, c1);
    };
    if constexpr (LG == 3) {
      merge(dpp<0xb1>(b1), dpp<0xb1>(b2));    // quad_perm 1 0 3 2
      merge(dpp<0x4e>(b1), dpp<0x4e>(b2));    // quad_perm 2 3 0 1
      merge(dpp<0x141>(b1), dpp<0x141>(b2));  // row_half_mirror: the other quad
    } else {
      for (int s = 1; s < P; s <<= 1) merge(__shfl_xor(b1, s, 64), __shfl_xor(b2, s, 64));
    }
    if (top2 && b2 > -INFINITY) b1 = b1 + b2;
    int before = 0;  // groups that come before this lane's
    for (int h = 0; h < G; h++) {
      const float c = read_lane(b1, h << lg);
      const int later = (h + 1) << lg;  // lanes of the groups after h: an equal value comes before theirs
      const uint64_t tied = later < 64 ? __ballot(c >= b1) & (~0ull << later) : 0;
      before += in_lanes(tied | __ballot(c > b1));
    }
#pragma unroll
    for (int i = 0; i < SLOTS; i++) v[i] = before < a.top_groups ? v[i] : -INFINITY;
  }

  float left[SLOTS];  // v without the chosen
#pragma unroll
  for (int i = 0; i < SLOTS; i++) left[i] = v[i];
  int my_lane = -1, my_slot = -1;  // round `lane`'s expert, the slot if it is known
  float my_v = 0.0f;
  // a value was there twice: what is left of it is no sign of its slot any more
  // (bf16 logits often are: they are searched without looking)
  bool equals = ZDT == X_BF16;
  for (int r = 0; r < a.k; r++) {
    const float b = wave_fmax(max_of(left));
    if (__float_as_uint(b) == 0xff800000u) break;  // (never NaN)
    uint64_t has[SLOTS], any = 0, twice = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      has[i] = __ballot(left[i] == b);  // (-0 == +0)
      twice |= any & has[i];
      any |= has[i];
    }
    int l = __builtin_ctzll(any);
    const bool mine = in_lanes(1ull << r);
    equals |= twice != 0 || (any & (any - 1)) != 0;
    if (!equals) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) left[i] = in_lanes(has[i]) ? -INFINITY : left[i];
    } else {
      const int first = l >> lg;  // the lowest group
      const uint64_t lanes = (~0ull >> (64 - P)) << (first << lg);
      uint64_t in_slot = 0;
      int slot = 0;
#pragma unroll
      for (int i = SLOTS - 1; i >= 0; i--)
        if (has[i] & lanes) {
          slot = i;
          in_slot = has[i] & lanes;
        }
      l = __builtin_ctzll(in_slot);
#pragma unroll
      for (int i = 0; i < SLOTS; i++) left[i] = slot == i && lane == l ? -INFINITY : left[i];
      my_slot = mine ? slot : my_slot;
    }
    my_lane = mine ? l : my_lane;
    my_v = mine ? b : my_v;
  }
  // The slot (where it was the only one with that value) and the logit.
  float my_z = -INFINITY;
  const int from = my_lane < 0 ? lane : my_lane;
#pragma unroll
  for (int i = 0; i < SLOTS; i++) {
    const float vi = __shfl(v[i], from, 64), zi = __shfl(z[i], from, 64);
    const bool is = my_slot < 0 ? vi == my_v : my_slot == i;
    if (is && my_lane >= 0) {
      my_slot = i;
      my_z = zi;
    }
  }
  const int my_e = my_lane < 0 ? -1 : (my_lane >> lg) * EG + (my_lane & (P - 1)) + P * my_slot;
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

template <int SLOTS, int LG, bool FULL>
static void launch_slots(const GateLaunch& a, int lg, int G, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 3) / 4));
  if (a.z_dtype == X_BF16)
    QMOE_LAUNCH((gate_kernel<SLOTS, X_BF16, LG, FULL>), grid, dim3(256), 0, s, a, lg, G, a.E / G);
  else
    QMOE_LAUNCH((gate_kernel<SLOTS, X_F32, LG, FULL>), grid, dim3(256), 0, s, a, lg, G, a.E / G);
}

// LG: all lanes one group (their offsets are constants), or 8 for each of up to
// 8 groups, or any other number.
template <int LG>
static void launch_lanes(const GateLaunch& a, int lg, int G, hipStream_t s) {
  const int EG = a.E / G, slots = (EG + (1 << lg) - 1) >> lg;  // at most 16 for powers of two, 32 for other G
  const bool full = (G << lg) == 64 && (EG & ((1 << lg) - 1)) == 0;
  if constexpr (LG >= 0) {
    if (full && slots == 4) return launch_slots<4, LG, true>(a, lg, G, s);
    if (full && slots == 6) return launch_slots<6, LG, true>(a, lg, G, s);
  }
  if (slots <= 4) return launch_slots<4, LG, false>(a, lg, G, s);
  if (slots <= 6) return launch_slots<6, LG, false>(a, lg, G, s);
  if (slots <= 8) return launch_slots<8, LG, false>(a, lg, G, s);
  if (slots <= 16) return launch_slots<16, LG, false>(a, lg, G, s);
  if constexpr (LG != 6) launch_slots<32, LG, false>(a, lg, G, s);
}

hipError_t launch_gate(const GateLaunch& a, hipStream_t s) {
  const int G = a.top_groups < a.n_groups ? a.n_groups : 1;
  int lg = 6;
  while ((G << lg) > 64) lg--;
  if (lg == 6)
    launch_lanes<6>(a, lg, G, s);
  else if (lg == 3)
    launch_lanes<3>(a, lg, G, s);
  else
    launch_lanes<-1>(a, lg, G, s);
  return hipGetLastError();
}

}  // namespace qmoe
