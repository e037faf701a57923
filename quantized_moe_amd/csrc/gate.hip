// Gate: scores, groups and top-k of given router logits (definition in
// include/moe.h).  Contraction is off in this file: the fp32 steps of the
// scores decide selections near a tie, so each is rounded on its own.
#include <math.h>

#include <type_traits>
#include <utility>

#include "common.hpp"
#include "kernels.hpp"
#include "topk.hpp"

#pragma clang fp contract(off)

namespace qmoe {

// e^t for t in [-80, 80]: the steps of sigmoid32 (include/moe.h).  Two of them
// in fewer instructions with the same bits: n ln2_hi has 22 bits at most, so a
// fused multiply-add rounds as the product and the difference do; and the sum
// with 1.5 2^23 ends in n, which is added to p's exponent (p 2^n is normal).
__device__ __forceinline__ float exp32(float t) {
  const float kf = t * 0x1.715476p+0f;
  const float shifted = kf + 0x1.8p+23f, n = shifted - 0x1.8p+23f;
  const float r = __builtin_fmaf(-n, 0x1.62e400p-1f, t) - n * 0x1.7f7d1cp-20f;
  float p = 0x1.6c16c2p-10f;
  p = p * r + 0x1.111112p-7f;
  p = p * r + 0x1.555556p-5f;
  p = p * r + 0x1.555556p-3f;
  p = p * r + 0.5f;
  p = p * r + 1.0f;
  p = p * r + 1.0f;
  return __uint_as_float((__float_as_uint(shifted) << 23) + __float_as_uint(p));
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
__device__ __forceinline__ float vmed3(float a, float b, float c) {
  float d;
  asm("v_med3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
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
// by one unit at most, and two Newton steps with residuals from fused
// multiply-adds leave the nearest fp32 number from any such start (tested on the
// CPU for every significand), but for x = 2 - 2^-23, whose start has to be the
// nearest and is (tested on the GPU: the score of every logit, bit for bit).
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

// sigmoid_score within 2^-21: four instructions (two of them at a quarter of
// the rate) where the exact steps take some 26.  Its argument's rounding moves
// it by |z| s (1 - s) 2^-23 <= 2^-25, the exponential by s (1 - s) 2^-23, the
// sum and the reciprocal by 2^-24 and 2^-23; the exact steps err by less than
// 2^-22.
__device__ __forceinline__ float sigmoid_near(float z) {
  float s;  // (written out with the wait that other written-out instructions need after a reciprocal)
  asm("v_rcp_f32 %0, %1\n\ts_nop 0" : "=v"(s) : "v"(1.0f + __builtin_amdgcn_exp2f(z * -0x1.715476p+0f)));
  return s;
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

// f(0), f(1), ... as constants, until one is false.
template <class F, int... R>
__device__ __forceinline__ void each_until(F&& f, std::integer_sequence<int, R...>) {
  (void)(f(std::integral_constant<int, R>{}) && ...);
}

// A wave per token, four tokens per block; everything stays in registers.
//
// P = 2^LG lanes hold a group (all 64 the one group when no groups are chosen):
// lane g P + p has experts g EG + p + P i, i < SLOTS, EG = E / groups.  A
// group's two best are then a butterfly over its lanes, its rank a count over
// the groups' values, and an expert that is out is a -inf in its slot.
//
// Only what orders the experts is computed for all of them, and that first to
// within a known error: a sigmoid in 4 instructions for the exact steps' 26, and
// the value's lowest bits give way to its slot's number, so that a lane's values
// are distinct and can be sorted.  If the groups that are kept and the best k + 1
// values lie further apart than the errors, this is the exact scores' order; if
// not (one token of some hundred), the token is done again with exact values.
// The chosen experts' scores are always the exact steps'.
//
// Bound by vector instructions, 380 a token at 384 experts (100 in the 7 rounds,
// 42 the scores, 24 the exact scores of the chosen).  Measured: 65536 tokens, 384
// experts in 8 groups with a bias 43 us (60 us with exact values throughout; 100
// MB of logits take 21 us at a large copy's rate); 1 token 3.1 us.
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
  float z[SLOTS], bias[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; i++) {
    const Z v = FULL ? zrow[at + (int64_t)(P * i)] : zrow[i < n_own ? at + P * i : at];
    if constexpr (ZDT == X_BF16)
      z[i] = bf16_bits_to_float(v);
    else
      z[i] = v;
  }
  if (a.bias) {  // (requested with the logits: one wait)
#pragma unroll
    for (int i = 0; i < SLOTS; i++) bias[i] = FULL ? a.bias[at + (int64_t)(P * i)] : a.bias[i < n_own ? at + P * i : at];
  }
#pragma unroll
  for (int i = 0; i < SLOTS; i++)  // (false for NaN)
    z[i] = i < n_own && z[i] > -0x1p127f ? z[i] : -INFINITY;
  const bool plain = !(a.bias || top2);  // the values are the logits
  if (plain || a.score == MOE_SCORE_SOFTMAX) {  // (sigmoid scores are the same)
#pragma unroll
    for (int i = 0; i < SLOTS; i++) z[i] = vmin(z[i], 3.402823466e38f);
  }

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
  int my_lane = -1, my_slot = -1;  // round `lane`'s expert
  float my_v;
  // (b1, b2), a lane's two best, to those of its group
  auto merge_lanes = [&](float& b1, float& b2) __attribute__((always_inline)) {
    if constexpr (LG == 3) {
      float t;
#define QMOE_MERGE(STEP)                                                                                           \
  asm("s_nop 1\n\tv_min_f32_dpp %0, %1, %1 " STEP " row_mask:0xf bank_mask:0xf\n\t"                                 \
      "v_max_f32_dpp %1, %1, %1 " STEP " row_mask:0xf bank_mask:0xf\n\t"                                           \
      "v_max_f32_dpp %2, %2, %2 " STEP " row_mask:0xf bank_mask:0xf"                                               \
      : "=&v"(t), "+v"(b1), "+v"(b2));                                                                             \
  b2 = vmax(b2, t);
      QMOE_MERGE("quad_perm:[1,0,3,2]")
      QMOE_MERGE("quad_perm:[2,3,0,1]")
      QMOE_MERGE("row_half_mirror")  // the other quad
#undef QMOE_MERGE
    } else {
      for (int s = 1; s < P; s <<= 1) {
        const float c1 = __shfl_xor(b1, s, 64), c2 = __shfl_xor(b2, s, 64);
        b2 = vmax3(b2, c2, vmin(b1, c1));
        b1 = vmax(b1, c1);
      }
    }
  };
  // Keys within near_err of the values, their lowest bits the slot: distinct in
  // a lane, whose QUEUE largest are sorted once, so that a round is the wave
  // maximum of the lanes' first and a step of one lane's queue.  False if the
  // keys do not decide the order, or a lane's queue runs out.
  // bf16 logits that are the values themselves have room for the expert's number
  // (the lower first of equal ones): such keys are the exact order.
  constexpr int SB = SLOTS <= 4 ? 4 : SLOTS <= 8 ? 8 : SLOTS <= 16 ? 16 : 32;  // slot numbers
  constexpr int QUEUE = 4;
  static_assert(SLOTS >= QUEUE, "every place is filled");
  // 2^-21 of a score, (SB + 1) 2^-23 |v| of its sum's rounding and the slot's
  // bits; a number also for -inf
  auto near_err = [](float x) {
    return (SB <= 16 ? 0x1p-18f : 0x1p-17f) * vmin(vmax(__builtin_fabsf(x), 1.0f), 3.402823466e38f);
  };
  const bool ordered = ZDT == X_BF16 && plain;
  auto select_near = [&]() __attribute__((always_inline)) -> bool {
    float key[SLOTS], q[QUEUE];
    if (plain) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) key[i] = z[i];
    } else {
      if (a.score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < SLOTS; i++) key[i] = sigmoid_near(z[i]);
      } else {
        const float r = __builtin_amdgcn_rcpf(total);
#pragma unroll
        for (int i = 0; i < SLOTS; i++) key[i] = v[i] * r;
      }
      if (a.bias) {  // (NaN to -inf)
#pragma unroll
        for (int i = 0; i < SLOTS; i++) key[i] = vmed3(key[i] + bias[i], -INFINITY, 3.402823466e38f);
      }
    }
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      const bool in = vmin(key[i], z[i]) > -INFINITY;
      uint32_t b = __float_as_uint(key[i]);
      if (ordered) {
        b = __float_as_uint(key[i] + 0.0f);  // (-0 is 0)
        const uint32_t e = e0 + P * i;
        b = (b & ~1023u) | ((int)b < 0 ? e : 1023u - e);
      } else {
        b = (b & ~(SB - 1u)) | i;
      }
      key[i] = in ? __uint_as_float(b) : -INFINITY;
    }
    q[0] = key[0];
#pragma unroll
    for (int j = 1; j < QUEUE; j++) q[j] = -INFINITY;
#pragma unroll
    for (int i = 1; i < SLOTS; i++) {  // into its place of the sorted queue
#pragma unroll
      for (int j = min(i, QUEUE - 1); j > 0; j--) q[j] = j == i ? vmin(q[j - 1], key[i]) : vmed3(q[j - 1], q[j], key[i]);
      q[0] = vmax(q[0], key[i]);
    }
    if (pick_groups) {
      float b1 = q[0], b2 = QUEUE > 1 ? q[1] : -INFINITY;
      merge_lanes(b1, b2);
      float err = ordered ? 0.0f : near_err(b1);
      if (top2 && b2 > -INFINITY) {
        err = err + near_err(b2);
        b1 = b1 + b2;
      }
      const float most = b1 + err, least = b1 - err;
      int before = -1;  // groups that may come before this lane's (not itself)
      if constexpr (LG == 3) {  // each of a group's 8 lanes compares it with another one
        const uint64_t m = __ballot(__shfl(most, p << 3, 64) >= least);
        before += __builtin_popcount((uint32_t)(m >> (g << 3)) & 0xffu);
      } else {
        for (int h = 0; h < G; h++) before += in_lanes(__ballot(read_lane(most, h << lg) >= least));
      }
      const bool kept = before < a.top_groups;
      if (!ordered && __popcll(__ballot(kept)) != a.top_groups << lg) return false;
#pragma unroll
      for (int j = 0; j < QUEUE; j++) q[j] = kept ? q[j] : -INFINITY;
    }
    my_lane = my_slot = -1;
    my_v = -INFINITY;
    uint64_t taken[QUEUE + 1] = {};  // lanes that have given that many
    const int rounds = ordered ? a.k : a.k + 1;
    bool decided = true;
    auto round = [&](auto rc) __attribute__((always_inline)) -> bool {
      constexpr int r = decltype(rc)::value;
      if (r >= rounds) return false;
      const uint32_t b = __float_as_uint(wave_fmax(q[0]));
      if (b == 0xff800000u) return false;
      const uint64_t has = __ballot(__float_as_uint(q[0]) == b);
      uint64_t not_one = has & (has - 1);
      if constexpr (SLOTS > QUEUE) {
        not_one |= taken[QUEUE - 1] & has;
#pragma unroll
        for (int j = QUEUE - 1; j > 0; j--) taken[j] |= j == 1 ? has : taken[j - 1] & has;
      }
      decided = not_one == 0;
      if (!decided) return false;
      // (two wait states from a comparison or a read lane to these)
      asm("s_nop 1\n\t"
          "v_cndmask_b32 %0, %0, %1, %6\n\tv_cndmask_b32 %1, %1, %2, %6\n\t"
          "v_cndmask_b32 %2, %2, %3, %6\n\tv_cndmask_b32 %3, %3, %9, %6\n\t"
          "v_writelane_b32 %4, %7, %8\n\tv_writelane_b32 %5, %10, %8"
          : "+&v"(q[0]), "+&v"(q[1]), "+&v"(q[2]), "+&v"(q[3]), "+v"(my_v), "+v"(my_lane)
          : "s"(has), "s"(b), "n"(r), "v"(-INFINITY), "s"((int)__builtin_ctzll(has)));
      return true;
    };
    each_until(round, std::make_integer_sequence<int, TOPK_MAX_K + 1>{});
    if (!decided) return false;
    if (ordered) {
      const uint32_t b = __float_as_uint(my_v) & 1023u;
      const int e = (int)__float_as_uint(my_v) < 0 ? b : 1023u - b;
      my_slot = (e - (my_lane >> lg) * EG) >> lg;
    } else {
      const float next = __shfl_down(my_v, 1, 64);  // each of the k against the next
      const bool apart = my_lane < 0 || my_v - next > near_err(my_v) + near_err(next);
      if (__ballot(lane < a.k && !apart)) return false;
      my_slot = __float_as_uint(my_v) & (SB - 1u);
    }
    return true;
  };
  // Any values: each round compares every slot with the wave's largest.  Nearly
  // always one slot of one lane has it: the comparisons' lane masks, which are
  // scalars, show that, clear the slot and name the lane; which slot it was, lane
  // r finds for round r at the end, all rounds at once.  Equal values take the
  // scalar search for the lowest index (group, slot, lane).
  auto select_any = [&]() __attribute__((always_inline)) {
    if (!plain) {
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
      merge_lanes(b1, b2);
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
    my_lane = my_slot = -1;
    my_v = -INFINITY;
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
    const int from = my_lane < 0 ? lane : my_lane;
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      const float vi = __shfl(v[i], from, 64);
      if (my_slot < 0 && my_lane >= 0 && vi == my_v) my_slot = i;
    }
  };
  // Queues do not last where fewer lanes are left than rounds: 32768 tokens, 16 of
  // 1024 experts in one of 8 groups 96 us without and 119 us with them; 16 of 512
  // in one of 4 groups (16 lanes) 57 and 55 us, 8 of 384 in 2 of 8 groups 31 and
  // 23 us, 6 of 384 by bf16 logits' sums, where ties are common, 38 and 32 us.
  const int lanes_kept = (pick_groups ? a.top_groups : 1) << lg;
  const bool try_near = SLOTS <= QUEUE || a.k <= lanes_kept;
  if (!try_near || !select_near()) select_any();
  float my_z = -INFINITY;
  const int from = my_lane < 0 ? lane : my_lane;
#pragma unroll
  for (int i = 0; i < SLOTS; i++) {
    const float zi = __shfl(z[i], from, 64);
    my_z = my_slot == i ? zi : my_z;
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
