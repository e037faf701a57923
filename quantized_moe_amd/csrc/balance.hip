// The router's balance: tokens and routes per expert of each sequence, the
// balance loss, and its gradient with respect to the logits.
//
// loss_s = alpha E / (k n_s^2) sum_t q_t with q_t = sum_e c_se p_te: the counts
// c_se come from the routes alone, so no column sum of probabilities over the
// tokens is ever kept; every token gives one number, and the gradient
//   dz_te = g_s alpha E / (k n_s^2) p_te (c_se - q_t)   (sigmoid: (1 - sigma_te) times that)
// needs the token's own row again and nothing else.  Bound by the logits' bytes.
#include "blockscale.hpp"

namespace qmoe {

namespace {

// The sequence of token t: the last of the S + 1 starts that is <= t (none: -1;
// the last start: S).  A wave looks at 64 places at a time.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int S, int t) {
  if (!starts) return 0;
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S + 1;  // starts[lo - 1] <= t < starts[lo + n]
  while (n > 0) {
    const int step = (n + 63) / 64, at = lane * step + step - 1;
    const bool below = at < n && starts[lo + at] <= t;
    const int c = __popcll(__ballot(below));  // whole steps at or below t
    lo += c * step;
    n = step == 1 ? 0 : min(step - 1, n - c * step);
  }
  return lo - 1;
}

// Tokens [first, end) of sequence s, inside [0, T).
__device__ __forceinline__ int bound_of(const int32_t* starts, int i, int T) {
  return starts ? min(max(starts[i], 0), T) : i == 0 ? 0 : T;
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f<0xb1>(v));
  v = fmaxf(v, dpp_f<0x4e>(v));
  v = fmaxf(v, dpp_f<0x141>(v));
  v = fmaxf(v, dpp_f<0x140>(v));
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<0xb1>(v);
  v += dpp_f<0x4e>(v);
  v += dpp_f<0x141>(v);
  v += dpp_f<0x140>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

constexpr float LOG2E = 1.4426950408889634f;

// One token in one wave, PER logits a lane (expert i * 64 + lane).  a = the
// scores (0: the expert is out), u = 1 - sigma of the sigmoid; sum = their sum,
// dot = sum c a.  false: no expert is in.
template <int PER>
struct TokenRow {
  float a[PER], u[PER];
  float sum, dot;
  template <int ZDT>
  __device__ __forceinline__ void load(const void* z, int64_t at, int E) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int e = i * 64 + lane;
      a[i] = -INFINITY;
      if (e < E)
        a[i] = ZDT == X_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(z)[at + e]) : static_cast<const float*>(z)[at + e];
    }
  }
  template <bool SOFTMAX>
  __device__ __forceinline__ void scores(const float (&c)[PER]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      // (a comparison that NaN fails; infinities count as the largest number)
      a[i] = a[i] > -0x1p127f ? fminf(a[i], 0x1.fffffep127f) : -INFINITY;
    }
    if (SOFTMAX) {
      m = a[0];
#pragma unroll
      for (int i = 1; i < PER; i++) m = fmaxf(m, a[i]);
      m = fmaxf(wave_max(m), -0x1p127f);  // (no expert in: every score is 0)
    }
    sum = 0.0f;
    dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      if (SOFTMAX) {
        a[i] = __builtin_amdgcn_exp2f((a[i] - m) * LOG2E);
      } else {
        const bool in = a[i] >= -0x1p127f;
        const float e = __builtin_amdgcn_exp2f(fminf(fmaxf(a[i], -80.0f), 80.0f) * -LOG2E);
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        a[i] = in ? s : 0.0f;
        u[i] = e * s;
      }
      sum += a[i];
      dot = __builtin_fmaf(c[i], a[i], dot);
    }
    sum = wave_sum(sum);
    dot = wave_sum(dot);
  }
  // sum_e c_e p_e
  __device__ __forceinline__ float share() const { return sum > 0.0f ? dot / sum : 0.0f; }
};

// Whether token t has a route.
__device__ __forceinline__ bool has_route(const int32_t* idx, int64_t t, int k, int E) {
  const int lane = threadIdx.x & 63;
  return __ballot(lane < k && (uint32_t)idx[t * k + min(lane, k - 1)] < (uint32_t)E) != 0;
}

}  // namespace

__global__ __launch_bounds__(256) void balance_clear_kernel(int32_t* counts, int64_t n, int32_t* tokens, int S) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) counts[i] = 0;
  if (i < S) tokens[i] = 0;
}

// 1024 tokens a block.  The counts of the block's first `held` sequences are
// added in LDS and then to memory; routes of later ones go to memory directly.
// Whole numbers: the order of the atomics changes nothing.
constexpr int COUNT_TOKENS = 1024, COUNT_HELD = 12288;
__global__ __launch_bounds__(1024) void balance_count_kernel(const int32_t* __restrict__ idx, int T, int k, int E,
                                                             const int32_t* __restrict__ starts, int S,
                                                             int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  __shared__ int hist[COUNT_HELD];
  __shared__ int live[COUNT_HELD / 8];  // (of E >= 8; fewer experts hold as many sequences as 8 would)
  const int t0 = blockIdx.x * COUNT_TOKENS, t1 = min(t0 + COUNT_TOKENS, T) - 1, t = t0 + threadIdx.x;
  const int s0 = max(sequence_of(starts, S, t0), 0), s1 = min(sequence_of(starts, S, t1), S - 1);
  const int held = min(COUNT_HELD / max(E, 8), s1 - s0 + 1);  // (<= 0: no token of any sequence)
  for (int i = threadIdx.x; i < held * E; i += 1024) hist[i] = 0;
  for (int i = threadIdx.x; i < held; i += 1024) live[i] = 0;
  __syncthreads();
  if (t <= t1 && s1 >= s0) {
    int s = 0;
    if (starts) {  // the last start of [s0, s1 + 1] that is <= t
      int lo = s0, hi = s1 + 2;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] <= t)
          lo = mid + 1;
        else
          hi = mid;
      }
      s = lo - 1;
    }
    if (s >= s0 && s <= s1) {
      bool any = false;
      for (int j = 0; j < k; j++) {
        const int e = idx[(int64_t)t * k + j];
        if ((uint32_t)e >= (uint32_t)E) continue;
        any = true;
        if (s - s0 < held)
          atomicAdd(&hist[(s - s0) * E + e], 1);
        else
          atomicAdd(&counts[(int64_t)s * E + e], 1);
      }
      if (any) atomicAdd(s - s0 < held ? &live[s - s0] : &tokens[s], 1);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < held * E; i += 1024)
    if (hist[i]) atomicAdd(&counts[(int64_t)s0 * E + i], hist[i]);
  for (int i = threadIdx.x; i < held; i += 1024)
    if (live[i]) atomicAdd(&tokens[s0 + i], live[i]);
}

// Every wave takes `run` tokens in a row: q[t] (forward) or the row of dz.
template <int ZDT, int PER, bool SOFTMAX, bool GRAD>
__global__ __launch_bounds__(256) void balance_rows_kernel(Balance a, int run) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (blockIdx.x * 4 + wave) * run, last = min(first + run, a.T);
  int s = -1, end = 0;  // the sequence, and the token that it ends before
  float c[PER], coef = 0.0f;
  for (int t = first; t < last; t++) {
    TokenRow<PER> row;
    row.template load<ZDT>(a.z, (int64_t)t * a.z_stride, a.E);
    if (t == first || t >= end) {
      s = sequence_of(a.starts, a.S, t);
      const bool in = s >= 0 && s < a.S;
      end = in ? bound_of(a.starts, s + 1, a.T) : s < 0 && a.starts ? a.starts[0] : a.T;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const int e = i * 64 + lane;
        c[i] = in && e < a.E ? (float)a.counts[(int64_t)s * a.E + e] : 0.0f;
      }
      if (GRAD && in) {
        const float n = (float)a.tokens[s];
        coef = a.grad[s] * (a.alpha * a.E / a.k) / (n * n);
      }
      if (!in) s = -1;
    }
    const bool live = s >= 0 && has_route(a.idx, t, a.k, a.E);
    row.template scores<SOFTMAX>(c);
    const float q = row.share();
    if (!GRAD) {
      if (lane == 0) a.q[t] = live ? q : 0.0f;
    } else {
      const float scale = row.sum > 0.0f ? coef / row.sum : 0.0f;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const int e = i * 64 + lane;
        float g = row.a[i] * scale * (c[i] - q);
        if (!SOFTMAX) g *= row.u[i];
        g = live && row.a[i] > 0.0f ? g : 0.0f;
        const int64_t at = (int64_t)t * a.dz_stride + e;
        if (e < a.E) {
          if constexpr (ZDT == X_BF16)
            static_cast<uint16_t*>(a.dz)[at] = bf16_bits(g);
          else
            static_cast<float*>(a.dz)[at] = g;
        }
      }
    }
  }
}

// loss[s] from the tokens' numbers, added in 64 bits in a fixed order.
__global__ __launch_bounds__(1024) void balance_sum_kernel(Balance a) {
  __shared__ double part[16];
  const int s = blockIdx.x, first = bound_of(a.starts, s, a.T), end = bound_of(a.starts, s + 1, a.T);
  double v = 0.0;
  for (int t = first + threadIdx.x; t < end; t += 1024) v += a.q[t];
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = part[0];
    for (int w = 1; w < 16; w++) v += part[w];
    const double n = a.tokens[s];
    a.loss[s] = n > 0.0 ? (float)((double)a.alpha * a.E / a.k * v / (n * n)) : 0.0f;
  }
}

size_t balance_ws(int T) { return ((size_t)T * 4 + 15) / 16 * 16; }

template <int ZDT, int PER, bool GRAD>
static hipError_t launch_per(const Balance& a, hipStream_t s) {
  const int run = (a.T + 8191) / 8192;
  const dim3 grid((unsigned)((a.T + 4 * run - 1) / (4 * run)));
  if (a.softmax)
    QMOE_LAUNCH((balance_rows_kernel<ZDT, PER, true, GRAD>), grid, dim3(256), 0, s, a, run);
  else
    QMOE_LAUNCH((balance_rows_kernel<ZDT, PER, false, GRAD>), grid, dim3(256), 0, s, a, run);
  return hipGetLastError();
}
template <int ZDT, bool GRAD>
static hipError_t launch_rows(const Balance& a, hipStream_t s) {
  if (a.E <= 64) return launch_per<ZDT, 1, GRAD>(a, s);
  if (a.E <= 128) return launch_per<ZDT, 2, GRAD>(a, s);
  if (a.E <= 256) return launch_per<ZDT, 4, GRAD>(a, s);
  if (a.E <= 384) return launch_per<ZDT, 6, GRAD>(a, s);
  if (a.E <= 512) return launch_per<ZDT, 8, GRAD>(a, s);
  return launch_per<ZDT, 16, GRAD>(a, s);
}

hipError_t launch_balance_loss(const Balance& a, hipStream_t s) {
  const int64_t n = (int64_t)a.S * a.E;
  int pid = prof_begin("balance_clear", s);
  QMOE_LAUNCH(balance_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.counts, n, a.tokens, a.S);
  prof_end(pid, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.T > 0) {
    pid = prof_begin("balance_count", s);
    QMOE_LAUNCH(balance_count_kernel, dim3((unsigned)((a.T + COUNT_TOKENS - 1) / COUNT_TOKENS)), dim3(1024), 0, s, a.idx, a.T,
                a.k, a.E, a.starts, a.S, a.counts, a.tokens);
    prof_end(pid, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    pid = prof_begin("balance_rows", s);
    e = a.z_dtype == X_BF16 ? launch_rows<X_BF16, false>(a, s) : launch_rows<X_F32, false>(a, s);
    prof_end(pid, s);
    if (e != hipSuccess) return e;
  }
  pid = prof_begin("balance_sum", s);
  QMOE_LAUNCH(balance_sum_kernel, dim3(a.S), dim3(1024), 0, s, a);
  prof_end(pid, s);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const Balance& a, hipStream_t s) {
  const int pid = prof_begin("balance_backward", s);
  const hipError_t e = a.z_dtype == X_BF16 ? launch_rows<X_BF16, true>(a, s) : launch_rows<X_F32, true>(a, s);
  prof_end(pid, s);
  return e;
}

}  // namespace qmoe
