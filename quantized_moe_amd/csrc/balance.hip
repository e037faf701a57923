// The router's balance: tokens and routes per expert of each sequence, the
// balance loss, and its gradient with respect to the logits.
//
// loss_s = alpha E / (k n_s^2) sum_t q_t with q_t = sum_e c_se p_te: the counts
// c_se come from the routes alone, so no column sum of probabilities over the
// tokens is ever kept; every token gives one number, and the gradient
//   dz_te = g_s alpha E / (k n_s^2) p_te (c_se - q_t)   (sigmoid: (1 - sigma_te) times that)
// needs the token's own row again and nothing else.  65536 tokens x 384 experts: fp32
// forward 20.5 us, 4.9 TB/s of logits, with vector instructions in 73 % of the cycles;
// backward 33, 6.1 TB/s, 75 %; bf16 19.7 and 25 us, bound by vector instructions (98 %).
#include "balance_places.hpp"
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

// The starts as a wave looks them up: up to 64 of them (S < 64) stay in its lanes, one
// load for every search.
struct Starts {
  const int32_t* p;
  int S, T, v;
  __device__ __forceinline__ Starts(const int32_t* starts, int S_, int T_) : p(starts), S(S_), T(T_) {
    const int lane = threadIdx.x & 63;
    v = p && S < 64 ? p[min(lane, S)] : 0;
  }
  // The sequence of token t (the same in every lane; -1: none), and the token that it,
  // or the gap that t is in, ends before.
  __device__ __forceinline__ int find(int t, int* end) const {
    *end = T;
    if (!p) return 0;
    if (S >= 64) {
      const int s = sequence_of(p, S, t);
      if (s < S) *end = bound_of(p, s + 1, T);
      return s < S ? s : -1;
    }
    const int c = __popcll(__ballot((int)(threadIdx.x & 63) <= S && v <= t));
    if (c <= S) *end = min(max(__builtin_amdgcn_readlane(v, c), 0), T);
    return c <= S ? c - 1 : -1;
  }
  // The same for a token of each lane: -1 .. S.
  __device__ __forceinline__ int find_lane(int t) const {
    if (!p) return 0;
    int n = 0, hi = S + 1;
    if (S < 64) {
      for (int i = 0; i <= S; i++) n += __builtin_amdgcn_readlane(v, i) <= t;
      return n - 1;
    }
    while (n < hi) {
      const int mid = (n + hi) / 2;
      if (p[mid] <= t)
        n = mid + 1;
      else
        hi = mid;
    }
    return n - 1;
  }
};

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
// v of the lanes 16 (32) away: both halves of a swap of v with itself.
template <class F>
__device__ __forceinline__ float over_rows(float v, F&& f) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f<0xb1>(v));
  v = fmaxf(v, dpp_f<0x4e>(v));
  v = fmaxf(v, dpp_f<0x141>(v));
  v = fmaxf(v, dpp_f<0x140>(v));
  return over_rows(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<0xb1>(v);
  v += dpp_f<0x4e>(v);
  v += dpp_f<0x141>(v);
  v += dpp_f<0x140>(v);
  return over_rows(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

constexpr float LOG2E = 1.4426950408889634f;

// The experts of a lane, i * 64 + lane; past the last one the last again, `in` false.
template <int PER>
struct Experts {
  uint32_t at[PER];
  bool in[PER];
  __device__ __forceinline__ explicit Experts(int E) {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int e = i * 64 + (threadIdx.x & 63);
      in[i] = e < E;
      at[i] = min(e, E - 1);
    }
  }
};

// One token in one wave, PER logits a lane.  a = the scores (0: the expert is out),
// u = 1 - sigma of the sigmoid; sum = their sum, dot = sum c a.
template <int PER>
struct TokenRow {
  float a[PER], u[PER];
  float sum, dot;
  template <int ZDT>
  __device__ __forceinline__ void load(const void* z, int64_t at, const Experts<PER>& x) {
    if constexpr (ZDT == X_BF16) {
      const uint16_t* row = static_cast<const uint16_t*>(z) + at;
#pragma unroll
      for (int i = 0; i < PER; i++) a[i] = __uint_as_float(row[x.at[i]]);  // (widened where it is used)
    } else {
      const float* row = static_cast<const float*>(z) + at;
#pragma unroll
      for (int i = 0; i < PER; i++) a[i] = row[x.at[i]];
    }
  }
  template <int ZDT, bool SOFTMAX>
  __device__ __forceinline__ void scores(const float (&c)[PER], const Experts<PER>& x) {
    float m = -0x1p127f;  // (no expert in: every score is 0)
    if (ZDT == X_BF16) {
#pragma unroll
      for (int i = 0; i < PER; i++) a[i] = bf16_bits_to_float(__float_as_uint(a[i]));
    }
    if (SOFTMAX) {
#pragma unroll
      for (int i = 0; i < PER; i++) {
        a[i] = x.in[i] && a[i] > -0x1p127f ? fminf(a[i], 0x1.fffffep127f) : -INFINITY;  // (NaN fails the comparison)
        m = fmaxf(m, a[i]);
      }
      m = wave_max(m);
    }
    sum = 0.0f;
    dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      if (SOFTMAX) {
        a[i] = __builtin_amdgcn_exp2f((a[i] - m) * LOG2E);
      } else {
        const bool in = x.in[i] && a[i] > -0x1p127f;
        const float e = __builtin_amdgcn_exp2f(__builtin_amdgcn_fmed3f(a[i], -80.0f, 80.0f) * -LOG2E);
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
__device__ __forceinline__ bool has_route(int32_t e, int k, int E) {
  return __ballot((int)(threadIdx.x & 63) < k && (uint32_t)e < (uint32_t)E) != 0;
}
// Lane j < k: the token's route j.
__device__ __forceinline__ int32_t route_of(const int32_t* idx, int64_t t, int k) {
  return idx[t * k + min((int)(threadIdx.x & 63), k - 1)];
}

}  // namespace

__global__ __launch_bounds__(256) void balance_clear_kernel(int32_t* counts, int64_t n, int32_t* tokens, int S) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) counts[i] = 0;
  if (i < S) tokens[i] = 0;
}

constexpr int COUNT_HELD = 12288;                // counts that a block holds in LDS ...
constexpr int COUNT_HELD_S = COUNT_HELD / 8;     // ... of so many sequences at most (with fewer than 8 experts too)
__device__ __host__ __forceinline__ int held_sequences(int E) { return COUNT_HELD / (E < 8 ? 8 : E); }

// n routes of a token added to its sequence's counts in LDS.  Whole numbers: the order
// of the atomics changes nothing.  true: one of them is a route.
__device__ __forceinline__ bool count_routes(const int (&e)[8], int n, int E, int* hist) {
  bool any = false;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    if (j >= n || (uint32_t)e[j] >= (uint32_t)E) continue;
    any = true;
    atomicAdd(&hist[e[j]], 1);
  }
  return any;
}
// 8 routes of token t from the jth on.
__device__ __forceinline__ void load_routes(const Balance& a, int t, int j, int (&e)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) e[i] = a.idx[(int64_t)t * a.k + min(j + i, a.k - 1)];
}

// Four threads a token (routes r, r + 4, ..: a thread's LDS atomics follow each other),
// 256 tokens at a time, all routes requested first.  WHOLE: one block takes all tokens
// and sequences and writes the counts; else they are added to cleared memory, from so
// many tokens a block that 64 blocks at most add to the same counts.
constexpr int COUNT_TOKENS = 1024;  // of a block at most
template <bool WHOLE>
__global__ __launch_bounds__(1024) void balance_count_kernel(Balance a, int per) {
  constexpr int N = COUNT_TOKENS / 256;
  __shared__ int hist[COUNT_HELD], live[COUNT_HELD_S];
  const int r = threadIdx.x & 3, t0 = blockIdx.x * per, t1 = min(t0 + per, a.T), first = t0 + (threadIdx.x >> 2);
  int e[N][4], end;
#pragma unroll
  for (int i = 0; i < N; i++)
    if (t0 + i * 256 < t1)
#pragma unroll
      for (int j = 0; j < 4; j++)
        e[i][j] = r + 4 * j < a.k ? a.idx[(int64_t)min(first + i * 256, a.T - 1) * a.k + r + 4 * j] : -1;
  const Starts starts(a.starts, a.S, a.T);
  int s0 = WHOLE ? 0 : max(starts.find(t0, &end), 0), s1 = a.S - 1;
  if (!WHOLE && a.S >= 64) {  // (fewer are taken whole)
    s0 = max(sequence_of(a.starts, a.S, t0), 0);
    s1 = min(sequence_of(a.starts, a.S, t1 - 1), a.S - 1);
  }
  const int held = WHOLE ? a.S : min(held_sequences(a.E), s1 - s0 + 1), n = held * a.E;  // (<= 0: no token of any sequence)
  for (int i = threadIdx.x; i < n; i += 1024) hist[i] = 0;
  for (int i = threadIdx.x; i < held; i += 1024) live[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; i++) {
    if (t0 + i * 256 >= t1) break;
    const int t = first + i * 256, s = starts.find_lane(t);
    const bool in = t < t1 && s >= s0 && s <= s1, here = WHOLE || s - s0 < held;
    bool any = false;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (!in || (uint32_t)e[i][j] >= (uint32_t)a.E) continue;
      any = true;
      if (here)
        atomicAdd(&hist[(s - s0) * a.E + e[i][j]], 1);
      else
        atomicAdd(&a.counts[(int64_t)s * a.E + e[i][j]], 1);
    }
    const bool routed = __ballot(any) >> (threadIdx.x & 60) & 15;  // one of the token's four threads
    if (r != 0 || !routed) continue;
    if (here)
      atomicAdd(&live[s - s0], 1);
    else
      atomicAdd(&a.tokens[s], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 1024) {
    if (WHOLE)
      a.counts[i] = hist[i];
    else if (hist[i])
      atomicAdd(&a.counts[(int64_t)s0 * a.E + i], hist[i]);
  }
  for (int i = threadIdx.x; i < held; i += 1024) {
    if (WHOLE)
      a.tokens[i] = live[i];
    else if (live[i])
      atomicAdd(&a.tokens[s0 + i], live[i]);
  }
}

__device__ __forceinline__ float loss_of(const Balance& a, double sum, int tokens) {
  const double n = tokens;
  return tokens > 0 ? (float)((double)a.alpha * a.E / a.k * sum / (n * n)) : 0.0f;
}

// The loss of sequence s, by one wave.
__device__ __forceinline__ double sequence_sum(const Balance& a, int s, int run) {
  const int lane = threadIdx.x & 63, per = ROW_WAVES * run;
  const int first = bound_of(a.starts, s, a.T), end = bound_of(a.starts, s + 1, a.T);
  double v = 0.0;
  const int block = block_from(first, run), at = wave_place(first, end, lane, run);
  if (lane < ROW_WAVES && at >= 0) v = a.q[at];
  for (int b = block + lane; b * per < end; b += 64 * 8) {  // (T and a stride of 512 blocks stay below 2^27)
    double part[8];
#pragma unroll
    for (int i = 0; i < 8; i++) part[i] = (b + 64 * i) * per < end ? a.q[(b + 64 * i) * per] : 0.0;
#pragma unroll
    for (int i = 0; i < 8; i++) v += part[i];
  }
  return wave_sum(v);
}

// A wave's tokens [first, last) in turn: use(t, row, has a route).  AHEAD of them are
// requested at a time, each into the registers of the one just used (moving loaded
// registers along would wait for the loads).
template <int ZDT, int PER, bool SOFTMAX, class Enter, class Use>
__device__ __forceinline__ void each_token(const Balance& a, int first, int last, const Experts<PER>& x, Enter&& enter, Use&& use) {
  constexpr int AHEAD = PER <= 8 ? 4 : 2;
  TokenRow<PER> row[AHEAD];
  int32_t route[AHEAD];
  auto request = [&](int t, int i) {
    if (t >= last) return;
    row[i].template load<ZDT>(a.z, (int64_t)t * a.z_stride, x);
    route[i] = route_of(a.idx, t, a.k);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; i++) request(first + i, i);
  for (int t0 = first; t0 < last; t0 += AHEAD)
#pragma unroll
    for (int i = 0; i < AHEAD; i++) {
      const int t = t0 + i;
      if (t >= last) break;
      const float(&c)[PER] = enter(t);
      row[i].template scores<ZDT, SOFTMAX>(c, x);
      use(t, row[i], has_route(route[i], a.k, a.E));
      request(t + AHEAD, i);
    }
}

// The sequence that a wave's tokens are in, with its counts.
template <int PER>
struct Sequence {
  int s = -1, end = 0;  // (-1: none), the token that it ends before
  float c[PER];
  __device__ __forceinline__ void enter(const Balance& a, const Starts& starts, int t, const Experts<PER>& x) {
    s = starts.find(t, &end);
    const int32_t* counts = a.counts + (int64_t)max(s, 0) * a.E;
    int32_t v[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) v[i] = counts[x.at[i]];
#pragma unroll
    for (int i = 0; i < PER; i++) c[i] = (float)v[i];
  }
};

// Forward: every wave takes `run` tokens in a row; q of its tokens in 64 bits, one
// sum for each sequence that it meets (balance_places.hpp says where it goes).
template <int ZDT, int PER, bool SOFTMAX>
__global__ __launch_bounds__(64 * ROW_WAVES) void balance_forward_kernel(Balance a, int run) {
  __shared__ double sums[ROW_WAVES];  // of the sequence of the block's first token
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block_first = blockIdx.x * ROW_WAVES * run;
  const int first = block_first + wave * run, last = min(first + run, a.T);
  const Starts starts(a.starts, a.S, a.T);
  int block_end;
  const int block_s = starts.find(block_first, &block_end);
  const Experts<PER> x(a.E);
  Sequence<PER> seq;
  int from = first;
  double total = 0.0;
  auto put = [&] {  // the sum of the tokens from .. of a sequence
    if (seq.s == block_s)
      sums[wave] = total;
    else if (lane == 0)
      a.q[from] = total;
  };
  sums[wave] = 0.0;
  each_token<ZDT, PER, SOFTMAX>(
      a, first, last, x,
      [&](int t) -> const float(&)[PER] {
        if (t == first || t >= seq.end) {
          if (t > first) put();
          total = 0.0;
          from = t;
          seq.enter(a, starts, t, x);
        }
        return seq.c;
      },
      [&](int, TokenRow<PER>& row, bool routed) {
        if (seq.s >= 0 && routed) total += row.share();
      });
  if (first < last) put();
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = sums[0];
#pragma unroll
    for (int w = 1; w < ROW_WAVES; w++) v += sums[w];
    a.q[block_first] = v;
  }
}

// The losses, a wave for each sequence.
__global__ __launch_bounds__(256) void balance_sum_kernel(Balance a, int run) {
  const int s = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (s >= a.S) return;
  const double v = sequence_sum(a, s, run);
  if ((threadIdx.x & 63) == 0) a.loss[s] = loss_of(a, v, a.tokens[s]);
}

// Backward: every wave takes `run` tokens in a row.  scale = alpha E / k.
template <int ZDT, int PER, bool SOFTMAX>
__global__ __launch_bounds__(256) void balance_backward_kernel(Balance a, int run, double scale) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (blockIdx.x * 4 + wave) * run, last = min(first + run, a.T);
  if (first >= last) return;
  float coef = 0.0f;
  const Starts starts(a.starts, a.S, a.T);
  const Experts<PER> x(a.E);
  Sequence<PER> seq;
  each_token<ZDT, PER, SOFTMAX>(
      a, first, last, x,
      [&](int t) -> const float(&)[PER] {
        if (t == first || t >= seq.end) {
          seq.enter(a, starts, t, x);
          if (seq.s >= 0) {
            const float n = (float)a.tokens[seq.s];
            coef = (float)((double)a.grad[seq.s] * scale * (1.0f / (n * n)));  // (parts of it may be past fp32)
          }
        }
        return seq.c;
      },
      [&](int t, TokenRow<PER>& row, bool routed) {
        const bool live = seq.s >= 0 && routed;
        const float q = row.share(), inv = row.sum > 0.0f ? 1.0f / row.sum : 0.0f;  // (sums are at least e^-80)
#pragma unroll
        for (int i = 0; i < PER; i++) {
          float g = row.a[i] * inv * (coef * (seq.c[i] - q));
          if (!SOFTMAX) g *= row.u[i];
          g = live && row.a[i] > 0.0f ? g : 0.0f;
          if constexpr (ZDT == X_BF16) {
            if (x.in[i]) __builtin_nontemporal_store(bf16_bits(g), static_cast<uint16_t*>(a.dz) + (int64_t)t * a.dz_stride + x.at[i]);
          } else {
            if (x.in[i]) __builtin_nontemporal_store(g, static_cast<float*>(a.dz) + (int64_t)t * a.dz_stride + x.at[i]);
          }
        }
      });
}

// Few tokens: all of it in one block, the counts in LDS.
constexpr int SMALL_TOKENS = 128;
template <int ZDT, int PER, bool SOFTMAX>
__global__ __launch_bounds__(1024) void balance_small_kernel(Balance a) {
  __shared__ int hist[COUNT_HELD], live[COUNT_HELD_S];
  __shared__ int seq[SMALL_TOKENS];  // -1: the token takes no part
  __shared__ double q[SMALL_TOKENS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Experts<PER> x(a.E);
  TokenRow<PER> row[2];
#pragma unroll
  for (int i = 0; i < 2; i++)
    if (wave + 16 * i < a.T) row[i].template load<ZDT>(a.z, (int64_t)(wave + 16 * i) * a.z_stride, x);
  const Starts starts(a.starts, a.S, a.T);
  const int counted = a.S * a.E, my = threadIdx.x;
  int e[8];
  if (my < a.T) load_routes(a, my, 0, e);
  for (int i = threadIdx.x; i < counted; i += 1024) hist[i] = 0;
  for (int i = threadIdx.x; i < a.S; i += 1024) live[i] = 0;
  const int my_s = starts.find_lane(my);
  __syncthreads();
  if (my < a.T) {
    bool any = my_s >= 0 && my_s < a.S;
    if (any) {
      any = count_routes(e, a.k, a.E, hist + my_s * a.E);
      if (a.k > 8) {
        load_routes(a, my, 8, e);
        any |= count_routes(e, a.k - 8, a.E, hist + my_s * a.E);
      }
      if (any) atomicAdd(&live[my_s], 1);
    }
    seq[my] = any ? my_s : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < counted; i += 1024) a.counts[i] = hist[i];
  for (int i = threadIdx.x; i < a.S; i += 1024) a.tokens[i] = live[i];
  for (int t0 = wave; t0 < a.T; t0 += 32)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int t = t0 + 16 * i;
      if (t >= a.T) break;
      const int s = max(seq[t], 0);
      float c[PER];
#pragma unroll
      for (int j = 0; j < PER; j++) c[j] = (float)hist[s * a.E + x.at[j]];
      row[i].template scores<ZDT, SOFTMAX>(c, x);
      if (lane == 0) q[t] = row[i].share();
      if (t + 32 < a.T) row[i].template load<ZDT>(a.z, (int64_t)(t + 32) * a.z_stride, x);
    }
  __syncthreads();
  for (int s = wave; s < a.S; s += 16) {
    double v = 0.0;
    for (int t = lane; t < a.T; t += 64) v += seq[t] == s ? q[t] : 0.0;
    v = wave_sum(v);
    if (lane == 0) a.loss[s] = loss_of(a, v, live[s]);
  }
}

static bool is_small(int T, int S, int E) { return T <= SMALL_TOKENS && S <= held_sequences(E); }

size_t balance_ws(int T, int S, int E) { return is_small(T, S, E) ? 0 : (size_t)T * 8; }

template <int ZDT, int PER>
static hipError_t launch_small(const Balance& a, hipStream_t s) {
  if (a.softmax)
    QMOE_LAUNCH((balance_small_kernel<ZDT, PER, true>), dim3(1), dim3(1024), 0, s, a);
  else
    QMOE_LAUNCH((balance_small_kernel<ZDT, PER, false>), dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}
template <int ZDT, int PER>
static hipError_t launch_forward(const Balance& a, hipStream_t s) {
  const int run = run_of(a.T);
  const dim3 grid((unsigned)((a.T + ROW_WAVES * run - 1) / (ROW_WAVES * run))), block(64 * ROW_WAVES);
  if (a.softmax)
    QMOE_LAUNCH((balance_forward_kernel<ZDT, PER, true>), grid, block, 0, s, a, run);
  else
    QMOE_LAUNCH((balance_forward_kernel<ZDT, PER, false>), grid, block, 0, s, a, run);
  return hipGetLastError();
}
template <int ZDT, int PER>
static hipError_t launch_backward(const Balance& a, hipStream_t s) {
  const int run = run_of(a.T);
  const dim3 grid((unsigned)((a.T + 4 * run - 1) / (4 * run)));
  const double scale = (double)a.alpha * a.E / a.k;
  if (a.softmax)
    QMOE_LAUNCH((balance_backward_kernel<ZDT, PER, true>), grid, dim3(256), 0, s, a, run, scale);
  else
    QMOE_LAUNCH((balance_backward_kernel<ZDT, PER, false>), grid, dim3(256), 0, s, a, run, scale);
  return hipGetLastError();
}

enum Pass { SMALL, FORWARD, BACKWARD };
template <Pass P, int ZDT, int PER>
static hipError_t launch_pass(const Balance& a, hipStream_t s) {
  if constexpr (P == SMALL)
    return launch_small<ZDT, PER>(a, s);
  else if constexpr (P == BACKWARD)
    return launch_backward<ZDT, PER>(a, s);
  else
    return launch_forward<ZDT, PER>(a, s);
}
template <Pass P, int ZDT>
static hipError_t launch_dtype(const Balance& a, hipStream_t s) {
  if (a.E <= 64) return launch_pass<P, ZDT, 1>(a, s);
  if (a.E <= 128) return launch_pass<P, ZDT, 2>(a, s);
  if (a.E <= 256) return launch_pass<P, ZDT, 4>(a, s);
  if (a.E <= 384) return launch_pass<P, ZDT, 6>(a, s);
  if (a.E <= 512) return launch_pass<P, ZDT, 8>(a, s);
  return launch_pass<P, ZDT, 16>(a, s);
}
template <Pass P>
static hipError_t launch(const char* name, const Balance& a, hipStream_t s) {
  const int pid = prof_begin(name, s);
  const hipError_t e = a.z_dtype == X_BF16 ? launch_dtype<P, X_BF16>(a, s) : launch_dtype<P, X_F32>(a, s);
  prof_end(pid, s);
  return e;
}

hipError_t launch_balance_loss(const Balance& a, hipStream_t s) {
  if (is_small(a.T, a.S, a.E)) return launch<SMALL>("balance_small", a, s);
  hipError_t e;
  int pid;
  if (a.T > 0 && a.T <= COUNT_TOKENS && a.S <= held_sequences(a.E)) {
    pid = prof_begin("balance_count", s);
    QMOE_LAUNCH(balance_count_kernel<true>, dim3(1), dim3(1024), 0, s, a, COUNT_TOKENS);
    prof_end(pid, s);
  } else {
    const int64_t n = (int64_t)a.S * a.E;
    pid = prof_begin("balance_clear", s);
    QMOE_LAUNCH(balance_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.counts, n, a.tokens, a.S);
    prof_end(pid, s);
    if (a.T > 0) {
      if ((e = hipGetLastError()) != hipSuccess) return e;
      const int per = min(COUNT_TOKENS, (a.T + 64 * 256 - 1) / (64 * 256) * 256);
      pid = prof_begin("balance_count", s);
      QMOE_LAUNCH(balance_count_kernel<false>, dim3((unsigned)((a.T + per - 1) / per)), dim3(1024), 0, s, a, per);
      prof_end(pid, s);
    }
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.T > 0 && (e = launch<FORWARD>("balance_forward", a, s)) != hipSuccess) return e;
  pid = prof_begin("balance_sum", s);
  QMOE_LAUNCH(balance_sum_kernel, dim3((unsigned)((a.S + 3) / 4)), dim3(256), 0, s, a, run_of(a.T));
  prof_end(pid, s);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const Balance& a, hipStream_t s) { return launch<BACKWARD>("balance_backward", a, s); }

}  // namespace qmoe
