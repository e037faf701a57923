// The routed experts' products on int8 weights: gate/up with SwiGLU, down with
// each token's weighted sum.
#include "int8_tile.hpp"

namespace qmoe {

// Weights that no other block reads (those of an expert with one M tile) go past the
// caches where a call's weights are more than these hold until the next call: us with
// and without, 1024 tokens' gate/up 966 and 1090 (6.7 TB/s), 8 tokens' 118 and 132,
// their down products 566 and 606, 65 and 73; but 1 token's gate/up (101 MB) 21.1 and
// 18.9, 4 tokens' over 64 experts x 2048 x 1408 (138 MB) 30.0 and 25.4, their down
// products 18.1 and 18.5, and with few M tiles of many rows each there is no such expert.
static bool read_once(int64_t n, int E, int64_t expert_bytes) {
  return (n < E ? n : E) * expert_bytes > (int64_t(160) << 20);
}

// A block owns BM bucket rows of one expert and BN hidden columns, gate and up.
template <class C, typename OUT>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void i8_gateup_kernel(I8Gateup a, TilePlan plan, bool once) {
  static_assert(C::NMAT == 2 && C::KS == 1, "gate and up");
  extern __shared__ __align__(1024) uint8_t lds[];
  ExpertTile t;
  if (!expert_tile<C::BM>(a.offsets, a.E, plan, &t)) return;
  const int n0 = t.nt * C::BN, rows_n = min(C::BN, a.f - n0);
  const int64_t row0 = (int64_t)t.e * a.f + n0, wbytes = (int64_t)rows_n * a.d;
  const __amdgpu_buffer_rsrc_t wbuf[2] = {buffer_of(a.w_gate + row0 * a.d, wbytes), buffer_of(a.w_up + row0 * a.d, wbytes)};
  const __amdgpu_buffer_rsrc_t wsbuf[2] = {buffer_of(a.s_gate + row0, rows_n * 4), buffer_of(a.s_up + row0, rows_n * 4)};
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq, (int64_t)a.T * a.d);
  const __amdgpu_buffer_rsrc_t xsbuf = buffer_of(a.xs, (int64_t)a.T * 4);
  auto token = [&](int i) { return a.perm[t.row0 + i] / a.k; };
  i32x16_t acc[2][C::TN][C::TM];
  auto xrow = [&](int i) { return i < t.rows ? (uint32_t)token(i) * a.d : BUFFER_OUT; };
  auto srow = [&](int i) { return i < t.rows ? (uint32_t)token(i) * 4 : BUFFER_OUT; };
  const int KB = (a.d + C::BK - 1) / C::BK;
  if (once && t.alone)
    i8_product<C, true>(lds, wbuf, wsbuf, a.d, xbuf, xsbuf, xrow, srow, 0, KB, acc);
  else
    i8_product<C>(lds, wbuf, wsbuf, a.d, xbuf, xsbuf, xrow, srow, 0, KB, acc);
  i8_store<C>(lds, static_cast<OUT*>(a.h) + (int64_t)t.row0 * a.f + n0, a.f, t.rows, rows_n, 16,  // f is a multiple of 16
              [&](int i, int j, int g, int n, float xs) {
                const f32x4_t gate = i8_values(i8_run(acc[0][i][j], g), xs, i8_wscale<C>(lds, 0, n));
                const f32x4_t up = i8_values(i8_run(acc[1][i][j], g), xs, i8_wscale<C>(lds, 1, n));
                f32x4_t h;
#pragma unroll
                for (int q = 0; q < 4; q++) h[q] = silu(gate[q]) * up[q];
                return h;
              });
}

template <class C, typename OUT>
static hipError_t launch_gateup(const I8Gateup& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k;
  const TilePlan plan = tile_plan<C>(n, a.E, a.f);
  auto* k = i8_gateup_kernel<C, OUT>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  QMOE_LAUNCH(k, dim3(plan.blocks), dim3(C::THREADS), C::LDS, s, a, plan, read_once(n, a.E, 2 * (int64_t)a.f * a.d));
  return hipGetLastError();
}

// Whether n rows of N outputs fill the CUs with tiles of bm x bn.
static bool fills(int64_t n, int N, int bm, int bn) { return n / bm * ((N + bn - 1) / bn) >= 256; }

// The tile, by the rows that an expert has on average, the large ones only where they
// fill the CUs.  Measured, 384 experts x 4096 x 2048 unless given, us for 64 rows x 64
// outputs (three stages) / 128 x 64 / 256 x 128:
//   0.02 rows (1 token) 18.9 / 24.8, 0.1 (8 tokens) 130 / 138, 4 (256) 1071 / 1184, 16 (1024) 1124 / 1277
//   (these four before weights went past the caches), 48 (1024, 128 experts) 364 / 373,
//   64 (4096) uniform 1417 / 1237, crowded 1403 / 1463, 96 (1024, 64 experts) 297 / 253 / 426,
//   256 (1024, 16 experts, crowded) 141 / 122 / 143, 384 (1024, 16 experts) 189 / 152 / 128,
//   384 (4096, 64 experts) 730 / 611 / 529, 4096 (one expert) 109 / 78 / 67, 1000 (one) 28 / 29 / 46
// One expert (a shared one) with few rows is far from its bytes: 15.4 us for 1 to 16 rows,
// 15.8 for 64, as 2048 outputs are 32 tiles, on an eighth of the CUs.
template <typename OUT>
static hipError_t pick_gateup(const I8Gateup& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k, E = a.E;
  if (n > 320 * E && fills(n, a.f, 256, 128)) return launch_gateup<I8Tile<2, 4, 2, 2, 64, 3, 1, 2>, OUT>(a, s);
  if (n > 64 * E && fills(n, a.f, 128, 64)) return launch_gateup<I8Tile<2, 2, 1, 2, 128, 2, 1, 2>, OUT>(a, s);
  return launch_gateup<I8Tile<2, 2, 1, 1, 128, 3, 1, 2>, OUT>(a, s);
}

hipError_t launch_i8_gateup(const I8Gateup& a, hipStream_t s) {
  return a.h_dtype == X_BF16 ? pick_gateup<uint16_t>(a, s) : pick_gateup<float>(a, s);
}

// ye[r][n] = (D_e h_r)[n] for the bucket rows.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void i8_down_kernel(I8Down a, TilePlan plan, bool once) {
  extern __shared__ __align__(1024) uint8_t lds[];
  ExpertTile t;
  if (!expert_tile<C::BM>(a.offsets, a.E, plan, &t)) return;
  const int n0 = t.nt * C::BN, rows_n = min(C::BN, a.d - n0);
  const int64_t row0 = (int64_t)t.e * a.d + n0;
  const __amdgpu_buffer_rsrc_t wbuf[1] = {buffer_of(a.w_down + row0 * a.f, (int64_t)rows_n * a.f)};
  const __amdgpu_buffer_rsrc_t wsbuf[1] = {buffer_of(a.s_down + row0, rows_n * 4)};
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.hq + (int64_t)t.row0 * a.f, (int64_t)t.rows * a.f);
  const __amdgpu_buffer_rsrc_t xsbuf = buffer_of(a.hs + t.row0, t.rows * 4);
  i32x16_t acc[1][C::TN][C::TM];
  auto xrow = [&](int i) { return i < t.rows ? (uint32_t)(i * a.f) : BUFFER_OUT; };
  auto srow = [&](int i) { return (uint32_t)(i * 4); };
  const int KB = (a.f + C::BK - 1) / C::BK;
  if (once && t.alone)
    i8_product<C, true>(lds, wbuf, wsbuf, a.f, xbuf, xsbuf, xrow, srow, 0, KB, acc);
  else
    i8_product<C>(lds, wbuf, wsbuf, a.f, xbuf, xsbuf, xrow, srow, 0, KB, acc);
  i8_store<C>(lds, a.ye + (int64_t)t.row0 * a.d + n0, a.d, t.rows, rows_n, 16, [&](int i, int j, int g, int n, float xs) {
    return i8_values(i8_run(acc[0][i][j], g), xs, i8_wscale<C>(lds, 0, n));
  });
}

// One or two tokens: one launch and no workspace.  A block owns 16 outputs of one
// token; its 16 waves share the runs of 128 inputs (and, where two groups of waves
// or more have one for each, the routes), straight from memory with U routes
// requested at a time.  Column j of the matrix steps' activations is route j's
// row; the product with route j's weights takes that column and zeros, so one
// accumulator serves every route.  The waves' sums are added, then the routes
// weighted in their order.  Bound by the weights, after two loads in a row (positions
// and offsets, then weights): 6 of 384 experts x 2048 x 4096, 1 token 11.2 us (4.5 TB/s
// over the whole call; weights past the caches 12.4), 2 tokens 20.9.
template <int U>
__global__ __launch_bounds__(1024) void i8_down_token_kernel(I8Down a) {
  constexpr int WAVES = 16;
  static_assert(TOPK_MAX_K == 16, "a column of the matrix step for each route");
  __shared__ i32x4_t part[WAVES][16][4];  // [wave][route][output / 4]
  __shared__ float route_y[16][16];
  __shared__ int route_row[16], route_e[16];
  __shared__ float route_wt[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16, t = blockIdx.y, KB = bs_blocks(a.f);
  const int64_t out = (int64_t)t * a.d + n0 + r;
  const float add = a.add && threadIdx.x < 16 ? a.add[out] : 0.0f;  // (requested early, as the weights of the routes)
  int row = -1, below = 0;
  float wt = 0.0f;
  if (wave < a.k) {  // wave j finds route j's row and expert: the last with offsets[e] <= row
    constexpr int MOST = MAX_EXPERTS / 64;
    row = a.pos[t * a.k + wave];
    wt = a.wt[t * a.k + wave];
    const __amdgpu_buffer_rsrc_t ends = buffer_of(a.offsets + 1, (int64_t)a.E * 4);
    int end[MOST];
#pragma unroll
    for (int i = 0; i < MOST; i++) end[i] = __float_as_int(buffer_load4(ends, (64 * i + lane) * 4));  // all at once
#pragma unroll
    for (int i = 0; i < MOST; i++) below += __popcll(__ballot(64 * i + lane < a.E && end[i] <= row));
  }
  if (lane == 0) {
    route_row[wave] = row < a.T * a.k ? row : -1;
    route_e[wave] = min(below, a.E - 1);
    route_wt[wave] = wt;
  }
  __syncthreads();
  row = route_row[r];
  const int e = route_e[r];
  const uint32_t valid = (uint32_t)__ballot(row >= 0) & 0xffffu;
  const int64_t x_row = max(row, 0);
  const int8_t* xp = a.hq + x_row * a.f;
  // thread (j, n) of the first 256 finishes route j's output n: its scales are requested with the codes
  const int fj = threadIdx.x >> 4 & 15, fn = threadIdx.x & 15;
  const bool finish = threadIdx.x < 256 && route_row[fj] >= 0;
  const float xs = finish ? a.hs[route_row[fj]] : 0.0f;
  const float ws = finish ? a.s_down[(int64_t)route_e[fj] * a.d + n0 + fn] : 0.0f;
  const int G = KB >= WAVES ? 1 : WAVES / KB;  // groups of waves that share the routes
  const int g = KB >= WAVES ? 0 : wave / KB;
  i32x4_t acc = {0, 0, 0, 0};
  for (int jb = g; jb < (g < G ? a.k : 0); jb += G * U)
    for (int kb = KB >= WAVES ? wave : wave - g * KB; kb < KB; kb += WAVES) {
      const int k0 = kb * BS + 16 * quad;
      const bool in0 = k0 < a.f, in1 = k0 + 64 < a.f;  // past f: some code of the row, times 0
      const int c0 = in0 ? k0 : 0, c1 = in1 ? k0 + 64 : 0;
      i32x4_t w0[U], w1[U];
#pragma unroll
      for (int i = 0; i < U; i++) {
        const int j = jb + G * i;
        const bool on = j < a.k && (valid >> (j & 15) & 1);  // (else a buffer of no bytes)
        const int64_t at = ((int64_t)__builtin_amdgcn_readlane(e, j & 15) * a.d + n0) * a.f;
        const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.w_down + at, on ? 16 * a.f : 0);
        w0[i] = buffer_load16(wbuf, r * a.f + c0);
        w1[i] = buffer_load16(wbuf, r * a.f + c1);
      }
      const i32x4_t zero = {0, 0, 0, 0};
      i32x4_t x0 = *reinterpret_cast<const i32x4_t*>(xp + c0), x1 = *reinterpret_cast<const i32x4_t*>(xp + c1);
      __builtin_amdgcn_sched_barrier(0);  // (else the loads go between the matrix steps, to save registers)
      x0 = in0 ? x0 : zero;
      x1 = in1 ? x1 : zero;
#pragma unroll
      for (int i = 0; i < U; i++) {
        const bool mine = r == jb + G * i;
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0[i], mine ? x0 : zero, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1[i], mine ? x1 : zero, acc, 0, 0, 0);
      }
    }
  part[wave][r][quad] = acc;  // (0 for the routes of other groups)
  __syncthreads();
  if (threadIdx.x < 256 && fj < a.k) {
    int s = part[0][fj][fn >> 2][fn & 3];
#pragma unroll
    for (int v = 1; v < WAVES; v++) s += part[v][fj][fn >> 2][fn & 3];
    route_y[fj][fn] = ((float)s * xs) * ws;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    float y = add;
#pragma unroll
    for (int i = 0; i < TOPK_MAX_K; i++) y = valid >> i & 1 ? __builtin_fmaf(route_wt[i], route_y[i][fn], y) : y;
    a.y[out] = y;
  }
}

constexpr int TOKEN_MAX_T = 2;

size_t i8_down_ws(int T, int k, int d) { return T <= TOKEN_MAX_T ? 0 : (size_t)T * k * d * 4; }

template <class C>
static hipError_t launch_down(const I8Down& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k;
  const TilePlan plan = tile_plan<C>(n, a.E, a.d);
  auto* k = i8_down_kernel<C>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  QMOE_LAUNCH(k, dim3(plan.blocks), dim3(C::THREADS), C::LDS, s, a, plan, read_once(n, a.E, (int64_t)a.f * a.d));
  return hipGetLastError();
}

// The tile, as for gate/up: 64 rows x 128 outputs on eight waves (to keep loads in
// flight), on two (fewer reads of LDS), 128 x 128 and 256 x 256.  The products without
// the sum, us:
//   0.06 rows (4 tokens) 33.6 / 37.5 / 48.6, 0.1 (8 tokens) 64.5 / 68.8 / 73.4, 1 (64) 314 / 318 / 362,
//   16 (1024) 566 / 567 / 609, 48 (512 over 64 experts) 114 / 116 / 124, 64 crowded 784 / 767 / 819 / 895,
//   64 uniform 783 / 760 / 705 / 839, 256 (1024, 16 experts, crowded) 86 / 87 / 77 / 74,
//   384 (64 experts) 430 / 414 / 359 / 308, 1024 (16 experts, crowded) 267 / 255 / 218 / 189
// Up to some hundred rows bound by memory: without its matrix steps the 64-row product
// took as long (819 us then), without its stores 680.
static hipError_t launch_down_products(const I8Down& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k, E = a.E;
  if (n >= 256 * E && fills(n, a.d, 256, 256)) return launch_down<I8Tile<4, 2, 2, 4, 128, 2, 1, 1>>(a, s);
  if (n > 128 * E && fills(n, a.d, 128, 128)) return launch_down<I8Tile<2, 2, 2, 2, 128, 2, 1, 1>>(a, s);
  if (n > 16 * E) return launch_down<I8Tile<2, 1, 2, 2, 128, 2, 1, 1>>(a, s);
  return launch_down<I8Tile<4, 2, 1, 1, 128, 2, 1, 1>>(a, s);
}

hipError_t launch_i8_down(const I8Down& a, hipStream_t s) {
  if (a.T <= TOKEN_MAX_T) {
    const int pid = prof_begin("i8_down_token", s);
    QMOE_LAUNCH(i8_down_token_kernel<6>, dim3(a.d / 16, a.T), dim3(1024), 0, s, a);
    prof_end(pid, s);
    return hipGetLastError();
  }
  const int pid = prof_begin("i8_down", s);
  const hipError_t e = launch_down_products(a, s);
  prof_end(pid, s);
  if (e != hipSuccess) return e;
  return launch_combine("i8_combine", a.ye, a.T, a.k, a.d, a.wt, a.pos, a.add, a.y, s);
}

}  // namespace qmoe
