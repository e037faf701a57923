// The routed experts' products on block-scaled E4M3 weights: gate/up with
// SwiGLU and requantisation, down with each token's weighted sum.
#include "blockscale_tile.hpp"

namespace qmoe {

struct ExpertTile {
  int e, row0, rows, nt;
};

// Which M tile and which outputs a block takes.
//
// Few tiles: ids run over the M tiles first, and an XCD takes a contiguous
// eighth of them.  Many tiles: the XCDs take turns at groups of 16 tiles with
// all their outputs, so that a row's codes are read by one XCD and not by each
// for its share of the outputs (0.8 GB of 4.1 at 4096 tokens' down), and the
// tiles of a crowded expert share the weights in its L2.  1024 tokens' gate/up
// 1229 -> 1118 us; groups of 4 and 8: 1185 and 1143 us.
constexpr int TILE_GROUP = 16;
struct TilePlan {
  int by_tile;  // many tiles
  int tiles;    // M tiles, or (by_tile) M tiles of an XCD: upper bounds
  int n_tiles;
  unsigned blocks;
};
template <class C>
static TilePlan tile_plan(int64_t n, int E, int N) {
  TilePlan p;
  p.n_tiles = (N + C::BN - 1) / C::BN;
  p.tiles = (int)max_tiles(n, E, C::BM);
  p.by_tile = n >= 8 * TILE_GROUP * C::BM;  // a group at least for each XCD
  if (p.by_tile) p.tiles = (p.tiles + 8 * TILE_GROUP - 1) / (8 * TILE_GROUP) * TILE_GROUP;
  p.blocks = (unsigned)p.tiles * p.n_tiles * (p.by_tile ? 8 : 1);
  return p;
}
template <int BM>
__device__ __forceinline__ bool expert_tile(const int32_t* offsets, int E, const TilePlan& p, ExpertTile* t) {
  int pick;
  if (p.by_tile) {
    const int i = blockIdx.x >> 3, round = i / (TILE_GROUP * p.n_tiles), in = i - round * TILE_GROUP * p.n_tiles;
    t->nt = in / TILE_GROUP;
    pick = (round * 8 + (blockIdx.x & 7)) * TILE_GROUP + in % TILE_GROUP;
  } else {
    const int id = xcd_order(blockIdx.x, gridDim.x);
    t->nt = id / p.tiles;
    pick = id - t->nt * p.tiles;
  }
  return find_tile<BM>(offsets, E, pick, &t->e, &t->row0, &t->rows);
}

// A block owns BM bucket rows of one expert and one group of 128 hidden
// columns, gate and up, so that the group's maximum stays in it.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void bs_gateup_kernel(BsGateup a, TilePlan plan) {
  static_assert(C::BN == BS && C::NMAT == 2, "one group of hidden columns");
  extern __shared__ __align__(1024) uint8_t lds[];
  ExpertTile t;
  if (!expert_tile<C::BM>(a.offsets, a.E, plan, &t)) return;
  const int KB = bs_blocks(a.d), FB = bs_blocks(a.f), n0 = t.nt * BS;
  const int64_t woff = ((int64_t)t.e * a.f + n0) * a.d, soff = ((int64_t)t.e * FB + t.nt) * KB;
  const int64_t wbytes = (int64_t)min(BS, a.f - n0) * a.d;
  const __amdgpu_buffer_rsrc_t wbuf[2] = {buffer_of(a.w_gate + woff, wbytes), buffer_of(a.w_up + woff, wbytes)};
  const float* const ws[2] = {a.s_gate + soff, a.s_up + soff};
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq, (int64_t)a.T * a.d);
  const __amdgpu_buffer_rsrc_t sbuf = buffer_of(a.xs, (int64_t)a.T * KB * 4);
  auto token = [&](int i) { return a.perm[t.row0 + i] / a.k; };
  f32x4_t acc[2][C::TN][C::TM];
  tile_product<C>(
      lds, wbuf, ws, 1, a.d, xbuf, sbuf, [&](int i) { return i < t.rows ? (uint32_t)token(i) * a.d : BUFFER_OUT; },
      [&](int i) { return i < t.rows ? (uint32_t)token(i) * KB * 4 : BUFFER_OUT; }, 0, KB, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, quad = lane >> 4;
  const int wn = wave % C::WN, wm = wave / C::WN;
  uint32_t* smax = reinterpret_cast<uint32_t*>(lds);  // [WN][BM]
  // (columns past f have zero weights: h = 0 there)
#pragma unroll
  for (int j = 0; j < C::TM; j++) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < C::TN; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        acc[0][i][j][q] = silu(acc[0][i][j][q]) * acc[1][i][j][q];
        mx = max(mx, abs_bits(acc[0][i][j][q]));
      }
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
    if (quad == 0) smax[wn * C::BM + (wm * C::TM + j) * 16 + r] = mx;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < C::TM; j++) {
    const int i_row = (wm * C::TM + j) * 16 + r;
    uint32_t mx = 0;
#pragma unroll
    for (int w = 0; w < C::WN; w++) mx = max(mx, smax[w * C::BM + i_row]);
    if (i_row >= t.rows) continue;
    const float sc = bs_scale(mx);
    const int64_t row = t.row0 + i_row;
#pragma unroll
    for (int i = 0; i < C::TN; i++) {
      const int n = n0 + (wn * C::TN + i) * 16 + 4 * quad;
      const f32x4_t h = acc[0][i][j];
      if (n < a.f)  // f is a multiple of 16
        *reinterpret_cast<uint32_t*>(a.hq + row * a.f + n) =
            mx >= 0x7f800000u ? 0u : e4m3x4(h[0] / sc, h[1] / sc, h[2] / sc, h[3] / sc);
    }
    if (wn == 0 && quad == 0) a.hs[row * FB + t.nt] = sc;
  }
}

template <class C>
static hipError_t launch_gateup(const BsGateup& a, hipStream_t s) {
  const TilePlan plan = tile_plan<C>((int64_t)a.T * a.k, a.E, a.f);
  auto* k = bs_gateup_kernel<C>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  QMOE_LAUNCH(k, dim3(plan.blocks), dim3(C::THREADS), C::LDS, s, a, plan);
  return hipGetLastError();
}

// The M tile, by the rows that an expert has on average (few enough tiles that
// most experts are one, and where they are not, enough matrix work a weight
// byte).  Measured, 384 experts x 4096 x 2048 unless given, us per call with
// tiles of 16 / 32 / 48 / 128 rows:
//   0.1 rows (8 tokens)      143 / 145 / 154 / 183   (1 token: 26 / 29 / 34 / 54)
//   1 row (64 tokens)        687 / 681 / 681 / 912
//   16 rows, uniform         1287 / 1111 .. 1365 / 1373 / 1548
//   48 rows (128, crowded)   784 / 565 / 544 / 631
//   96 rows (64, crowded)    645 / 405 / 358 / 388
//   384 rows (16, 2048 x 512, crowded)  91 / 49 / 47 / 37
hipError_t launch_bs_gateup(const BsGateup& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k, E = a.E;
  if (n <= 4 * E) return launch_gateup<Tile<8, 1, 1, 1, 4, 1, 2, true>>(a, s);
  if (n <= 32 * E) return launch_gateup<Tile<8, 1, 1, 2, 2, 1, 2, true>>(a, s);
  if (n <= 160 * E) return launch_gateup<Tile<8, 1, 1, 3, 2, 1, 2, true>>(a, s);
  return launch_gateup<Tile<4, 2, 2, 4, 3, 1, 2, true>>(a, s);
}

// ye[r][n] = (D_e h_r)[n] for the bucket rows.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void bs_down_kernel(BsDown a, TilePlan plan) {
  extern __shared__ __align__(1024) uint8_t lds[];
  ExpertTile t;
  if (!expert_tile<C::BM>(a.offsets, a.E, plan, &t)) return;
  const int KB = bs_blocks(a.f), DB = bs_blocks(a.d), n0 = t.nt * C::BN;
  const __amdgpu_buffer_rsrc_t wbuf[1] = {
      buffer_of(a.w_down + ((int64_t)t.e * a.d + n0) * a.f, (int64_t)min(C::BN, a.d - n0) * a.f)};
  const float* const ws[1] = {a.s_down + ((int64_t)t.e * DB + n0 / BS) * KB};
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.hq + (int64_t)t.row0 * a.f, (int64_t)t.rows * a.f);
  const __amdgpu_buffer_rsrc_t sbuf = buffer_of(a.hs + (int64_t)t.row0 * KB, (int64_t)t.rows * KB * 4);
  f32x4_t acc[1][C::TN][C::TM];
  tile_product<C>(
      lds, wbuf, ws, DB - n0 / BS, a.f, xbuf, sbuf, [&](int i) { return i < t.rows ? (uint32_t)(i * a.f) : BUFFER_OUT; },
      [&](int i) { return i < t.rows ? (uint32_t)(i * KB * 4) : BUFFER_OUT; }, 0, KB, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, quad = lane >> 4;
  const int wn = wave % C::WN, wm = wave / C::WN;
#pragma unroll
  for (int j = 0; j < C::TM; j++) {
    const int i_row = (wm * C::TM + j) * 16 + r;
    if (i_row >= t.rows) continue;
    float* row = a.ye + (int64_t)(t.row0 + i_row) * a.d;
#pragma unroll
    for (int i = 0; i < C::TN; i++) {
      const int n = n0 + (wn * C::TN + i) * 16 + 4 * quad;
      store4(row + n, acc[0][i][j], a.d - n, true);  // d is a multiple of 16
    }
  }
}

// y[t] = add[t] + sum_j wt[t][j] ye[pos[t k + j]], 4 outputs per thread.
__global__ __launch_bounds__(256) void bs_combine_kernel(BsDown a) {
  const int d4 = a.d / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.T * d4) return;
  const int64_t t = i / d4;
  const int c = (int)(i - t * d4);
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.add) y = reinterpret_cast<const f32x4_t*>(a.add)[i];
  for (int j = 0; j < a.k; j++) {
    const int p = a.pos[t * a.k + j];
    if ((uint32_t)p >= (uint32_t)(a.T * a.k)) continue;  // a route without a place
    const float w = a.wt[t * a.k + j];
    const f32x4_t v = reinterpret_cast<const f32x4_t*>(a.ye)[(int64_t)p * d4 + c];
#pragma unroll
    for (int q = 0; q < 4; q++) y[q] = __builtin_fmaf(w, v[q], y[q]);
  }
  reinterpret_cast<f32x4_t*>(a.y)[i] = y;
}

// Few tokens: one launch and no workspace.  A block owns 16 outputs of one
// token; its 16 waves take equal stretches of the token's (route, K block)
// pairs, straight from memory with U pairs requested at a time (all of them at
// 6 routes of 2048 inputs: one round trip).  Every column of the matrix step
// holds the same row.  A wave's sum of each route goes to LDS; they are added
// in the order of the waves, then the routes weighted in their order.
template <int U>
__global__ __launch_bounds__(1024) void bs_down_token_kernel(BsDown a) {
  constexpr int WAVES = 16;
  __shared__ float part[TOPK_MAX_K][WAVES][16];
  __shared__ float route_y[TOPK_MAX_K][16];
  __shared__ int route_row[TOPK_MAX_K], route_e[TOPK_MAX_K];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16, t = blockIdx.y, KB = bs_blocks(a.f), DB = bs_blocks(a.d);
  for (int i = threadIdx.x; i < TOPK_MAX_K * WAVES * 16; i += 1024) (&part[0][0][0])[i] = 0.0f;
  if (wave < a.k) {  // wave j finds route j's row and expert: the last with offsets[e] <= row
    const int row = a.pos[t * a.k + wave];
    int below = 0;
#pragma unroll
    for (int i = 0; i < MAX_EXPERTS / 64; i++)
      if (64 * i < a.E) {
        const int e = 64 * i + lane;
        below += __popcll(__ballot(e < a.E && a.offsets[min(e, a.E - 1) + 1] <= row));
      }
    if (lane == 0) {
      route_row[wave] = row < a.T * a.k ? row : -1;
      route_e[wave] = min(below, a.E - 1);
    }
  }
  __syncthreads();
  const int pairs = a.k * KB, u0 = wave * pairs / WAVES, u1 = (wave + 1) * pairs / WAVES;
  const i32x4_t zero = {0, 0, 0, 0};
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int ub = u0; ub < u1; ub += U) {
    i32x8_t w[U], x[U];
    float sc[U];
#pragma unroll
    for (int i = 0; i < U; i++) {
      const int u = min(ub + i, u1 - 1), j = u / KB, kb = u - j * KB;
      const int row = __builtin_amdgcn_readfirstlane(route_row[j]), e = __builtin_amdgcn_readfirstlane(route_e[j]);
      const bool on = ub + i < u1 && row >= 0;
      const int k0 = kb * BS + 16 * quad;
      const uint8_t* wp = a.w_down + ((int64_t)e * a.d + n0 + r) * a.f + k0;
      const uint8_t* xp = a.hq + (int64_t)row * a.f + k0;
      const bool in0 = on && k0 < a.f, in1 = on && k0 + 64 < a.f;
      w[i] = join_pieces(in0 ? *reinterpret_cast<const i32x4_t*>(wp) : zero,
                         in1 ? *reinterpret_cast<const i32x4_t*>(wp + 64) : zero);
      x[i] = join_pieces(in0 ? *reinterpret_cast<const i32x4_t*>(xp) : zero,
                         in1 ? *reinterpret_cast<const i32x4_t*>(xp + 64) : zero);
      sc[i] = on ? a.hs[(int64_t)row * KB + kb] * a.s_down[((int64_t)e * DB + n0 / BS) * KB + kb] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < U; i++) {
      const int u = ub + i, j = u / KB;
      if (u >= u1) continue;
      F16Block wf, xf;
      wf.set(w[i]);
      xf.set(x[i]);
      const f32x4_t p = mfma_block(wf, xf);
#pragma unroll
      for (int q = 0; q < 4; q++) acc[q] = __builtin_fmaf(p[q], sc[i], acc[q]);
      if (u + 1 == u1 || (u + 1) / KB != j) {  // the wave's last pair of this route
        if (r == 0) *reinterpret_cast<f32x4_t*>(&part[j][wave][4 * quad]) = acc;
        acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  }
  __syncthreads();
  const int j = threadIdx.x >> 4, n = threadIdx.x & 15;
  if (j < a.k) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; v++) s += part[j][v][n];
    route_y[j][n] = s;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const int64_t at = (int64_t)t * a.d + n0 + n;
    float y = a.add ? a.add[at] : 0.0f;
    for (int i = 0; i < a.k; i++)
      if (route_row[i] >= 0) y = __builtin_fmaf(a.wt[t * a.k + i], route_y[i][n], y);
    a.y[at] = y;
  }
}

// (2 tokens: 27.6 us so, 25.6 us as products and a combine)
constexpr int TOKEN_MAX_T = 1;

size_t bs_down_ws(int T, int k, int d) { return T <= TOKEN_MAX_T ? 0 : (size_t)T * k * d * 4; }

template <class C>
static hipError_t launch_down(const BsDown& a, hipStream_t s) {
  const TilePlan plan = tile_plan<C>((int64_t)a.T * a.k, a.E, a.d);
  auto* k = bs_down_kernel<C>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  QMOE_LAUNCH(k, dim3(plan.blocks), dim3(C::THREADS), C::LDS, s, a, plan);
  return hipGetLastError();
}

// As for gate/up; tiles of 16 (128 outputs) / 32 / 48 / 128 rows (256 outputs):
//   0.1 rows (8 tokens)   78 / 84 / 86 / 99
//   4 rows                582 / 573 / 577 / 749
//   16 rows               749 / 658 / 650 / 800
//   64 rows, crowded      1726 / 1080 / 999 / 1139
//   384 rows (64 experts) 1348 / 740 / 655 / 630
static hipError_t launch_down_products(const BsDown& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k, E = a.E;
  if (n <= 2 * E) return launch_down<Tile<8, 1, 1, 1, 4, 1, 1, true>>(a, s);
  if (n <= 12 * E) return launch_down<Tile<8, 1, 2, 2, 2, 1, 1, true>>(a, s);
  if (n <= 200 * E) return launch_down<Tile<8, 1, 2, 3, 2, 1, 1, true>>(a, s);
  return launch_down<Tile<4, 2, 4, 4, 3, 1, 1, true>>(a, s);
}

hipError_t launch_bs_down(const BsDown& a, hipStream_t s) {
  if (a.T <= TOKEN_MAX_T) {
    const int pid = prof_begin("bs_down_token", s);
    QMOE_LAUNCH(bs_down_token_kernel<6>, dim3(a.d / 16, a.T), dim3(1024), 0, s, a);
    prof_end(pid, s);
    return hipGetLastError();
  }
  int pid = prof_begin("bs_down", s);
  hipError_t e = launch_down_products(a, s);
  prof_end(pid, s);
  if (e != hipSuccess) return e;
  pid = prof_begin("bs_combine", s);
  QMOE_LAUNCH(bs_combine_kernel, dim3((unsigned)(((int64_t)a.T * (a.d / 4) + 255) / 256)), dim3(256), 0, s, a);
  prof_end(pid, s);
  return hipGetLastError();
}

}  // namespace qmoe
