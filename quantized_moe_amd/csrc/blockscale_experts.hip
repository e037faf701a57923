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
// 1229 -> 1118 us; groups of 4 and 8: 1185 and 1143 us.  The groups are as large
// as gives every XCD the same number of them: 1024 crowded tokens' down products
// over 64 experts (170 tiles) 300 -> 216 us, gate/up over 128 experts 571 -> 516.
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
  const TileScan<BM> scan(offsets, E);
  int pick;
  if (p.by_tile) {
    const int tiles = scan.tiles(), rounds = (tiles + 8 * TILE_GROUP - 1) / (8 * TILE_GROUP);
    if (tiles == 0) return false;
    const int group = (tiles + 8 * rounds - 1) / (8 * rounds);  // equal ones, so that every XCD has as many tiles
    const int i = blockIdx.x >> 3, round = i / (group * p.n_tiles), in = i - round * group * p.n_tiles;
    t->nt = in / group;
    pick = (round * 8 + (blockIdx.x & 7)) * group + in % group;
  } else {
    const int id = xcd_order(blockIdx.x, gridDim.x);
    t->nt = id / p.tiles;
    pick = id - t->nt * p.tiles;
  }
  return scan.find(pick, &t->e, &t->row0, &t->rows);
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
//   11 rows                  1177 / 1184 / 1305 / -
//   16 rows, uniform         1294 / 1125 / 1122 / 1548;  24 rows (256): - / 815 / 741 / -
//   48 rows (128, crowded)   784 / 565 / 544 / 631
//   96 rows (64, crowded)    645 / 405 / 358 / 388
//   384 rows (16, 2048 x 512, crowded)  91 / 49 / 47 / 37
// 48 rows on four waves, each with twice the outputs, for eight: fewer reads of
// LDS and conversions a matrix step (48 rows crowded 502 -> 486, 24 rows 752 ->
// 741); 32 rows on four: 538 for 561 crowded, but 1211 for 1184 at 11 rows.
hipError_t launch_bs_gateup(const BsGateup& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k, E = a.E;
  if (n <= 4 * E) return launch_gateup<Tile<8, 1, 1, 1, 4, 1, 2>>(a, s);
  if (n <= 16 * E) return launch_gateup<Tile<8, 1, 1, 2, 2, 1, 2>>(a, s);
  if (n <= 160 * E) return launch_gateup<Tile<4, 1, 2, 3, 2, 1, 2>>(a, s);
  return launch_gateup<Tile<4, 2, 2, 4, 3, 1, 2>>(a, s);
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

// One or two tokens: one launch and no workspace.  A block owns 16 outputs of
// one token; its 16 waves share the K blocks (and, where two groups of waves or
// more have one for each, the routes), straight from memory with U routes
// requested at a time.  With U = 6 and more than 1024 inputs up to 6 routes are
// one round trip for each 2048 inputs, 7 to 12 are two and 13 to 16 three.  Column j of the matrix steps' activations is route
// j's row, for all routes at once; of the product with route j's weights column j
// is kept, so that a lane needs its own route's scales only and one accumulator
// serves every route.  The waves' sums are added in their order, then the routes
// weighted in theirs.  Bound by the weights, after two loads in a row (positions
// and offsets, then weights).
template <int U>
__global__ __launch_bounds__(1024) void bs_down_token_kernel(BsDown a) {
  constexpr int WAVES = 16;
  static_assert(TOPK_MAX_K == 16, "a column of the matrix step for each route");
  __shared__ f32x4_t part[WAVES][16][4];  // [wave][route][output / 4]
  __shared__ float route_y[16][16];
  __shared__ int route_row[16], route_e[16];
  __shared__ float route_wt[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16, t = blockIdx.y, KB = bs_blocks(a.f), DB = bs_blocks(a.d);
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
  const uint8_t* xp = a.hq + x_row * a.f;
  const float *hp = a.hs + x_row * KB, *sp = a.s_down + ((int64_t)e * DB + n0 / BS) * KB;
  const int G = KB >= WAVES ? 1 : WAVES / KB;  // groups of waves that share the routes
  const int g = KB >= WAVES ? 0 : wave / KB;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int jb = g; jb < (g < G ? a.k : 0); jb += G * U)
    for (int kb = KB >= WAVES ? wave : wave - g * KB; kb < KB; kb += WAVES) {
      const int k0 = kb * BS + 16 * quad;
      const bool in0 = k0 < a.f, in1 = k0 + 64 < a.f;  // past f: some code of the row, times 0
      const int c0 = in0 ? k0 : 0, c1 = in1 ? k0 + 64 : 0;
      i32x8_t w[U];
#pragma unroll
      for (int i = 0; i < U; i++) {
        const int j = jb + G * i;
        const bool on = j < a.k && (valid >> (j & 15) & 1);  // (else a buffer of no bytes)
        const int64_t at = ((int64_t)__builtin_amdgcn_readlane(e, j & 15) * a.d + n0) * a.f;
        const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.w_down + at, on ? 16 * a.f : 0);
        w[i] = join_pieces(buffer_load16(wbuf, r * a.f + c0), buffer_load16(wbuf, r * a.f + c1));
      }
      const i32x4_t zero = {0, 0, 0, 0};
      const i32x4_t x0 = *reinterpret_cast<const i32x4_t*>(xp + c0), x1 = *reinterpret_cast<const i32x4_t*>(xp + c1);
      const float hs = hp[kb], ws = sp[kb];
      __builtin_amdgcn_sched_barrier(0);  // (else the loads go between the matrix steps, to save registers)
      const float sc = hs * ws;
      F16Block xf;
      xf.set(join_pieces(in0 ? x0 : zero, in1 ? x1 : zero));
#pragma unroll
      for (int i = 0; i < U; i++) {
        const int j = jb + G * i;
        F16Block wf;
        wf.set(w[i]);
        const f32x4_t p = mfma_block(wf, xf);
#pragma unroll
        for (int q = 0; q < 4; q++) acc[q] = r == j ? __builtin_fmaf(p[q], sc, acc[q]) : acc[q];
      }
    }
  part[wave][r][quad] = acc;  // (0 for the routes of other groups)
  __syncthreads();
  const int j = threadIdx.x >> 4, n = threadIdx.x & 15;
  if (j < a.k) {
    float s = part[0][j][n >> 2][n & 3];
#pragma unroll
    for (int v = 1; v < WAVES; v++) s += part[v][j][n >> 2][n & 3];
    route_y[j][n] = s;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    float y = add;
#pragma unroll
    for (int i = 0; i < TOPK_MAX_K; i++)
      y = valid >> i & 1 ? __builtin_fmaf(route_wt[i], route_y[i][n], y) : y;
    a.y[out] = y;
  }
}

// Measured so / as products and a combine: 6 of 384 experts x 2048 x 4096, 1
// token 11.4 us, 2 tokens 22.3 / 25.9; 4 of 64 x 1408 x 2048, 2 tokens 8.0 / 11.7;
// but 4 tokens 45.1 / 44.9 and, where they share experts (16), 32.0 / 19.3.
constexpr int TOKEN_MAX_T = 2;

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
// 48 rows on four waves for eight: 64 rows, crowded 993 -> 952, uniform 970 -> 960
// (64 rows x 128 outputs, three blocks a CU: 965 and 926, but 56 for 48 at 500
// tokens over 64 experts x 1408 x 2000).
static hipError_t launch_down_products(const BsDown& a, hipStream_t s) {
  const int64_t n = (int64_t)a.T * a.k, E = a.E;
  if (n <= 2 * E) return launch_down<Tile<8, 1, 1, 1, 4, 1, 1>>(a, s);
  if (n <= 12 * E) return launch_down<Tile<8, 1, 2, 2, 2, 1, 1>>(a, s);
  if (n <= 200 * E) return launch_down<Tile<4, 1, 4, 3, 2, 1, 1>>(a, s);
  return launch_down<Tile<4, 2, 4, 4, 3, 1, 1>>(a, s);
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
