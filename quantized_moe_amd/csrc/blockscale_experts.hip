// The routed experts' products on block-scaled E4M3 weights: gate/up with
// SwiGLU and requantisation, down with each token's weighted sum.
#include "blockscale.hpp"

namespace qmoe {

__device__ __forceinline__ i32x8_t load_frag(const uint8_t* row, bool ok, int kb, int K, int quad) {
  const i32x4_t z = {0, 0, 0, 0};
  const int k0 = kb * BS + 16 * quad, k1 = k0 + 64;
  const i32x4_t a = ok && k0 < K ? *reinterpret_cast<const i32x4_t*>(row + k0) : z;
  const i32x4_t b = ok && k1 < K ? *reinterpret_cast<const i32x4_t*>(row + k1) : z;
  return join_pieces(a, b);
}

// Simplest form: a block owns 16 bucket rows of one expert and one group of
// 128 hidden columns (8 waves of 16), so the group's maximum stays in it.
__global__ __launch_bounds__(512) void bs_gateup_kernel(BsGateup a, int n_tiles) {
  __shared__ uint32_t smax[8][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, quad = lane >> 4;
  const int nt = blockIdx.x % n_tiles;
  int e, row0, rows;
  if (!find_tile(a.offsets, a.E, 16, blockIdx.x / n_tiles, &e, &row0, &rows)) return;
  const int KB = bs_blocks(a.d), FB = bs_blocks(a.f);
  const int n0 = nt * BS + wave * 16;
  const bool rok = r < rows, nok = n0 + r < a.f;
  const int64_t t = rok ? a.perm[row0 + r] / a.k : 0;
  const uint8_t* xrow = a.xq + t * a.d;
  const int64_t woff = ((int64_t)e * a.f + n0 + r) * a.d, soff = ((int64_t)e * FB + nt) * KB;
  f32x4_t g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
  for (int kb = 0; kb < KB; kb++) {
    const i32x8_t x = load_frag(xrow, rok, kb, a.d, quad);
    const f32x4_t pg = mfma_block(load_frag(a.w_gate + woff, nok, kb, a.d, quad), x);
    const f32x4_t pu = mfma_block(load_frag(a.w_up + woff, nok, kb, a.d, quad), x);
    const float xsc = rok ? a.xs[t * KB + kb] : 0.0f;
    const float sg = xsc * a.s_gate[soff + kb], su = xsc * a.s_up[soff + kb];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      g[i] = __builtin_fmaf(pg[i], sg, g[i]);
      u[i] = __builtin_fmaf(pu[i], su, u[i]);
    }
  }
  float h[4];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    h[i] = silu(g[i]) * u[i];
    if (n0 + 4 * quad + i < a.f) mx = max(mx, abs_bits(h[i]));
  }
  mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
  mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
  if (quad == 0) smax[wave][r] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; w++) mx = max(mx, smax[w][r]);
  if (!rok) return;
  const float sc = bs_scale(mx);
  const int64_t row = row0 + r;
  if (n0 + 4 * quad < a.f)  // f is a multiple of 16
    *reinterpret_cast<uint32_t*>(a.hq + row * a.f + n0 + 4 * quad) =
        mx >= 0x7f800000u ? 0u : e4m3x4(h[0] / sc, h[1] / sc, h[2] / sc, h[3] / sc);
  if (wave == 0 && quad == 0) a.hs[row * FB + nt] = sc;
}

hipError_t launch_bs_gateup(const BsGateup& a, hipStream_t s) {
  const int n_tiles = bs_blocks(a.f);
  const int64_t tiles = max_tiles((int64_t)a.T * a.k, a.E, 16);
  QMOE_LAUNCH(bs_gateup_kernel, dim3((unsigned)(tiles * n_tiles)), dim3(512), 0, s, a, n_tiles);
  return hipGetLastError();
}

// ye[r][n] = (D_e h_r)[n] for the bucket rows.
__global__ __launch_bounds__(256) void bs_down_kernel(BsDown a, int n_tiles) {
  const int lane = threadIdx.x & 63, r = lane & 15, quad = lane >> 4;
  const int nt = blockIdx.x % n_tiles;
  int e, row0, rows;
  if (!find_tile(a.offsets, a.E, 16, blockIdx.x / n_tiles, &e, &row0, &rows)) return;
  const int KB = bs_blocks(a.f), DB = bs_blocks(a.d);
  const int n0 = nt * 64 + (threadIdx.x >> 6) * 16;
  if (n0 >= a.d) return;
  const bool rok = r < rows;
  const int64_t row = row0 + (rok ? r : 0);
  const int64_t woff = ((int64_t)e * a.d + n0 + r) * a.f, soff = ((int64_t)e * DB + n0 / BS) * KB;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = 0; kb < KB; kb++) {
    const f32x4_t p = mfma_block(load_frag(a.w_down + woff, n0 + r < a.d, kb, a.f, quad),
                                 load_frag(a.hq + row * a.f, rok, kb, a.f, quad));
    const float sc = a.hs[row * KB + kb] * a.s_down[soff + kb];
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(p[i], sc, acc[i]);
  }
  if (rok && n0 + 4 * quad < a.d) *reinterpret_cast<f32x4_t*>(a.ye + row * a.d + n0 + 4 * quad) = acc;
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
    if (p >= a.T * a.k) continue;  // a route without a place
    const float w = a.wt[t * a.k + j];
    const f32x4_t v = reinterpret_cast<const f32x4_t*>(a.ye)[(int64_t)p * d4 + c];
#pragma unroll
    for (int q = 0; q < 4; q++) y[q] = __builtin_fmaf(w, v[q], y[q]);
  }
  reinterpret_cast<f32x4_t*>(a.y)[i] = y;
}

size_t bs_down_ws(int T, int k, int d) { return (size_t)T * k * d * 4; }

hipError_t launch_bs_down(const BsDown& a, hipStream_t s) {
  const int n_tiles = (a.d + 63) / 64;
  const int64_t tiles = max_tiles((int64_t)a.T * a.k, a.E, 16);
  int pid = prof_begin("bs_down", s);
  QMOE_LAUNCH(bs_down_kernel, dim3((unsigned)(tiles * n_tiles)), dim3(256), 0, s, a, n_tiles);
  prof_end(pid, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  pid = prof_begin("bs_combine", s);
  QMOE_LAUNCH(bs_combine_kernel, dim3((unsigned)(((int64_t)a.T * (a.d / 4) + 255) / 256)), dim3(256), 0, s, a);
  prof_end(pid, s);
  return hipGetLastError();
}

}  // namespace qmoe
