// Dense product of block-scaled E4M3 matrices.
#include "blockscale_tile.hpp"

namespace qmoe {

// Few rows (M <= 16 TM): bound by the weights' bytes, each read once.  A block
// owns 16 TN outputs and all rows, its 8 waves share the K blocks (wave w takes
// blocks w, w + 8, ...) and add their sums in the order of the waves; operands
// go straight to registers, U blocks requested at a time, so that a call of a
// few MB is one round trip to memory.
template <int TN, int TM, int U, typename OUT>
__global__ __launch_bounds__(512) void bs_matmul_rows_kernel(BsMatmul a) {
  __shared__ f32x4_t part[8][TN * TM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16 * TN, KB = bs_blocks(a.K);
  const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)min(16 * TN, a.N - n0) * a.K);
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq, (a.M - 1) * a.ldx + a.K);
  const __amdgpu_buffer_rsrc_t sbuf = buffer_of(a.xs, (int64_t)a.M * KB * 4);
  const float* wsr = a.ws + (int64_t)(n0 / BS) * KB;
  const uint32_t woff = r * a.K + 16 * quad;
  uint32_t xoff[TM], soff[TM];
#pragma unroll
  for (int j = 0; j < TM; j++) {
    const int m = 16 * j + r;
    xoff[j] = m < a.M ? (uint32_t)(m * a.ldx) + 16 * quad : BUFFER_OUT;
    soff[j] = m * KB * 4;
  }
  f32x4_t acc[TN][TM] = {};
  for (int k0 = wave; k0 < KB; k0 += 8 * U) {
    i32x8_t w[U][TN], x[U][TM];
    float wsc[U], xsc[U][TM];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int kb = k0 + 8 * u, c = kb * BS + 16 * quad;
      const uint32_t o0 = c < a.K ? kb * BS : BUFFER_OUT, o1 = c + 64 < a.K ? kb * BS + 64 : BUFFER_OUT;
#pragma unroll
      for (int i = 0; i < TN; i++)
        w[u][i] = join_pieces(buffer_load16(wbuf, woff + 16 * i * a.K + o0), buffer_load16(wbuf, woff + 16 * i * a.K + o1));
      wsc[u] = kb < KB ? wsr[kb] : 0.0f;
#pragma unroll
      for (int j = 0; j < TM; j++) {
        x[u][j] = join_pieces(buffer_load16(xbuf, out_or_sum(xoff[j], o0)), buffer_load16(xbuf, out_or_sum(xoff[j], o1)));
        xsc[u][j] = buffer_load4(sbuf, kb < KB ? soff[j] + kb * 4 : BUFFER_OUT);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      F16Block wf[TN];
#pragma unroll
      for (int i = 0; i < TN; i++) wf[i].set(w[u][i]);
#pragma unroll
      for (int j = 0; j < TM; j++) {
        F16Block xf;
        xf.set(x[u][j]);
        const float sc = xsc[u][j] * wsc[u];
#pragma unroll
        for (int i = 0; i < TN; i++) {
          const f32x4_t p = mfma_block(wf[i], xf);
#pragma unroll
          for (int q = 0; q < 4; q++) acc[i][j][q] = __builtin_fmaf(p[q], sc, acc[i][j][q]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TN * TM; i++) part[wave][i][lane] = acc[i / TM][i % TM];
  __syncthreads();
  const int v = threadIdx.x >> 6;  // wave v adds tile v
  if (v >= TN * TM) return;
  f32x4_t y = part[0][v][lane];
#pragma unroll
  for (int u = 1; u < 8; u++) y += part[u][v][lane];
  const int m = 16 * (v % TM) + r, n = n0 + 16 * (v / TM) + 4 * quad;
  const bool vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(OUT) - 1)) == 0;
  if (m < a.M) store4(static_cast<OUT*>(a.y) + m * a.ldy + n, y, a.N - n, vec);
}

// grid.y > 1: K is shared by that many blocks of a tile; each leaves its sums in
// a.part, and bs_matmul_sum_kernel adds them in their order.
template <class C, typename OUT>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void bs_matmul_tile_kernel(BsMatmul a, int n_tiles, int m_tiles) {
  extern __shared__ __align__(1024) uint8_t lds[];
  // an XCD (block id mod 8) takes a contiguous eighth of the tiles, in strips
  // of 8 M tiles so that neighbours in time share operands in its L2
  const int id = xcd_order(blockIdx.x, n_tiles * m_tiles);
  const int strip = id / (8 * n_tiles), in_strip = id - strip * 8 * n_tiles;
  const int strip_m = min(8, m_tiles - 8 * strip);
  const int mt = 8 * strip + in_strip % strip_m, nt = in_strip / strip_m;
  const int n0 = nt * C::BN, m0 = mt * C::BM;
  const int KB = bs_blocks(a.K);
  const int rows_n = min(C::BN, a.N - n0), rows_m = min(C::BM, a.M - m0);
  const __amdgpu_buffer_rsrc_t wbuf[1] = {buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)rows_n * a.K)};
  const float* const ws[1] = {a.ws + (int64_t)(n0 / BS) * KB};
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq + m0 * a.ldx, (rows_m - 1) * a.ldx + a.K);
  const __amdgpu_buffer_rsrc_t sbuf = buffer_of(a.xs + (int64_t)m0 * KB, (int64_t)rows_m * KB * 4);
  f32x4_t acc[1][C::TN][C::TM];
  if (!tile_product<C>(
          lds, wbuf, ws, bs_blocks(a.N) - n0 / BS, a.K, xbuf, sbuf,
          [&](int i) { return i < rows_m ? (uint32_t)(i * a.ldx) : BUFFER_OUT; },
          [&](int i) { return (uint32_t)(i * KB * 4); }, (int)(blockIdx.y * KB / gridDim.y),
          (int)((blockIdx.y + 1) * KB / gridDim.y), acc))
    return;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, quad = lane >> 4;
  const int wn = wave % C::WN, wm = wave / C::WN;
  if (gridDim.y > 1) {
    float* part = a.part + (int64_t)blockIdx.y * a.M * a.N;
#pragma unroll
    for (int j = 0; j < C::TM; j++) {
      const int m = m0 + (wm * C::TM + j) * 16 + r;
      if (m >= a.M) continue;
#pragma unroll
      for (int i = 0; i < C::TN; i++) {
        const int n = n0 + (wn * C::TN + i) * 16 + 4 * quad;
        store4(part + (int64_t)m * a.N + n, acc[0][i][j], a.N - n, a.N % 4 == 0);
      }
    }
    return;
  }
  OUT* y = static_cast<OUT*>(a.y);
  // four outputs leave as one store where every row allows it
  const bool vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(OUT) - 1)) == 0;
#pragma unroll
  for (int j = 0; j < C::TM; j++) {
    const int m = m0 + (wm * C::TM + j) * 16 + r;
    if (m >= a.M) continue;
    OUT* row = y + m * a.ldy;
#pragma unroll
    for (int i = 0; i < C::TN; i++) {
      const int n = n0 + (wn * C::TN + i) * 16 + 4 * quad;
      store4(row + n, acc[0][i][j], a.N - n, vec);
    }
  }
}

template <typename OUT>
__global__ __launch_bounds__(256) void bs_matmul_sum_kernel(BsMatmul a, int parts) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, size = (int64_t)a.M * a.N;
  if (i >= size) return;
  float s = a.part[i];
  for (int p = 1; p < parts; p++) s += a.part[p * size + i];
  const int64_t m = i / a.N;
  OUT* y = static_cast<OUT*>(a.y) + m * a.ldy + (i - m * a.N);
  if constexpr (sizeof(OUT) == 2)
    *y = bf16_bits(s);
  else
    *y = s;
}

static int64_t tile_count(int M, int N, int bm, int bn) {
  return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

// Blocks that share a tile's K: where the 64 x 64 tiles leave half of the CUs
// idle and K is long, so many that each still has 8 blocks of 128.  Measured
// with the sum's launch, fp16 steps, us alone and shared: 100 x 300 x 8192 26.2
// and 10.4, 250 x 1000 x 8192 26.8 and 13.1, 250 x 2000 x 8192 25.5 and 18.2,
// 128 x 4096 x 4096 14.7 and 13.2; of 17 blocks 10.0 and 11.2 (250 x 2000).
static int split_k(int M, int N, int K) {
  const int64_t tiles = tile_count(M, N, 64, 64);
  const int KB = bs_blocks(K);
  if (M <= 32 || tiles > 128 || KB < 32) return 1;
  const int64_t s = 256 / tiles < KB / 8 ? 256 / tiles : KB / 8;
  return (int)s;
}

size_t bs_matmul_ws(int M, int N, int K) {
  const int s = split_k(M, N, K);
  return s > 1 ? (size_t)s * M * N * 4 : 0;
}

template <int WN, int WM, int TN, int TM, int ST, int KS, typename OUT>
static hipError_t launch_tile(const BsMatmul& a, hipStream_t s, int parts = 1) {
  using C = Tile<WN, WM, TN, TM, ST, KS, 1>;
  const int n_tiles = (a.N + C::BN - 1) / C::BN, m_tiles = (a.M + C::BM - 1) / C::BM;
  auto* k = bs_matmul_tile_kernel<C, OUT>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  int pid = prof_begin("bs_matmul", s);
  QMOE_LAUNCH(k, dim3((unsigned)(n_tiles * m_tiles), parts), dim3(C::THREADS), C::LDS, s, a, n_tiles, m_tiles);
  prof_end(pid, s);
  if (parts > 1) {
    if ((e = hipGetLastError()) != hipSuccess) return e;
    pid = prof_begin("bs_matmul_sum", s);
    QMOE_LAUNCH(bs_matmul_sum_kernel<OUT>, dim3((unsigned)(((int64_t)a.M * a.N + 255) / 256)), dim3(256), 0, s, a, parts);
    prof_end(pid, s);
  }
  return hipGetLastError();
}

template <int TN, int TM, int U, typename OUT>
static hipError_t launch_rows(const BsMatmul& a, hipStream_t s) {
  auto* k = bs_matmul_rows_kernel<TN, TM, U, OUT>;
  const int pid = prof_begin("bs_matmul", s);
  QMOE_LAUNCH(k, dim3((a.N + 16 * TN - 1) / (16 * TN)), dim3(512), 0, s, a);
  prof_end(pid, s);
  return hipGetLastError();
}

// The variant: by rows, then the largest tile of which there are enough for
// the 256 CUs.  Measured on both sides of each step, N = K = 4096 and fp32
// outputs unless given (us; bf16 outputs take up to 4 % less):
//   M 32: rows 9.9;  33: 64 x 64 tiles 9.8;  64: rows 15.3, tiles 10.4
//   M 32, 32 outputs a block instead of 16: 11.1 and 9.9, at N = K = 8192 22.6 and 30.2
//   M 128 (64 tiles of 128 x 64): 20.2 on them, 15.2 on 64 x 64, whose K is
//     shared besides: 12.6
//   M 1000, N 1100, K 2064 (144): 15.3 on 128 x 64, 19.3 on 64 x 64 (288: a
//     second round of few), 13.0 on 64 x 96 (198); 700 x 1500 x 1040 9.6 and
//     8.3, but M 512 (384 tiles of 64 x 96) 23.5 and 34.3
//   64 x 64 and 64 x 96 with three groups and two stages, and with two groups:
//     512 x 2048 x 4096 14.8 and 15.4, 512 x 1024 x 1040 6.4 and 7.0, 64 x
//     4096 x 2048 8.7 and 9.3; 64 x 96 13.0 and 13.6, 1500 x 700 x 8192 30.9 and 32.7
//   M 512 (128 tiles of 128 x 128): 32.0 on them, 21.9 to 22.6 on 128 x 64
//   M 1024 (256): 34.6 on 128 x 128 with two groups, 38.4 with one group and
//     two stages, 42.6 on 128 x 64
//   M 2048 (512): 71.0 with one group and two stages, 66.9 with two groups
//   M 4096 (1024): 123 on 128 x 128, 132 with two groups
//   M = N = K = 8192 to bf16: 914 to 927 (1.2 PFLOP/s; the library's 16-bit
//     product of 8192^3, without scales, reaches 1.46)
template <typename OUT>
static hipError_t launch_matmul(const BsMatmul& a, hipStream_t s) {
  if (a.M <= 16) return launch_rows<1, 1, 4, OUT>(a, s);
  if (a.M <= 32) return a.N >= 6144 ? launch_rows<2, 2, 2, OUT>(a, s) : launch_rows<1, 2, 2, OUT>(a, s);
  auto tiles = [&](int bn, int bm) { return tile_count(a.M, a.N, bm, bn); };
  const int parts = split_k(a.M, a.N, a.K);
  if (tiles(128, 128) >= 768) return launch_tile<2, 2, 4, 4, 2, 1, OUT>(a, s);
  if (tiles(128, 128) >= 192) return launch_tile<2, 2, 4, 4, 2, 2, OUT>(a, s);
  if (tiles(128, 64) >= 128) {
    // one round of 64 x 96 tiles where they are enough for the CUs but not more
    if (tiles(64, 96) <= 256) return launch_tile<2, 2, 2, 3, 2, 3, OUT>(a, s);
    return launch_tile<2, 2, 4, 2, 3, 2, OUT>(a, s);
  }
  return launch_tile<2, 2, 2, 2, 2, 3, OUT>(a, s, parts);
}

hipError_t launch_bs_matmul(const BsMatmul& a, hipStream_t s) {
  return a.y_dtype == X_BF16 ? launch_matmul<uint16_t>(a, s) : launch_matmul<float>(a, s);
}

}  // namespace qmoe
