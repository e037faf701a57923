// Dense product of int8 matrices with a scale per row and per output channel.
#include "int8_tile.hpp"

namespace qmoe {

// Few rows (M <= 16 TM): bound by the weights' bytes, each read once.  A block
// owns 16 TN outputs and all rows, its 8 waves share K 128 inputs at a time;
// operands go straight to registers, U runs of 128 requested at a time, so that a
// call of a few MB is one round trip to memory.
template <int TN, int TM, int U, typename OUT>
__global__ __launch_bounds__(512) void i8_matmul_rows_kernel(I8Matmul a) {
  using Step = I8Step<16>;
  __shared__ i32x4_t part[8][TN * TM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16 * TN, KB = bs_blocks(a.K);
  const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)min(16 * TN, a.N - n0) * a.K);
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq, (a.M - 1) * a.ldx + a.K);
  const uint32_t woff = r * a.K + 16 * quad;
  uint32_t xoff[TM];
#pragma unroll
  for (int j = 0; j < TM; j++) xoff[j] = 16 * j + r < a.M ? (uint32_t)((16 * j + r) * a.ldx) + 16 * quad : BUFFER_OUT;
  // wave v stores tile v: its scales are requested with the codes
  const int m = 16 * (wave % TM) + r, n = n0 + 16 * (wave / TM) + 4 * quad;
  const __amdgpu_buffer_rsrc_t xsbuf = buffer_of(a.xs, (int64_t)a.M * 4), wsbuf = buffer_of(a.ws, (int64_t)a.N * 4);
  const float xs = buffer_load4(xsbuf, wave < TN * TM ? m * 4 : BUFFER_OUT);
  f32x4_t ws;
#pragma unroll
  for (int q = 0; q < 4; q++) ws[q] = buffer_load4(wsbuf, wave < TN * TM ? (n + q) * 4 : BUFFER_OUT);
  typename Step::Acc acc[TN][TM] = {};
  for (int k0 = wave; k0 < KB; k0 += 8 * U) {
    i32x4_t w[U][TN][2], x[U][TM][2];
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c = (k0 + 8 * u) * BS + 64 * h;
        const uint32_t o = c + 16 * quad < a.K ? c : BUFFER_OUT;
#pragma unroll
        for (int i = 0; i < TN; i++) w[u][i][h] = buffer_load16(wbuf, woff + 16 * i * a.K + o);
#pragma unroll
        for (int j = 0; j < TM; j++) x[u][j][h] = buffer_load16(xbuf, out_or_sum(xoff[j], o));
      }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < TN; i++)
#pragma unroll
          for (int j = 0; j < TM; j++) acc[i][j] = Step::mul(w[u][i][h], x[u][j][h], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < TN * TM; i++) part[wave][i][lane] = acc[i / TM][i % TM];
  __syncthreads();
  if (wave >= TN * TM) return;
  i32x4_t y = part[0][wave][lane];
#pragma unroll
  for (int u = 1; u < 8; u++) y += part[u][wave][lane];
  const bool vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(OUT) - 1)) == 0;
  if (m < a.M) store4(static_cast<OUT*>(a.y) + m * a.ldy + n, i8_values(y, xs, ws), a.N - n, vec);
}

// grid.y > 1: K is shared by that many blocks of a tile; each leaves its sums in
// a.part, and i8_matmul_sum_kernel adds them.
template <class C, typename OUT>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void i8_matmul_tile_kernel(I8Matmul a, int n_tiles, int m_tiles) {
  extern __shared__ __align__(1024) uint8_t lds[];
  // an XCD (block id mod 8) takes a contiguous eighth of the tiles, in strips
  // of 8 M tiles so that neighbours in time share operands in its L2
  const int id = xcd_order(blockIdx.x, n_tiles * m_tiles);
  const int strip = id / (8 * n_tiles), in_strip = id - strip * 8 * n_tiles;
  const int strip_m = min(8, m_tiles - 8 * strip);
  const int mt = 8 * strip + in_strip % strip_m, nt = in_strip / strip_m;
  const int n0 = nt * C::BN, m0 = mt * C::BM;
  const int KB = (a.K + C::BK - 1) / C::BK;
  const int rows_n = min(C::BN, a.N - n0), rows_m = min(C::BM, a.M - m0);
  const __amdgpu_buffer_rsrc_t wbuf[1] = {buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)rows_n * a.K)};
  const __amdgpu_buffer_rsrc_t wsbuf[1] = {buffer_of(a.ws + n0, (int64_t)rows_n * 4)};
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq + m0 * a.ldx, (rows_m - 1) * a.ldx + a.K);
  const __amdgpu_buffer_rsrc_t xsbuf = buffer_of(a.xs + m0, (int64_t)rows_m * 4);
  typename C::Acc acc[1][C::TN][C::TM];
  if (!i8_product<C>(
          lds, wbuf, wsbuf, a.K, xbuf, xsbuf, [&](int i) { return i < rows_m ? (uint32_t)(i * a.ldx) : BUFFER_OUT; },
          [&](int i) { return (uint32_t)(i * 4); }, (int)(blockIdx.y * KB / gridDim.y),
          (int)((blockIdx.y + 1) * KB / gridDim.y), acc))
    return;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & (C::MF - 1), half = lane / C::MF;
  const int wn = wave % C::WN, wm = wave / C::WN;
  if (gridDim.y > 1) {
    int* part = a.part + (int64_t)blockIdx.y * a.M * a.N;
#pragma unroll
    for (int j = 0; j < C::TM; j++) {
      const int m = m0 + (wm * C::TM + j) * C::MF + r;
      if (m >= a.M) continue;
#pragma unroll
      for (int i = 0; i < C::TN; i++)
#pragma unroll
        for (int g = 0; g < C::Step::RUNS; g++) {
          const int n = n0 + (wn * C::TN + i) * C::MF + 8 * g + 4 * half;
          store4(reinterpret_cast<float*>(part) + (int64_t)m * a.N + n, __builtin_bit_cast(f32x4_t, i8_run(acc[0][i][j], g)),
                 a.N - n, a.N % 4 == 0);
        }
    }
    return;
  }
  OUT* y = static_cast<OUT*>(a.y);
  // four outputs leave as one store where every row allows it
  const bool vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(OUT) - 1)) == 0;
#pragma unroll
  for (int j = 0; j < C::TM; j++) {
    const int mi = (wm * C::TM + j) * C::MF + r, m = m0 + mi;
    if (m >= a.M) continue;
    const float xs = i8_xscale<C>(lds, mi);
    OUT* row = y + m * a.ldy;
#pragma unroll
    for (int i = 0; i < C::TN; i++)
#pragma unroll
      for (int g = 0; g < C::Step::RUNS; g++) {
        const int ni = (wn * C::TN + i) * C::MF + 8 * g + 4 * half;
        store4(row + n0 + ni, i8_values(i8_run(acc[0][i][j], g), xs, i8_wscale<C>(lds, 0, ni)), a.N - n0 - ni, vec);
      }
  }
}

template <typename OUT>
__global__ __launch_bounds__(256) void i8_matmul_sum_kernel(I8Matmul a, int parts) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, size = (int64_t)a.M * a.N;
  if (i >= size) return;
  int s = a.part[i];
  for (int p = 1; p < parts; p++) s += a.part[p * size + i];
  const int64_t m = i / a.N, n = i - m * a.N;
  const float v = ((float)s * a.xs[m]) * a.ws[n];
  OUT* y = static_cast<OUT*>(a.y) + m * a.ldy + n;
  if constexpr (sizeof(OUT) == 2)
    *y = bf16_bits(v);
  else
    *y = v;
}

static int64_t tile_count(int M, int N, int bm, int bn) {
  return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

static int split_k(int M, int N, int K) {
  const int64_t tiles = tile_count(M, N, 64, 64);
  const int KB = bs_blocks(K);
  if (M <= 32 || tiles > 128 || KB < 32) return 1;
  const int64_t s = 256 / tiles < KB / 8 ? 256 / tiles : KB / 8;
  return (int)s;
}

size_t i8_matmul_ws(int M, int N, int K) {
  const int s = split_k(M, N, K);
  return s > 1 ? (size_t)s * M * N * 4 : 0;
}

template <class C, typename OUT>
static hipError_t launch_tile(const I8Matmul& a, hipStream_t s, int parts = 1) {
  const int n_tiles = (a.N + C::BN - 1) / C::BN, m_tiles = (a.M + C::BM - 1) / C::BM;
  auto* k = i8_matmul_tile_kernel<C, OUT>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  int pid = prof_begin("i8_matmul", s);
  QMOE_LAUNCH(k, dim3((unsigned)(n_tiles * m_tiles), parts), dim3(C::THREADS), C::LDS, s, a, n_tiles, m_tiles);
  prof_end(pid, s);
  if (parts > 1) {
    if ((e = hipGetLastError()) != hipSuccess) return e;
    pid = prof_begin("i8_matmul_sum", s);
    QMOE_LAUNCH(i8_matmul_sum_kernel<OUT>, dim3((unsigned)(((int64_t)a.M * a.N + 255) / 256)), dim3(256), 0, s, a, parts);
    prof_end(pid, s);
  }
  return hipGetLastError();
}

template <int TN, int TM, int U, typename OUT>
static hipError_t launch_rows(const I8Matmul& a, hipStream_t s) {
  auto* k = i8_matmul_rows_kernel<TN, TM, U, OUT>;
  const int pid = prof_begin("i8_matmul", s);
  QMOE_LAUNCH(k, dim3((a.N + 16 * TN - 1) / (16 * TN)), dim3(512), 0, s, a);
  prof_end(pid, s);
  return hipGetLastError();
}

template <typename OUT>
static hipError_t launch_matmul(const I8Matmul& a, hipStream_t s) {
  if (a.M <= 16) return launch_rows<1, 1, 4, OUT>(a, s);
  if (a.M <= 32) return launch_rows<1, 2, 2, OUT>(a, s);
  auto tiles = [&](int bn, int bm) { return tile_count(a.M, a.N, bm, bn); };
  if (tiles(256, 256) >= 192) return launch_tile<I8Tile<32, 2, 2, 4, 4, 64, 4, 1, 1>, OUT>(a, s);
  if (tiles(128, 128) >= 128) return launch_tile<I8Tile<32, 2, 2, 2, 2, 128, 2, 2, 1>, OUT>(a, s);
  return launch_tile<I8Tile<32, 2, 2, 1, 1, 128, 2, 3, 1>, OUT>(a, s, split_k(a.M, a.N, a.K));
}

hipError_t launch_i8_matmul(const I8Matmul& a, hipStream_t s) {
  return a.y_dtype == X_BF16 ? launch_matmul<uint16_t>(a, s) : launch_matmul<float>(a, s);
}

}  // namespace qmoe
