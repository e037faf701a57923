// Dense product of int8 matrices with a scale per row and per output channel.
#include "int8_tile.hpp"

namespace qmoe {

// Few rows (M <= 16): bound by the weights' bytes, each read once.  A block owns 16
// outputs and all rows, its 8 waves share K 128 inputs at a time; operands go straight
// to registers, U runs of 128 requested at a time, so that a call of a few MB is one
// round trip to memory.
template <int U, typename OUT>
__global__ __launch_bounds__(512) void i8_matmul_rows_kernel(I8Matmul a) {
  __shared__ i32x4_t part[8][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16, KB = bs_blocks(a.K);
  const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)min(16, a.N - n0) * a.K);
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq, (a.M - 1) * a.ldx + a.K);
  const uint32_t woff = r * a.K + 16 * quad;
  const uint32_t xoff = r < a.M ? (uint32_t)(r * a.ldx) + 16 * quad : BUFFER_OUT;
  // wave 0 stores: its scales are requested with the codes
  const int n = n0 + 4 * quad;
  const __amdgpu_buffer_rsrc_t xsbuf = buffer_of(a.xs, (int64_t)a.M * 4), wsbuf = buffer_of(a.ws, (int64_t)a.N * 4);
  const float xs = buffer_load4(xsbuf, wave == 0 ? r * 4 : BUFFER_OUT);
  f32x4_t ws;
#pragma unroll
  for (int q = 0; q < 4; q++) ws[q] = buffer_load4(wsbuf, wave == 0 ? (n + q) * 4 : BUFFER_OUT);
  i32x4_t acc = {0, 0, 0, 0};
  for (int k0 = wave; k0 < KB; k0 += 8 * U) {
    i32x4_t w[U][2], x[U][2];
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c = (k0 + 8 * u) * BS + 64 * h;
        const uint32_t o = c + 16 * quad < a.K ? c : BUFFER_OUT;
        w[u][h] = buffer_load16(wbuf, woff + o);
        x[u][h] = buffer_load16(xbuf, out_or_sum(xoff, o));
      }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int h = 0; h < 2; h++) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][h], x[u][h], acc, 0, 0, 0);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  i32x4_t y = part[0][lane];
#pragma unroll
  for (int u = 1; u < 8; u++) y += part[u][lane];
  const bool vec = a.ldy % 4 == 0;  // (y itself is 16-byte aligned)
  if (r < a.M) store4(static_cast<OUT*>(a.y) + r * a.ldy + n, i8_values(y, xs, ws), a.N - n, vec);
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
  i32x16_t acc[1][C::TN][C::TM];
  if (!i8_product<C>(
          lds, wbuf, wsbuf, a.K, xbuf, xsbuf, [&](int i) { return i < rows_m ? (uint32_t)(i * a.ldx) : BUFFER_OUT; },
          [&](int i) { return (uint32_t)(i * 4); }, (int)(blockIdx.y * KB / gridDim.y),
          (int)((blockIdx.y + 1) * KB / gridDim.y), acc))
    return;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, half = lane >> 5;
  const int wn = wave % C::WN, wm = wave / C::WN;
  if (gridDim.y > 1) {
    int* part = a.part + (int64_t)blockIdx.y * a.M * a.N;
#pragma unroll
    for (int j = 0; j < C::TM; j++) {
      const int m = m0 + (wm * C::TM + j) * 32 + r;
      if (m >= a.M) continue;
#pragma unroll
      for (int i = 0; i < C::TN; i++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const int n = n0 + (wn * C::TN + i) * 32 + 8 * g + 4 * half;
          store4(reinterpret_cast<float*>(part) + (int64_t)m * a.N + n, __builtin_bit_cast(f32x4_t, i8_run(acc[0][i][j], g)),
                 a.N - n, a.N % 4 == 0);
        }
    }
    return;
  }
  OUT* y = static_cast<OUT*>(a.y) + m0 * a.ldy + n0;
  if constexpr (C::KS == 1) {
    const uint32_t bits = (uint32_t)(a.ldy * sizeof(OUT));  // (y itself is 16-byte aligned)
    const int align = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
    i8_store<C>(lds, y, a.ldy, rows_m, rows_n, align, [&](int i, int j, int g, int n, float xs) {
      return i8_values(i8_run(acc[0][i][j], g), xs, i8_wscale<C>(lds, 0, n));
    });
  } else {
    // four outputs leave as one store where every row allows it
    const bool vec = a.ldy % 4 == 0;
#pragma unroll
    for (int j = 0; j < C::TM; j++) {
      const int mi = (wm * C::TM + j) * 32 + r;
      if (mi >= rows_m) continue;
      const float xs = i8_xscale<C>(lds, mi);
#pragma unroll
      for (int i = 0; i < C::TN; i++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const int ni = (wn * C::TN + i) * 32 + 8 * g + 4 * half;
          store4(y + mi * a.ldy + ni, i8_values(i8_run(acc[0][i][j], g), xs, i8_wscale<C>(lds, 0, ni)), rows_n - ni, vec);
        }
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

// Blocks that share a tile's K: four, with a launch more to add their sums, where the
// 32 x 32 tiles leave three quarters of the CUs idle and K is past 8192.  us for one
// and four: 33 x 256 x 16384 12.0 and 8.8, x 8192 8.1 and 7.9 (24 x 256: 8.1 and 7.7).
static int split_k(int M, int N, int K) { return K > 8192 && tile_count(M, N, 32, 32) <= 64 ? 4 : 1; }

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

template <typename OUT>
static hipError_t launch_rows(const I8Matmul& a, hipStream_t s) {
  auto* k = i8_matmul_rows_kernel<4, OUT>;
  const int pid = prof_begin("i8_matmul", s);
  QMOE_LAUNCH(k, dim3((a.N + 15) / 16), dim3(512), 0, s, a);
  prof_end(pid, s);
  return hipGetLastError();
}

// The variant: up to 16 rows straight from memory; else the tile (rows x outputs)
// that costs least, as a part for each begun round of tiles over the CUs and a part
// for the tiles themselves (more of them at work lower the clock).  Fitted to N = K =
// 4096, bf16 outputs, us at M rows (in brackets what the model says):
//    32 x 32, 8 wave groups share K   64 7.2 (6.5)    128 12.5 (13)
//    64 x 32, 4                       64 8.4 (8.1)    128 8.7 (8.6)    256 15.8 (17.2)
//    64 x 64, 2                       128 10.3 (9.8)  256 10.7 (10.7)  512 19.8 (21.4)   704 30.1 (31.6)
//    64 x 128                         384 13.8 (13.9) 512 14.8 (14.8)  640 28.2 (26.9)
//   128 x 128, four stages            640 19.8 (19.7) 768 20.3 (20.7)  1024 22.2 (22.8)  2048 45.1 (45.6)
//   128 x 128, two, two blocks a CU   1024 26.6 (26.5) 1500 32.8 (32.8) 2048 39.0 (39.0) 2800 59 (62)  5000 93 (104)
//   256 x 256                         2048 45.7 (45.5) 2800 48.4 (51.3) 4096 61.3 (61.0)  5000 110 (99)
// At K = 272, 1040, 2320, 4096 and 8192 with N = 4096 and 1300, M = 33 to 4096 and both
// output types the model's tile was the fastest (within 0.5 %) in 122 of 130 cases; else it was 1 to 7 %
// slower, in two of K = 272 11 and 14 % (128 x 4096 to bf16 4.8 and 4.4 us, 4096 x 4096
// to fp32 20.0 and 17.6).
// 8192 x 8192 x 8192 on 256 x 256: 441 to 479 (2.3 to 2.5 POP/s; the library's int8 product
// without scales 526).  There the card's power is the bound: 738 to 766 thousand cycles,
// the matrix units busy for 524 of them, at 1.6 to 1.7 GHz; tiles of 128 x 128 a wave (fewer
// reads of LDS) 927 thousand at 1.96 GHz in as much time (474), and the loop without its
// copies into LDS took 367.
// Rows against 32 x 32 tiles at M = 1, 8 and 16: 4096 x 4096 5.3, 6.0 and 6.6 for 6.6;
// 8192 x 8192 14.1, 15.3 and 17.8 for 13; 700 x 1040 3.8 for 4.9.
template <typename OUT>
static hipError_t launch_matmul(const I8Matmul& a, hipStream_t s) {
  const int parts = split_k(a.M, a.N, a.K);
  if (a.M <= 16 && a.N <= 4096 && parts == 1) return launch_rows<OUT>(a, s);
  static constexpr struct {
    int bm, bn, round;
    float begun, full;
  } TILES[7] = {{32, 32, 256, 5.8f, 0.7f},    {64, 32, 256, 7.6f, 1.0f},     {64, 64, 256, 8.8f, 1.9f},  {64, 128, 256, 11.2f, 3.6f},
                {128, 128, 256, 14.5f, 8.3f}, {128, 128, 512, 14.0f, 25.0f}, {256, 256, 256, 30.0f, 31.0f}};
  int best = 0;
  float least = INFINITY;
  for (int i = 0; i < (parts == 1 ? 7 : 1); i++) {
    const auto& x = TILES[i];
    const int64_t n = tile_count(a.M, a.N, x.bm, x.bn);
    const float cost = x.begun * (float)((n + x.round - 1) / x.round) + x.full * (float)n / (float)x.round;
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  switch (best) {
    case 0: return launch_tile<I8Tile<1, 1, 1, 1, 64, 3, 8, 1>, OUT>(a, s, parts);
    case 1: return launch_tile<I8Tile<1, 2, 1, 1, 128, 3, 4, 1>, OUT>(a, s);
    case 2: return launch_tile<I8Tile<2, 2, 1, 1, 128, 4, 2, 1>, OUT>(a, s);
    case 3: return launch_tile<I8Tile<4, 2, 1, 1, 128, 4, 1, 1>, OUT>(a, s);
    case 4: return launch_tile<I8Tile<4, 2, 1, 2, 64, 4, 1, 1>, OUT>(a, s);
    case 5: return launch_tile<I8Tile<4, 2, 1, 2, 128, 2, 1, 1>, OUT>(a, s);
    default: return launch_tile<I8Tile<4, 2, 2, 4, 128, 2, 1, 1>, OUT>(a, s);
  }
}

hipError_t launch_i8_matmul(const I8Matmul& a, hipStream_t s) {
  return a.y_dtype == X_BF16 ? launch_matmul<uint16_t>(a, s) : launch_matmul<float>(a, s);
}

}  // namespace qmoe
