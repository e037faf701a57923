// Dense product of block-scaled E4M3 matrices.
#include "blockscale.hpp"

namespace qmoe {

// Few rows (M <= 16 TM): bound by the weights' bytes, each read once.  A block
// owns 16 outputs and all rows, its 8 waves share the K blocks (wave w takes
// blocks w, w + 8, ...) and add their sums in the order of the waves; operands
// go straight to registers, U blocks requested at a time, so that a call of a
// few MB is one round trip to memory.
template <int TM, int U, typename OUT>
__global__ __launch_bounds__(512) void bs_matmul_rows_kernel(BsMatmul a) {
  __shared__ f32x4_t part[8][TM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16, KB = bs_blocks(a.K);
  const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)min(16, a.N - n0) * a.K);
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
  f32x4_t acc[TM] = {};
  for (int k0 = wave; k0 < KB; k0 += 8 * U) {
    i32x8_t w[U], x[U][TM];
    float wsc[U], xsc[U][TM];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int kb = k0 + 8 * u, c = kb * BS + 16 * quad;
      const uint32_t o0 = c < a.K ? kb * BS : BUFFER_OUT, o1 = c + 64 < a.K ? kb * BS + 64 : BUFFER_OUT;
      w[u] = join_pieces(buffer_load16(wbuf, woff + o0), buffer_load16(wbuf, woff + o1));
      wsc[u] = kb < KB ? wsr[kb] : 0.0f;
#pragma unroll
      for (int j = 0; j < TM; j++) {
        x[u][j] = join_pieces(buffer_load16(xbuf, out_or_sum(xoff[j], o0)), buffer_load16(xbuf, out_or_sum(xoff[j], o1)));
        xsc[u][j] = buffer_load4(sbuf, kb < KB ? soff[j] + kb * 4 : BUFFER_OUT);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      F16Block wf;
      wf.set(w[u]);
#pragma unroll
      for (int j = 0; j < TM; j++) {
        F16Block xf;
        xf.set(x[u][j]);
        const f32x4_t p = mfma_block(wf, xf);
        const float sc = xsc[u][j] * wsc[u];
#pragma unroll
        for (int q = 0; q < 4; q++) acc[j][q] = __builtin_fmaf(p[q], sc, acc[j][q]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TM; j++) part[wave][j][lane] = acc[j];
  __syncthreads();
  const int j = threadIdx.x >> 6;  // wave j adds tile j
  if (j >= TM) return;
  f32x4_t y = part[0][j][lane];
#pragma unroll
  for (int v = 1; v < 8; v++) y += part[v][j][lane];
  const int m = 16 * j + r, n = n0 + 4 * quad;
  const bool vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(OUT) - 1)) == 0;
  if (m < a.M) store4(static_cast<OUT*>(a.y) + m * a.ldy + n, y, a.N - n, vec);
}

// Tiled form: WN x WM waves, each TN x TM tiles of 16 outputs x 16 rows.  The
// operands of a block of 128 inputs go to LDS by asynchronous copies while the
// STAGES - 1 blocks before it are multiplied; 16-byte piece p of row i lies at place p ^ (i %
// 8), so the 8 rows that a read touches at once are in different banks.
// KS groups of such waves share the K blocks (group g takes blocks g, g + KS,
// ...), each with stages of its own, and add their sums in the order of the
// groups: where tiles are few, a CU has more waves and half the steps.
// EXACT: fp16 steps (fp32 outputs); else the unit's E4M3 steps, twice as fast.
template <int WN, int WM, int TN, int TM, int ST, int KS, bool EXACT>
struct Tile {
  static constexpr int STAGES = ST;
  static constexpr int BN = WN * TN * 16, BM = WM * TM * 16, WAVES = WN * WM, THREADS = 64 * WAVES * KS;
  static constexpr int W_BYTES = BN * BS, X_BYTES = BM * BS, S_BYTES = BM * 4;
  static constexpr int STAGE = W_BYTES + X_BYTES + S_BYTES;
  static constexpr int NB = (BN + BS - 1) / BS;                 // weight scale rows of a tile
  static constexpr int SCALES = KS * STAGES * STAGE;                      // ... kept whole behind the stages
  static constexpr int LDS = SCALES + NB * (BS_MAX_K / BS) * 4;
  static constexpr int W_COPIES = BN / 8 / (WN * WM), X_COPIES = BM / 8 / (WN * WM);  // per wave and block
  static constexpr int COPIES = W_COPIES + X_COPIES, ROWS = TN > 1 ? TN / 2 : 1;  // tile rows that copies go with
  static constexpr int PER_ROW = (COPIES + ROWS - 1) / ROWS;
  static_assert(TN * 16 <= BS && BS % (TN * 16) == 0, "one weight scale per wave and block");
  static_assert((KS - 1) * WAVES * 64 * TN * TM * 16 <= SCALES, "the groups' sums fit the stages");
  static_assert(BM % 64 == 0 && (WN * WM) % (BM / 64) == 0, "scale copies");
  static_assert(W_COPIES * 8 * WN * WM == BN && X_COPIES * 8 * WN * WM == BM, "whole copies");
};

template <int WN, int WM, int TN, int TM, int ST, int KS, bool EXACT, typename OUT>
__global__ __launch_bounds__(64 * WN * WM * KS, 2) void bs_matmul_tile_kernel(BsMatmul a, int n_tiles, int m_tiles) {
  using C = Tile<WN, WM, TN, TM, ST, KS, EXACT>;
  extern __shared__ __align__(1024) uint8_t lds[];
  constexpr int WAVES = C::WAVES;
  const int lane = threadIdx.x & 63, block_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = block_wave / WAVES, wave = block_wave % WAVES;
  const int r = lane & 15, quad = lane >> 4;
  // an XCD (block id mod 8) takes a contiguous eighth of the tiles, in strips
  // of 4 M tiles so that neighbours in time share operands in its L2
  const int tiles = n_tiles * m_tiles;
  const int id = xcd_order(blockIdx.x, tiles);
  const int strip = id / (4 * n_tiles), in_strip = id - strip * 4 * n_tiles;
  const int strip_m = min(4, m_tiles - 4 * strip);
  const int mt = 4 * strip + in_strip % strip_m, nt = in_strip / strip_m;
  const int n0 = nt * C::BN, m0 = mt * C::BM;
  const int KB = bs_blocks(a.K);
  const int rows_n = min(C::BN, a.N - n0), rows_m = min(C::BM, a.M - m0);

  const __amdgpu_buffer_rsrc_t wbuf = buffer_of(a.wq + (int64_t)n0 * a.K, (int64_t)rows_n * a.K);
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.xq + m0 * a.ldx, (rows_m - 1) * a.ldx + a.K);
  const __amdgpu_buffer_rsrc_t sbuf = buffer_of(a.xs + (int64_t)m0 * KB, (int64_t)rows_m * KB * 4);
  // copy i of a wave brings rows 8 (wave + i waves) .. + 7; lane l row l / 8
  const int col = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t woff[C::W_COPIES], xoff[C::X_COPIES];
#pragma unroll
  for (int i = 0; i < C::W_COPIES; i++) woff[i] = (uint32_t)(8 * (wave + i * WAVES) + (lane >> 3)) * a.K + col;
#pragma unroll
  for (int i = 0; i < C::X_COPIES; i++) {
    const int row = 8 * (wave + i * WAVES) + (lane >> 3);
    xoff[i] = row < rows_m ? (uint32_t)(row * a.ldx) + col : BUFFER_OUT;
  }
  // the rows' scales, 64 a copy; with more than two stages every wave makes one
  // (some the same ones), as all need the same number of copies in flight
  const int srow = wave % (C::BM / 64) * 64;
  const uint32_t soff = (uint32_t)(srow + lane) * KB * 4;
  const uint8_t* stages = lds + group * C::STAGES * C::STAGE;
  const uint32_t base = lds_address(stages);
  // Copy i of block kb, i < COPIES (the scales go with copy 0).
  auto fetch = [&](int kb, int stage, int i) {
    const uint32_t at = base + stage * C::STAGE;
    if (i < C::W_COPIES)
      lds_copy16(wbuf, at + (wave + i * WAVES) * 1024, woff[i], kb * BS);
    else
      lds_copy16(xbuf, at + C::W_BYTES + (wave + (i - C::W_COPIES) * WAVES) * 1024, xoff[i - C::W_COPIES], kb * BS);
    if (i == 0 && (C::STAGES > 2 || wave < C::BM / 64))
      lds_copy4(sbuf, at + C::W_BYTES + C::X_BYTES + srow * 4, soff, kb * 4);
  };
  // In a short last block the pieces past K are zeros, not the next row's.
  auto cut_last = [&](int kb) {
    if (kb * BS + BS <= a.K) return;
    const uint32_t out = kb * BS + col < a.K ? 0u : BUFFER_OUT;
#pragma unroll
    for (int i = 0; i < C::W_COPIES; i++) woff[i] |= out;
#pragma unroll
    for (int i = 0; i < C::X_COPIES; i++) xoff[i] |= out;
  };

  const int wn = wave % WN, wm = wave / WN;
  // The weight scales of the whole tile are staged once: loads of them in the
  // loop would wait for the copies in flight (one counter counts both).
  float* wsc_all = reinterpret_cast<float*>(lds + C::SCALES);
  for (int i = threadIdx.x; i < C::NB * KB; i += C::THREADS) {
    const int b = min(n0 / BS + i / KB, bs_blocks(a.N) - 1);
    wsc_all[i] = a.ws[(int64_t)b * KB + i % KB];
  }
  const float* wsr = wsc_all + (wn * TN * 16) / BS * KB;
  const int swz0 = (quad ^ (r & 7)) * 16, swz1 = ((quad + 4) ^ (r & 7)) * 16;
  auto frag = [&](const uint8_t* tile, int row) {  // the lane's 32 bytes of the tile's row (row % 8 == r % 8)
    const uint8_t* p = tile + row * BS;
    return join_pieces(*reinterpret_cast<const i32x4_t*>(p + swz0), *reinterpret_cast<const i32x4_t*>(p + swz1));
  };
  f32x4_t acc[TN][TM] = {};
  // (blocks past the last: the last again, into a stage that nothing reads)
#pragma unroll
  for (int b = 0; b < C::STAGES - 1; b++) {
    const int kb = min(group + b * KS, KB - 1);
    cut_last(kb);
#pragma unroll
    for (int i = 0; i < C::COPIES; i++) fetch(kb, b, i);
  }
  int stage = 0;
  for (int k0 = 0; k0 < KB; k0 += KS) {
    const int kb = k0 + group;
    lds_landed<(C::STAGES - 2) * (C::COPIES + 1)>();
    const int fill = stage == 0 ? C::STAGES - 1 : stage - 1;
    if (KS > 1 && kb >= KB) break;  // (the last round has no block for this group)
    const uint8_t* st = stages + stage * C::STAGE;
    // The copies into the free stage are spread over the tile rows of this
    // block: all at once they fill the address queue and hold up the waves.
    const int next = min(kb + (C::STAGES - 1) * KS, KB - 1);
    cut_last(next);
    auto fetch_some = [&](int i) {
#pragma unroll
      for (int c = i * C::PER_ROW; c < (i + 1) * C::PER_ROW && c < C::COPIES; c++) fetch(next, fill, c);
    };
    const uint8_t* wt = st + wn * TN * 16 * BS;
    const uint8_t* xt = st + C::W_BYTES + wm * TM * 16 * BS;
    const float* xsc = reinterpret_cast<const float*>(st + C::W_BYTES + C::X_BYTES) + wm * TM * 16;
    const float wsc = wsr[kb];
    float sc[TM];
#pragma unroll
    for (int j = 0; j < TM; j++) sc[j] = xsc[j * 16 + r] * wsc;
    if constexpr (EXACT) {
      F16Block x[TM], w;
      i32x8_t raw = frag(wt, r);
#pragma unroll
      for (int j = 0; j < TM; j++) x[j].set(frag(xt, j * 16 + r));
      w.set(raw);
      // As below, and a quarter of the next row's conversion beside each tile.
      f32x4_t p[2][TM];
#pragma unroll
      for (int i = 0; i <= TN; i++) {
        fetch_some(i);
        F16Block w_next;
        if (i + 1 < TN) raw = frag(wt, (i + 1) * 16 + r);
#pragma unroll
        for (int j = 0; j < TM; j++) {
          if (i < TN) p[i & 1][j] = mfma_block(w, x[j]);
          if (i + 1 < TN && j > 0) {
#pragma unroll
            for (int s = 4 * (j - 1) / (TM - 1); s < 4 * j / (TM - 1); s++) w_next.s[s] = e4m3_to_f16(raw[2 * s], raw[2 * s + 1]);
          }
          if (i > 0) {
#pragma unroll
            for (int q = 0; q < 4; q++)
              acc[i - 1][j][q] = __builtin_fmaf(p[(i - 1) & 1][j][q], sc[j], acc[i - 1][j][q]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        w = w_next;
      }
    } else {
      i32x8_t x[TM];
#pragma unroll
      for (int j = 0; j < TM; j++) x[j] = frag(xt, j * 16 + r);
      // Tile row i is multiplied while row i - 1's sums are scaled: one matrix
      // step, then the four multiply-adds that run in its shadow.
      i32x8_t w = frag(wt, r);
      f32x4_t p[2][TM];
#pragma unroll
      for (int i = 0; i <= TN; i++) {
        fetch_some(i);
        i32x8_t w_next = w;
        if (i + 1 < TN) w_next = frag(wt, (i + 1) * 16 + r);
#pragma unroll
        for (int j = 0; j < TM; j++) {
          if (i < TN) p[i & 1][j] = mfma_block_e4m3(w, x[j]);
          if (i > 0) {
#pragma unroll
            for (int q = 0; q < 4; q++)
              acc[i - 1][j][q] = __builtin_fmaf(p[(i - 1) & 1][j][q], sc[j], acc[i - 1][j][q]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        w = w_next;
      }
    }
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
  }
  lds_landed<0>();  // no copy outlives the block
  if constexpr (KS > 1) {
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds);  // [group - 1][tile][thread of a group]
    const int gt = wave * 64 + lane;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < TN * TM; i++) sums[((group - 1) * TN * TM + i) * WAVES * 64 + gt] = acc[i / TM][i % TM];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < KS; g++)
#pragma unroll
      for (int i = 0; i < TN * TM; i++) acc[i / TM][i % TM] += sums[((g - 1) * TN * TM + i) * WAVES * 64 + gt];
  }

  OUT* y = static_cast<OUT*>(a.y);
  // four outputs leave as one store where every row allows it
  const bool vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(OUT) - 1)) == 0;
#pragma unroll
  for (int j = 0; j < TM; j++) {
    const int m = m0 + (wm * TM + j) * 16 + r;
    if (m >= a.M) continue;
    OUT* row = y + m * a.ldy;
#pragma unroll
    for (int i = 0; i < TN; i++) {
      const int n = n0 + (wn * TN + i) * 16 + 4 * quad;
      store4(row + n, acc[i][j], a.N - n, vec);
    }
  }
}

size_t bs_matmul_ws(int, int, int) { return 0; }

template <int WN, int WM, int TN, int TM, int ST, int KS, bool EXACT, typename OUT>
static hipError_t launch_tile(const BsMatmul& a, hipStream_t s) {
  using C = Tile<WN, WM, TN, TM, ST, KS, EXACT>;
  const int n_tiles = (a.N + C::BN - 1) / C::BN, m_tiles = (a.M + C::BM - 1) / C::BM;
  auto* k = bs_matmul_tile_kernel<WN, WM, TN, TM, ST, KS, EXACT, OUT>;
  int per_cu, cus;
  hipError_t e = launch_shape((const void*)k, C::THREADS, C::LDS, C::LDS, &per_cu, &cus);
  if (e != hipSuccess) return e;
  QMOE_LAUNCH(k, dim3((unsigned)(n_tiles * m_tiles)), dim3(C::THREADS), C::LDS, s, a, n_tiles, m_tiles);
  return hipGetLastError();
}

template <int TM, int U, typename OUT>
static hipError_t launch_rows(const BsMatmul& a, hipStream_t s) {
  auto* k = bs_matmul_rows_kernel<TM, U, OUT>;
  QMOE_LAUNCH(k, dim3((a.N + 15) / 16), dim3(512), 0, s, a);
  return hipGetLastError();
}

// The variant: by rows, then the largest tile of which there are enough for
// the 256 CUs.  Measured on both sides of each step, N = K = 4096 unless
// given (us, fp16 steps / E4M3 steps):
//   M 32: rows 9.8, 64 x 64 tiles 14.9 / 12.1;   64: rows 15.3, tiles 14.9 / 12.1
//   M 128 (64 tiles of 128 x 64): 20.2 / 17.2 on them, 15.2 / 12.0 on 64 x 64
//   M 1000, N 1100, K 2064 (144): 14.4 / 12.3 on 128 x 64, 19.3 / 16.5 on 64 x 64
//   M 512 (128 tiles of 128 x 128): 32.0 / 24.4 on them, 22.6 / 18.2 on 128 x 64
//   M 1024 (256): 34.6 (two groups) / 26.0 (four stages) on 128 x 128, 38.4 /
//     32.6 with one group and two stages, 42.6 / 29.1 on 128 x 64
//   M 2048 (512; 128 of 256 x 256): 71.0 / 42.9 with one group and two stages,
//     66.9 / 53.6 with two groups; 256 x 256 E4M3 61
//   M 4096 (1024; 256 of 256 x 256): 123 / 82.8 on 128 x 128, 132 with two
//     groups; 256 x 256 E4M3 71.4
// The E4M3 steps round a sum by 1.4e-5 of it, bf16 by 2e-3: they serve bf16
// outputs, and sums of eight blocks or more, where the errors average out.
template <typename OUT>
static hipError_t launch_matmul(const BsMatmul& a, hipStream_t s) {
  if (a.M <= 16) return launch_rows<1, 4, OUT>(a, s);
  if (a.M <= 32) return launch_rows<2, 2, OUT>(a, s);
  auto tiles = [&](int bn, int bm) { return (int64_t)((a.N + bn - 1) / bn) * ((a.M + bm - 1) / bm); };
  if constexpr (sizeof(OUT) == 2) {
    if (a.K >= 8 * BS) {
      if (tiles(256, 256) >= 192) return launch_tile<2, 4, 8, 4, 2, 1, false, OUT>(a, s);
      if (tiles(128, 128) >= 384) return launch_tile<2, 2, 4, 4, 2, 1, false, OUT>(a, s);
      if (tiles(128, 128) >= 192) return launch_tile<2, 2, 4, 4, 4, 1, false, OUT>(a, s);
      if (tiles(128, 64) >= 128) return launch_tile<2, 2, 4, 2, 3, 1, false, OUT>(a, s);
      return launch_tile<2, 2, 2, 2, 3, 2, false, OUT>(a, s);
    }
  }
  if (tiles(128, 128) >= 768) return launch_tile<2, 2, 4, 4, 2, 1, true, OUT>(a, s);
  if (tiles(128, 128) >= 192) return launch_tile<2, 2, 4, 4, 2, 2, true, OUT>(a, s);
  if (tiles(128, 64) >= 128) return launch_tile<2, 2, 4, 2, 3, 2, true, OUT>(a, s);
  return launch_tile<2, 2, 2, 2, 3, 2, true, OUT>(a, s);
}

hipError_t launch_bs_matmul(const BsMatmul& a, hipStream_t s) {
  const int pid = prof_begin("bs_matmul", s);
  const hipError_t e = a.y_dtype == X_BF16 ? launch_matmul<uint16_t>(a, s) : launch_matmul<float>(a, s);
  prof_end(pid, s);
  return e;
}

}  // namespace qmoe
