// The tiled product of block-scaled E4M3 matrices, used by the dense product and
// by the experts' products.
#pragma once

#include "blockscale.hpp"

namespace qmoe {

// A block's tile: NMAT weight matrices x WN x TN tiles of 16 outputs by WM x
// TM tiles of 16 rows, WN x WM waves.  The operands of a block of 128 inputs
// go to LDS by asynchronous copies while the STAGES - 1 blocks before it are
// multiplied; 16-byte piece p of row i lies at place p ^ (i % 8), so the 8
// rows that a read touches at once are in different banks.
// KS groups of such waves share the K blocks (group g takes blocks g, g + KS,
// ...), each with stages of its own, and add their sums in the order of the
// groups: where tiles are few, a CU has more waves and half the steps.
template <int WN_, int WM_, int TN_, int TM_, int ST, int KS_, int NMAT_>
struct Tile {
  static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, STAGES = ST, KS = KS_, NMAT = NMAT_;
  static constexpr int WAVES = WN * WM, THREADS = 64 * WAVES * KS;
  static constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
  static constexpr int S_ROWS = (BM + 63) / 64 * 64;  // a copy of scales brings 64
  static constexpr int W_BYTES = NMAT * BN * BS, X_BYTES = BM * BS, S_BYTES = S_ROWS * 4;
  static constexpr int STAGE = W_BYTES + X_BYTES + S_BYTES;
  static constexpr int NB = (BN + BS - 1) / BS;         // weight scale rows of a matrix's tile ...
  static constexpr int SCALES = KS * STAGES * STAGE;    // ... kept whole behind the stages
  static constexpr int LDS = SCALES + NMAT * NB * (BS_MAX_K / BS) * 4;
  // copies of 8 rows per wave and block; where the rows are not 8 (or 16, ...)
  // per wave, some waves bring the same ones
  static constexpr int W_COPIES = BN / 8 / WAVES, X_UNITS = BM / 8;
  static constexpr int X_COPIES = (X_UNITS + WAVES - 1) / WAVES;
  static constexpr int COPIES = NMAT * W_COPIES + X_COPIES;
  static constexpr int TILE_ROWS = NMAT * TN;                           // tiles of 16 outputs of a wave
  static constexpr int SPREAD = TILE_ROWS == 1 ? 1 : TILE_ROWS / 2;     // those that copies go with
  static constexpr int PER_ROW = (COPIES + SPREAD - 1) / SPREAD;
  // registers: where two blocks of 8 small waves fit a CU's LDS, they fit its registers too
  static constexpr int WAVES_PER_SIMD = 2 * LDS <= 160 * 1024 && THREADS == 512 && TILE_ROWS * TM <= 6 ? 4 : 2;
  static_assert((KS - 1) * WAVES * 64 * TILE_ROWS * TM * 16 <= SCALES, "the groups' sums fit the stages");
  static_assert(S_ROWS % 64 == 0 && WAVES % (S_ROWS / 64) == 0, "scale copies");
  static_assert(W_COPIES * 8 * WAVES == BN, "whole copies");
  static_assert(TN * 16 <= BS && BS % (TN * 16) == 0, "one weight scale per wave, matrix and block");
  static_assert(LDS <= 160 * 1024, "LDS of a CU");
};

// acc[mat][i][j] = the wave's tiles.  wbuf: the tile's rows of each matrix,
// K bytes apart; ws: the scales [ws_rows][KB] of their first block on; xbuf,
// sbuf with xrow(i), srow(i): the byte offsets of row i's codes and scales
// (BUFFER_OUT: no such row); K blocks kb0 <= kb < kb1 of the ones that K has.
// With KS > 1 the sums are group 0's; false for the other groups' threads.
template <class C, class XRow, class SRow>
__device__ __forceinline__ bool tile_product(uint8_t* lds, const __amdgpu_buffer_rsrc_t (&wbuf)[C::NMAT],
                                             const float* const (&ws)[C::NMAT], int ws_rows, int K,
                                             __amdgpu_buffer_rsrc_t xbuf, __amdgpu_buffer_rsrc_t sbuf, XRow xrow,
                                             SRow srow, int kb0, int kb1, f32x4_t (&acc)[C::NMAT][C::TN][C::TM]) {
  constexpr int WAVES = C::WAVES, TN = C::TN, TM = C::TM, KS = C::KS, ROWS = C::TILE_ROWS;
  const int lane = threadIdx.x & 63, block_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = block_wave / WAVES, wave = block_wave % WAVES;
  const int r = lane & 15, quad = lane >> 4;
  const int KB = bs_blocks(K);
  // copy i of a wave brings rows 8 (wave + i waves) .. + 7; lane l row l / 8
  const int col = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t woff[C::W_COPIES], xoff[C::X_COPIES];
#pragma unroll
  for (int i = 0; i < C::W_COPIES; i++) woff[i] = (uint32_t)(8 * (wave + i * WAVES) + (lane >> 3)) * K + col;
#pragma unroll
  for (int i = 0; i < C::X_COPIES; i++) {
    const uint32_t o = xrow(8 * ((wave + i * WAVES) % C::X_UNITS) + (lane >> 3));
    xoff[i] = o == BUFFER_OUT ? o : o + col;
  }
  // the rows' scales, 64 a copy; with more than two stages every wave makes one
  // (some the same ones), as all need the same number of copies in flight
  const int s0 = wave % (C::S_ROWS / 64) * 64;
  const uint32_t soff = s0 + lane < C::BM ? srow(s0 + lane) : BUFFER_OUT;
  const uint8_t* stages = lds + group * C::STAGES * C::STAGE;
  const uint32_t base = lds_address(stages);
  // Copy i of block kb, i < COPIES (the scales go with copy 0).
  auto fetch = [&](int kb, int stage, int i) {
    const uint32_t at = base + stage * C::STAGE;
    if (i < C::NMAT * C::W_COPIES) {
      const int mat = i / C::W_COPIES, c = i % C::W_COPIES;
      lds_copy16(wbuf[mat], at + mat * C::BN * BS + (wave + c * WAVES) * 1024, woff[c], kb * BS);
    } else {
      const int c = i - C::NMAT * C::W_COPIES;
      lds_copy16(xbuf, at + C::W_BYTES + (wave + c * WAVES) % C::X_UNITS * 1024, xoff[c], kb * BS);
    }
    if (i == 0 && (C::STAGES > 2 || wave < C::S_ROWS / 64))
      lds_copy4(sbuf, at + C::W_BYTES + C::X_BYTES + s0 * 4, soff, kb * 4);
  };
  // In a short last block the pieces past K are zeros, not the next row's.
  auto cut_last = [&](int kb) {
    if (kb * BS + BS <= K) return;
    const uint32_t out = kb * BS + col < K ? 0u : BUFFER_OUT;
#pragma unroll
    for (int i = 0; i < C::W_COPIES; i++) woff[i] |= out;
#pragma unroll
    for (int i = 0; i < C::X_COPIES; i++) xoff[i] |= out;
  };

  const int wn = wave % C::WN, wm = wave / C::WN;
  float* wsc_all = reinterpret_cast<float*>(lds + C::SCALES);  // [mat][NB][KB]
  const float* wsr = wsc_all + (wn * TN * 16) / BS * KB;
  const int swz0 = (quad ^ (r & 7)) * 16, swz1 = ((quad + 4) ^ (r & 7)) * 16;
  auto frag = [&](const uint8_t* tile, int row) {  // the lane's 32 bytes of the tile's row (row % 8 == r % 8)
    const uint8_t* p = tile + row * BS;
    return join_pieces(*reinterpret_cast<const i32x4_t*>(p + swz0), *reinterpret_cast<const i32x4_t*>(p + swz1));
  };
#pragma unroll
  for (int i = 0; i < ROWS * TM; i++) acc[i / TM / TN][i / TM % TN][i % TM] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // (blocks past the last: the last again, into a stage that nothing reads)
#pragma unroll
  for (int b = 0; b < C::STAGES - 1; b++) {
    const int kb = min(kb0 + group + b * KS, kb1 - 1);
    cut_last(kb);
#pragma unroll
    for (int i = 0; i < C::COPIES; i++) fetch(kb, b, i);
  }
  // The weight scales of the whole tile are staged once: loads of them in the
  // loop would wait for the copies in flight (one counter counts both).  Here they
  // wait for the first stages', which the first step needs anyway.
#pragma unroll
  for (int mat = 0; mat < C::NMAT; mat++)
    for (int i = threadIdx.x; i < C::NB * KB; i += C::THREADS) {
      const int b = C::NB == 1 ? 0 : min(i / KB, ws_rows - 1);
      wsc_all[mat * C::NB * KB + i] = ws[mat][b * KB + (C::NB == 1 ? i : i % KB)];
    }
  int stage = 0;
  for (int k0 = kb0; k0 < kb1; k0 += KS) {
    const int kb = k0 + group;
    lds_landed<(C::STAGES - 2) * (C::COPIES + 1)>();
    const int fill = stage == 0 ? C::STAGES - 1 : stage - 1;
    if (KS > 1 && kb >= kb1) break;  // (the last round has no block for this group)
    const uint8_t* st = stages + stage * C::STAGE;
    // The copies into the free stage are spread over the tile rows of this
    // block: all at once they fill the address queue and hold up the waves.
    const int next = min(kb + (C::STAGES - 1) * KS, kb1 - 1);
    cut_last(next);
    auto fetch_some = [&](int i) {
#pragma unroll
      for (int c = i * C::PER_ROW; c < (i + 1) * C::PER_ROW && c < C::COPIES; c++) fetch(next, fill, c);
    };
    const uint8_t* wt = st + (wn * TN * 16 + r) * BS;
    const uint8_t* xt = st + C::W_BYTES + (wm * TM * 16 + r) * BS;
    auto wfrag = [&](int i) { return frag(wt, i / TN * C::BN + i % TN * 16); };
    const float* xsc = reinterpret_cast<const float*>(st + C::W_BYTES + C::X_BYTES) + wm * TM * 16;
    float sc[C::NMAT][TM];
#pragma unroll
    for (int mat = 0; mat < C::NMAT; mat++) {
      const float wsc = wsr[mat * C::NB * KB + kb];
#pragma unroll
      for (int j = 0; j < TM; j++) sc[mat][j] = xsc[j * 16 + r] * wsc;
    }
    // Tile row i is multiplied while row i - 1's sums are scaled: one matrix
    // step, then the four multiply-adds that run in its shadow and a part of
    // the next row's conversion.
    f32x4_t p[2][TM];
    auto scale = [&](int i, int j) {
#pragma unroll
      for (int q = 0; q < 4; q++)
        acc[i / TN][i % TN][j][q] = __builtin_fmaf(p[i & 1][j][q], sc[i / TN][j], acc[i / TN][i % TN][j][q]);
    };
    F16Block x[TM], w;
    i32x8_t raw = wfrag(0);
#pragma unroll
    for (int j = 0; j < TM; j++) x[j].set(frag(xt, j * 16));
    w.set(raw);
#pragma unroll
    for (int i = 0; i <= ROWS; i++) {
      fetch_some(i);
      F16Block w_next;
      if (i + 1 < ROWS) raw = wfrag(i + 1);
#pragma unroll
      for (int j = 0; j < TM; j++) {
        if (i < ROWS) p[i & 1][j] = mfma_block(w, x[j]);
        if (i + 1 < ROWS && (j > 0 || TM == 1)) {
          constexpr int D = TM > 1 ? TM - 1 : 1;
          const int s0 = TM > 1 ? 4 * (j - 1) / D : 0, s1 = TM > 1 ? 4 * j / D : 4;
#pragma unroll
          for (int s = s0; s < s1; s++) w_next.s[s] = e4m3_to_f16(raw[2 * s], raw[2 * s + 1]);
        }
        if (i > 0) scale(i - 1, j);
        __builtin_amdgcn_sched_barrier(0);
      }
      w = w_next;
    }
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
  }
  lds_landed<0>();  // no copy outlives the block
  if constexpr (KS > 1) {
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds);  // [group - 1][tile][thread of a group]
    const int gt = wave * 64 + lane;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < ROWS * TM; i++)
        sums[((group - 1) * ROWS * TM + i) * WAVES * 64 + gt] = acc[i / TM / TN][i / TM % TN][i % TM];
    }
    __syncthreads();
    if (group > 0) return false;
#pragma unroll
    for (int g = 1; g < KS; g++)
#pragma unroll
      for (int i = 0; i < ROWS * TM; i++)
        acc[i / TM / TN][i / TM % TN][i % TM] += sums[((g - 1) * ROWS * TM + i) * WAVES * 64 + gt];
  }
  return true;
}

}  // namespace qmoe
