// The tiled product of int8 matrices, used by the dense product and by the
// experts' products (contracts: include/moe.h).
//
// y[m][n] = (xs[m] ws[n]) sum_i xq[m][i] wq[n][i]: with one scale per row and
// one per output channel the whole sum over K stays in the matrix unit's 32-bit
// integers (|sum| <= 2^14 K <= 2^28), so it is exact whatever the order in which
// steps, waves and blocks add it, and the scales are met once at the end.
//
// Matrix-unit steps: 32x32x32 runs at 4.3 to 4.7 POP/s, 16x16x64 at 2.4 to 2.6
// (independent accumulators, no operands read), so the 16-wide one is for calls of at
// most 16 rows, which are bound by the weights' bytes.  The operands are taken as
// (weights, activations): the result's columns (lane % 32) are activation rows, and a
// lane's 16 values are 4 runs of 4 consecutive outputs of one row, run g at 8 g + 4
// (lane / 32).
#pragma once

#include "blockscale.hpp"

namespace qmoe {

typedef int i32x16_t __attribute__((ext_vector_type(16)));

// A block's tile: NMAT weight matrices x WN x TN tiles of 32 outputs by WM x TM
// tiles of 32 rows, WN x WM waves.  BK inputs at a time go to LDS by
// asynchronous copies, ST stages deep; the 16-byte pieces of a row are swizzled
// so that what a read touches at once is in different banks.  KS groups of
// such waves share the K blocks (group g takes blocks g, g + KS, ...), each with
// stages of its own, and their sums are added at the end: where tiles are few, a
// CU has more waves and a shorter chain of steps.
template <int WN_, int WM_, int TN_, int TM_, int BK_, int ST_, int KS_, int NMAT_>
struct I8Tile {
  static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, BK = BK_, ST = ST_, KS = KS_, NMAT = NMAT_;
  static constexpr int WAVES = WN * WM, THREADS = 64 * WAVES * KS;
  static constexpr int BN = WN * TN * 32, BM = WM * TM * 32;
  static constexpr int SUBS = BK / 32;  // matrix steps of a K block
  static constexpr int PIECES = BK / 16, COPY_ROWS = 64 / PIECES;
  static constexpr int W_BYTES = NMAT * BN * BK, STAGE = W_BYTES + BM * BK;
  static constexpr int SCALES = KS * ST * STAGE;  // [NMAT][BN] of the outputs, [BM] of the rows, behind the stages
  static constexpr int S_ROWS = (BM + 63) / 64 * 64;
  static constexpr int LDS = SCALES + (NMAT * ((BN + 63) / 64 * 64) + S_ROWS) * 4;
  static constexpr int W_UNITS = BN / COPY_ROWS, X_UNITS = BM / COPY_ROWS;
  static constexpr int W_COPIES = (W_UNITS + WAVES - 1) / WAVES;  // (waves past the units bring some again)
  static constexpr int X_COPIES = (X_UNITS + WAVES - 1) / WAVES;
  static constexpr int COPIES = NMAT * W_COPIES + X_COPIES;
  static constexpr int ROWS = NMAT * TN, FRAGS = ROWS + TM, MULS = ROWS * TM;
  static constexpr int REGS = 16 * MULS;  // accumulators of a lane
  // blocks that fit a CU's LDS, and the registers to match
  static constexpr int BLOCKS = 160 * 1024 / LDS;
  static constexpr int WAVES_PER_SIMD_LDS = BLOCKS * WAVES * KS / 4 > 0 ? BLOCKS * WAVES * KS / 4 : 1;
  static constexpr int WAVES_PER_SIMD_REG = REGS > 128 ? 1 : REGS > 64 ? 2 : 4;
  static constexpr int WAVES_PER_SIMD = WAVES_PER_SIMD_LDS < WAVES_PER_SIMD_REG ? WAVES_PER_SIMD_LDS : WAVES_PER_SIMD_REG;
  static_assert(SUBS % 2 == 0, "operands alternate between two sets of registers");
  static_assert(W_UNITS * COPY_ROWS == BN && X_UNITS * COPY_ROWS == BM, "whole copies");
  static_assert((KS - 1) * WAVES * 64 * REGS * 4 <= SCALES, "the groups' sums fit the stages");
  static_assert(ST >= 2 && (ST - 1) * COPIES <= 63, "copies in flight are counted in 6 bits");
  static_assert(LDS <= 160 * 1024, "LDS of a CU");
};

// Where 16-byte piece p of row r lies in a stage's row: so that the same piece of
// 16 consecutive rows, which one cycle of a read takes, is in 16 different places
// of LDS's 64 banks.
template <int BK>
__device__ __forceinline__ int i8_place(int r, int p) {
  return BK == 128 ? p ^ ((r >> 1) & 7) : p ^ ((r >> 2) & 3);
}

// acc[mat][i][j] = the wave's tiles of exact sums.  wbuf: the tile's rows of each
// matrix, K bytes apart; xbuf with xrow(i): the byte offset of row i's codes
// (BUFFER_OUT: no such row); K blocks (of BK) kb0 <= kb < kb1.  wsbuf, xsbuf with
// srow(i) (row i's): the scales, left in LDS behind the stages.  ONCE: no other block
// reads these weights, which then go past the caches.  With KS > 1 the sums are group
// 0's; false for the other groups' threads.
template <class C, bool ONCE = false, class XRow, class SRow>
__device__ __forceinline__ bool i8_product(uint8_t* lds, const __amdgpu_buffer_rsrc_t (&wbuf)[C::NMAT],
                                           const __amdgpu_buffer_rsrc_t (&wsbuf)[C::NMAT], int K,
                                           __amdgpu_buffer_rsrc_t xbuf, __amdgpu_buffer_rsrc_t xsbuf, XRow xrow, SRow srow,
                                           int kb0, int kb1, i32x16_t (&acc)[C::NMAT][C::TN][C::TM]) {
  constexpr int WAVES = C::WAVES, TN = C::TN, TM = C::TM, KS = C::KS, ROWS = C::ROWS, BK = C::BK;
  const int lane = threadIdx.x & 63, block_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = block_wave / WAVES, wave = block_wave % WAVES;
  // A copy brings COPY_ROWS rows of BK bytes; lane l row l / PIECES, its place
  // l % PIECES (an involution: the piece that lies there).
  const int crow = lane / C::PIECES;
  uint32_t woff[C::W_COPIES], xoff[C::X_COPIES];
  static_assert(C::COPY_ROWS * WAVES % 16 == 0, "every copy of a wave is swizzled alike");  // (as BN and BM % 16 == 0)
  const int col = i8_place<BK>(C::COPY_ROWS * wave + crow, lane % C::PIECES) * 16;
#pragma unroll
  for (int i = 0; i < C::W_COPIES; i++) woff[i] = (uint32_t)(C::COPY_ROWS * ((wave + i * WAVES) % C::W_UNITS) + crow) * K + col;
#pragma unroll
  for (int i = 0; i < C::X_COPIES; i++) {
    const uint32_t o = xrow(C::COPY_ROWS * ((wave + i * WAVES) % C::X_UNITS) + crow);
    xoff[i] = o == BUFFER_OUT ? o : o + col;
  }
  const uint8_t* stages = lds + group * C::ST * C::STAGE;
  const uint32_t base = lds_address(stages);
  auto fetch = [&](int kb, int stage, int i) {
    const uint32_t at = base + stage * C::STAGE;
    if (i < C::NMAT * C::W_COPIES) {
      const int mat = i / C::W_COPIES, c = i % C::W_COPIES;
      const uint32_t to = at + mat * C::BN * BK + (wave + c * WAVES) % C::W_UNITS * 1024;
      if (ONCE)
        lds_copy16_once(wbuf[mat], to, woff[c], kb * BK);
      else
        lds_copy16(wbuf[mat], to, woff[c], kb * BK);
    } else {
      const int c = i - C::NMAT * C::W_COPIES;
      lds_copy16(xbuf, at + C::W_BYTES + (wave + c * WAVES) % C::X_UNITS * 1024, xoff[c], kb * BK);
    }
  };
  // Pieces past K, and blocks past the last, are zeros (kb only grows).
  auto cut = [&](int kb) {
    if (kb < kb1 && kb * BK + BK <= K) return;
    const uint32_t out = kb < kb1 && kb * BK + col < K ? 0u : BUFFER_OUT;
#pragma unroll
    for (int i = 0; i < C::W_COPIES; i++) woff[i] |= out;
#pragma unroll
    for (int i = 0; i < C::X_COPIES; i++) xoff[i] |= out;
  };

  // the scales, 64 a copy, ahead of the codes
  {
    const uint32_t at = lds_address(lds + C::SCALES);
    constexpr int WS_UNITS = (C::BN + 63) / 64;
    for (int u = block_wave; u < C::NMAT * WS_UNITS + C::S_ROWS / 64; u += WAVES * KS) {
      if (u < C::NMAT * WS_UNITS) {
        const int in = u % WS_UNITS * 64 + lane;
        const uint32_t off = in < C::BN ? in * 4 : BUFFER_OUT;
        if (C::NMAT == 1 || u < WS_UNITS)
          lds_copy4(wsbuf[0], at + u * 256, off, 0);
        else
          lds_copy4(wsbuf[C::NMAT - 1], at + u * 256, off, 0);
      } else {
        const int i = (u - C::NMAT * WS_UNITS) * 64 + lane;
        lds_copy4(xsbuf, at + u * 256, i < C::BM ? srow(i) : BUFFER_OUT, 0);
      }
    }
  }

  const int wn = wave % C::WN, wm = wave / C::WN;
  const int r = lane & 31, half = lane >> 5;
  i32x16_t* flat = &acc[0][0][0];
#pragma unroll
  for (int i = 0; i < C::MULS; i++)
#pragma unroll
    for (int q = 0; q < 16; q++) flat[i][q] = 0;
#pragma unroll
  for (int b = 0; b < C::ST; b++) {
    const int kb = kb0 + group + b * KS;
    cut(kb);
#pragma unroll
    for (int i = 0; i < C::COPIES; i++) fetch(kb, b, i);
  }
  // Operands of step `sub` of a stage: ROWS of weights, then TM of activations.
  int place[C::SUBS];
#pragma unroll
  for (int s = 0; s < C::SUBS; s++) place[s] = i8_place<BK>(r, 2 * s + half) * 16;
  const int wrow = (wn * TN * 32 + r) * BK, xrow0 = C::W_BYTES + (wm * TM * 32 + r) * BK;
  i32x4_t f[2][C::FRAGS];
  auto read = [&](const uint8_t* st, int sub, int i, int to) {
    const int at = i < ROWS ? wrow + (i / TN * C::BN + i % TN * 32) * BK : xrow0 + (i - ROWS) * 32 * BK;
    f[to][i] = *reinterpret_cast<const i32x4_t*>(st + at + place[sub]);
  };
  lds_landed<(C::ST - 1) * C::COPIES>();
#pragma unroll
  for (int i = 0; i < C::FRAGS; i++) read(stages, 0, i, 0);
  int stage = 0;
  // Step `sub` is multiplied while the operands of the next one are read.  By a
  // block's last step all of its reads are done: there the waves meet, the next
  // stage has landed, and the copies of block kb + ST go into this one, one behind
  // each matrix step.
  const int rounds = (kb1 - kb0 + KS - 1) / KS;
  for (int k = 0; k < rounds; k++) {
    const int next = stage + 1 == C::ST ? 0 : stage + 1, kb = kb0 + group + (k + C::ST) * KS;
#pragma unroll
    for (int sub = 0; sub < C::SUBS; sub++) {
      const bool last = sub + 1 == C::SUBS;
      if (last) {
        lds_landed<(C::ST - 2) * C::COPIES>();
        cut(kb);
      }
      const uint8_t* from = stages + (last ? next : stage) * C::STAGE;
      constexpr int READS = (C::FRAGS + C::MULS - 1) / C::MULS, FETCHES = (C::COPIES + C::MULS - 1) / C::MULS;
#pragma unroll
      for (int m = 0; m < C::MULS; m++) {
        const int i = m / TM, j = m % TM;
        flat[m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[sub & 1][i], f[sub & 1][ROWS + j], flat[m], 0, 0, 0);
#pragma unroll
        for (int q = m * READS; q < (m + 1) * READS && q < C::FRAGS; q++)
          read(from, last ? 0 : sub + 1, q, (sub + 1) & 1);
        if (last)
#pragma unroll
          for (int q = m * FETCHES; q < (m + 1) * FETCHES && q < C::COPIES; q++) fetch(kb, stage, q);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    stage = next;
  }
  lds_landed<0>();  // no copy outlives the block
  if constexpr (KS > 1) {
    int* sums = reinterpret_cast<int*>(lds);  // [group - 1][value][thread of a group]
    const int gt = wave * 64 + lane;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < C::REGS; i++)
        sums[((group - 1) * C::REGS + i) * WAVES * 64 + gt] = flat[i / 16][i % 16];
    }
    __syncthreads();
    if (group > 0) return false;
#pragma unroll
    for (int g = 1; g < KS; g++)
#pragma unroll
      for (int i = 0; i < C::REGS; i++)
        flat[i / 16][i % 16] += sums[((g - 1) * C::REGS + i) * WAVES * 64 + gt];
  }
  return true;
}

// The staged scales: of 4 of the tile's outputs from n_in_tile on, and of its row m_in_tile.
template <class C>
__device__ __forceinline__ f32x4_t i8_wscale(const uint8_t* lds, int mat, int n_in_tile) {
  return *reinterpret_cast<const f32x4_t*>(lds + C::SCALES + (mat * ((C::BN + 63) / 64 * 64) + n_in_tile) * 4);
}
template <class C>
__device__ __forceinline__ float i8_xscale(const uint8_t* lds, int m_in_tile) {
  return *reinterpret_cast<const float*>(lds + C::SCALES + (C::NMAT * ((C::BN + 63) / 64 * 64) + m_in_tile) * 4);
}

// Sums to values: each of the two products is rounded to fp32 on its own.
__device__ __forceinline__ f32x4_t i8_values(i32x4_t sum, float xs, f32x4_t ws) {
  f32x4_t y;
#pragma unroll
  for (int q = 0; q < 4; q++) y[q] = ((float)sum[q] * xs) * ws[q];
  return y;
}
__device__ __forceinline__ i32x4_t i8_run(const i32x16_t& a, int g) {
  return i32x4_t{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
}

// Stores the wave's tiles: value(i, j, g, n, xs) gives run g of tile (i, j), four
// outputs from column n of the block's tile on, for a row of scale xs.  The lanes hold 4 outputs of
// 32 rows each, 16 or 32 bytes a row of one store; through the stages (free by then,
// each wave in a part of its own) they leave as whole lines, past the caches.  align:
// bytes that every row of the result is aligned to; rows, cols: how many the block's
// tile has.
template <class C, typename OUT, class Value>
__device__ __forceinline__ void i8_store(uint8_t* lds, OUT* out, int64_t ld, int rows, int cols, int align, Value&& value) {
  static_assert(C::KS == 1, "every wave stores");
  constexpr int W = C::TN * 32, PIECE = 16 / sizeof(OUT), STRIDE = W * sizeof(OUT) + 16;
  constexpr int LANES = W / PIECE, AT_ONCE = 64 / LANES;  // lanes of a row, rows of a store
  static_assert(C::WAVES * 32 * STRIDE <= C::SCALES, "a part for every wave");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, half = lane >> 5;
  const int wn = wave % C::WN, wm = wave / C::WN;
  uint8_t* mine = lds + wave * 32 * STRIDE;
  const bool whole = align >= 16 && rows >= C::BM && cols >= C::BN;
#pragma unroll
  for (int j = 0; j < C::TM; j++) {
    const int m0 = (wm * C::TM + j) * 32;
    const float xs = i8_xscale<C>(lds, m0 + r);
#pragma unroll
    for (int i = 0; i < C::TN; i++)
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int n = i * 32 + 8 * g + 4 * half;
        store4(reinterpret_cast<OUT*>(mine + r * STRIDE) + n, value(i, j, g, wn * W + n, xs), 4, true);
      }
    auto piece = [&](int q) {
      return *reinterpret_cast<const u32x4_t*>(mine + (q * AT_ONCE + lane / LANES) * STRIDE + lane % LANES * 16);
    };
    const int m = m0 + lane / LANES, n = wn * W + lane % LANES * PIECE;
    OUT* to = out + m * ld + n;
    if (whole) {
#pragma unroll
      for (int q = 0; q < 32 / AT_ONCE; q++) __builtin_nontemporal_store(piece(q), reinterpret_cast<u32x4_t*>(to + q * AT_ONCE * ld));
    } else {
#pragma unroll 1
      for (int q = 0; q < 32 / AT_ONCE; q++) {
        const u32x4_t v = piece(q);
        if (m + q * AT_ONCE >= rows) break;
        OUT* p = to + q * AT_ONCE * ld;
        if (align >= 16 && n + PIECE <= cols) {
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
        } else if (align >= 8 && n + PIECE <= cols) {
          __builtin_nontemporal_store(u32x2_t{v[0], v[1]}, reinterpret_cast<u32x2_t*>(p));
          __builtin_nontemporal_store(u32x2_t{v[2], v[3]}, reinterpret_cast<u32x2_t*>(p) + 1);
        } else if (align >= 4 && n + PIECE <= cols) {
#pragma unroll
          for (int e = 0; e < 4; e++) __builtin_nontemporal_store(v[e], reinterpret_cast<uint32_t*>(p) + e);
        } else {
#pragma unroll
          for (int e = 0; e < PIECE; e++) {
            OUT o;
            if constexpr (sizeof(OUT) == 4)
              o = __uint_as_float(v[e]);
            else
              o = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
            if (n + e < cols) p[e] = o;
          }
        }
      }
    }
  }
}

}  // namespace qmoe
