// Shared pieces of the 8-bit operators (contracts: include/moe.h): the block-scaled E4M3
// ones, and what the int8 ones and the balance loss take from here (buffers, copies into
// LDS, waits, exact quotients, the M tiles of experts).
//
// The block-scaled operators:
// Matrix-unit step: a block of 128 inputs is 16 x 16 dot products that leave
// the matrix unit on their own and meet the product of their two scales in one
// fused multiply-add.  The E4M3 codes enter as fp16, which holds each exactly,
// through 16x16x32 steps whose sums are fp32.  The unit's own E4M3 steps, twice
// as fast, drop what lies some 14 bits below the largest of eight products: where
// large ones cancel, what is left of the sum is lost (2064 whole-number products
// with the sum -316 gave -208), so no product uses them.
// The operands are taken as (weights, activations): the result's 16 columns
// (lane % 16) are activation rows, so a lane needs one activation scale per
// tile, and its 4 values are 4 consecutive outputs of that row (rows 4 (lane /
// 16) .. + 3), which leave as one store.
// Operand layout: lane l holds row l % 16, 32 bytes of the block.  Which 32
// does not matter as long as both operands agree: lane l takes the 16-byte
// pieces l / 16 and 4 + l / 16, so each load instruction covers 64 contiguous
// bytes of a row, and step s takes bytes 8 s .. 8 s + 7 of its 32.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace qmoe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr int BS = 128;  // inputs (and, for weights, outputs) per scale
__host__ __device__ constexpr int bs_blocks(int n) { return (n + BS - 1) / BS; }

// 8 E4M3 bytes (two words) as fp16.
__device__ __forceinline__ f16x8_t e4m3_to_f16(int a, int b) {
  const f16x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const f16x2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const f16x2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const f16x2_t v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return f16x8_t{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// 16 x 16 dot products over one block of 128.
__device__ __forceinline__ f32x4_t mfma_block(i32x8_t w, i32x8_t x) {
  f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; s++)
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3_to_f16(w[2 * s], w[2 * s + 1]),
                                               e4m3_to_f16(x[2 * s], x[2 * s + 1]), p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ i32x8_t join_pieces(i32x4_t a, i32x4_t b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Four fp32 values (|v| <= 448) to E4M3 bytes, nearest even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// The scale of a group whose largest magnitude has the bits `amax` (order of
// non-negative floats = order of their bits; infinities and NaN come last).
__device__ __forceinline__ float bs_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(amax), 0x1p-100f) / 448.0f;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// x / s correctly rounded for r = 1 / s correctly rounded: each step adds the
// residual, exact by the fused multiply-add, times r.  The first leaves a
// neighbour of the quotient, the second the nearest.  6 instructions for the
// general division's 10; s >= 2^-80 keeps the residuals of all quotients that
// E4M3 or whole numbers tell from 0 out of the subnormal range.
__device__ __forceinline__ float divide_exact(float x, float s, float r) {
  float q = x * r;
  q = __builtin_fmaf(__builtin_fmaf(-s, q, x), r, q);
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-s, q, x), r, q), x);  // (-0 stays -0)
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}

// One output value, fp32 or bf16 (nearest even).
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// One lane's operand of a block as fp16, converted once and used for several
// tiles.
struct F16Block {
  f16x8_t s[4];
  __device__ __forceinline__ void set(i32x8_t v) {
#pragma unroll
    for (int i = 0; i < 4; i++) s[i] = e4m3_to_f16(v[2 * i], v[2 * i + 1]);
  }
};
__device__ __forceinline__ f32x4_t mfma_block(const F16Block& w, const F16Block& x) {
  f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; i++) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.s[i], x.s[i], p, 0, 0, 0);
  return p;
}

// Asynchronous copies from a buffer straight into LDS: lane l's 16 (or 4)
// bytes at off + soff land at LDS byte address lds + 16 l (4 l); a lane whose
// off is outside the buffer gets zeros.  Written out because the compiler cannot
// tell the LDS buffers of a pipeline apart and would wait for every copy in
// flight before each read of LDS.  They have no output registers; the waits are
// lds_landed() below.  m0 holds the address (the compiler, which sets it anew
// before each use of its own, notes that it is not preserved).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"s"(lds), "v"(off), "s"(r), "s"(soff)
               : "memory", "m0");
}
// The same past the caches: for bytes that no other block reads.
__device__ __forceinline__ void lds_copy16_once(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
               ::"s"(lds), "v"(off), "s"(r), "s"(soff)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_copy4(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               ::"s"(lds), "v"(off), "s"(r), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// All but the N youngest copies of this wave have landed, its reads of LDS are
// done, and so it is for every wave of the block.
template <int N>
__device__ __forceinline__ void lds_landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
// A buffer of `bytes` (< 2^31) bytes at p (the same in every lane).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
constexpr uint32_t BUFFER_OUT = 0x80000000u;  // an offset outside every such buffer
// Offset a + b, outside if one of them is (both below 2^31 otherwise, as is
// their sum).
__device__ __forceinline__ uint32_t out_or_sum(uint32_t a, uint32_t b) { return (a + b) | ((a | b) & BUFFER_OUT); }
// Loads into registers; outside the buffer they give zeros.
__device__ __forceinline__ i32x4_t buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ float buffer_load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}

// Work ids such that the blocks of one XCD (block id mod 8) take a contiguous
// eighth of them: a bijection on [0, n).
__device__ __forceinline__ int xcd_order(int block, int n) {
  const int xcd = block & 7, i = block >> 3, base = n >> 3, more = n & 7;
  return xcd * base + min(xcd, more) + i;
}

// Four consecutive outputs; `left` of them exist (<= 0: none).
__device__ __forceinline__ void store4(float* p, f32x4_t v, int left, bool vec) {
  if (vec && left >= 4) {
    *reinterpret_cast<f32x4_t*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < left) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, f32x4_t v, int left, bool vec) {
  if (vec && left >= 4) {
    const uint32_t lo = bf16_bits(v[0]) | (uint32_t)bf16_bits(v[1]) << 16;
    const uint32_t hi = bf16_bits(v[2]) | (uint32_t)bf16_bits(v[3]) << 16;
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < left) p[i] = bf16_bits(v[i]);
  }
}

// The M tiles of BM bucket rows over all experts.  Every lane of a wave makes
// the calls alike; lane l counts the tiles of experts C l .. C l + C - 1, all
// offsets requested at once.
template <int BM>
struct TileScan {
  static constexpr int MOST = MAX_EXPERTS / 64;
  int off[MOST + 1], C, e0, before, upto;  // tiles before the lane's experts, and with them

  __device__ __forceinline__ TileScan(const int32_t* __restrict__ offsets, int E) {
    const int lane = threadIdx.x & 63;
    C = (E + 63) / 64;
    e0 = lane * C;
    off[0] = offsets[min(e0, E)];
#pragma unroll
    for (int i = 0; i < MOST; i++)
      if (i < C) off[i + 1] = offsets[min(e0 + i + 1, E)];
    int n = 0;
#pragma unroll
    for (int i = 0; i < MOST; i++)
      if (i < C) n += (off[i + 1] - off[i] + BM - 1) / BM;
    upto = n;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(upto, s, 64);
      if (lane >= s) upto += o;
    }
    before = upto - n;
  }
  __device__ __forceinline__ int tiles() const { return __builtin_amdgcn_readlane(upto, 63); }
  // Tile `tile`'s expert, first row and row count, and whether it is that expert's
  // only one.  false: there are fewer.
  __device__ __forceinline__ bool find(int tile, int* e_out, int* row0, int* rows, bool* alone) const {
    const uint64_t has = __ballot(tile < upto);
    if (has == 0) return false;
    int left = tile - before, e = e0, first = 0, count = 0, of = 0;
#pragma unroll
    for (int i = 0; i < MOST; i++)
      if (i < C) {
        const int t = (off[i + 1] - off[i] + BM - 1) / BM;
        if (left >= 0 && left < t) {
          e = e0 + i;
          first = off[i] + left * BM;
          count = min(BM, off[i + 1] - first);
          of = t;
        }
        left -= t;
      }
    const int src = __builtin_ctzll(has);
    *e_out = __builtin_amdgcn_readlane(e, src);
    *row0 = __builtin_amdgcn_readlane(first, src);
    *rows = __builtin_amdgcn_readlane(count, src);
    *alone = __builtin_amdgcn_readlane(of, src) == 1;
    return true;
  }
};

// Upper bound on the number of M tiles of n rows in E buckets.
inline int64_t max_tiles(int64_t n, int E, int bm) {
  const int64_t full = n / bm + (E < n ? E : n);
  return full < n ? full : n;
}

struct ExpertTile {
  int e, row0, rows, nt;
  bool alone;  // the only M tile of its expert
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
  return scan.find(pick, &t->e, &t->row0, &t->rows, &t->alone);
}

}  // namespace qmoe
