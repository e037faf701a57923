// Dense product of block-scaled E4M3 matrices.
#include "blockscale.hpp"

namespace qmoe {

// The 32 bytes of one lane's operand row in block kb (see blockscale.hpp), 0
// past K or for a row that does not exist.
__device__ __forceinline__ i32x8_t load_frag(const uint8_t* row, bool ok, int kb, int K, int quad) {
  const i32x4_t z = {0, 0, 0, 0};
  const int k0 = kb * BS + 16 * quad, k1 = k0 + 64;
  const i32x4_t a = ok && k0 < K ? *reinterpret_cast<const i32x4_t*>(row + k0) : z;
  const i32x4_t b = ok && k1 < K ? *reinterpret_cast<const i32x4_t*>(row + k1) : z;
  return join_pieces(a, b);
}

// Simplest form: a wave owns 16 outputs x 16 rows and reads its operands from
// global memory block by block.
template <typename OUT>
__global__ __launch_bounds__(256) void bs_matmul_kernel(const uint8_t* __restrict__ xq, int64_t ldx,
                                                        const float* __restrict__ xs, int M,
                                                        const uint8_t* __restrict__ wq, const float* __restrict__ ws,
                                                        int N, int K, OUT* __restrict__ y, int64_t ldy, int n_tiles) {
  const int lane = threadIdx.x & 63, r = lane & 15, quad = lane >> 4;
  const int nt = blockIdx.x % n_tiles, mt = blockIdx.x / n_tiles;
  const int n0 = nt * 64 + (threadIdx.x >> 6) * 16, m = mt * 16 + r;
  if (n0 >= N) return;
  const int KB = bs_blocks(K);
  const uint8_t* wrow = wq + (int64_t)(n0 + r) * K;
  const uint8_t* xrow = xq + (int64_t)m * ldx;
  const float* wsr = ws + (int64_t)(n0 / BS) * KB;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = 0; kb < KB; kb++) {
    const f32x4_t p = mfma_block(load_frag(wrow, n0 + r < N, kb, K, quad), load_frag(xrow, m < M, kb, K, quad));
    const float sc = m < M ? xs[(int64_t)m * KB + kb] * wsr[kb] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(p[i], sc, acc[i]);
  }
  if (m >= M) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int n = n0 + 4 * quad + i;
    if (n >= N) continue;
    if constexpr (sizeof(OUT) == 2)
      y[(int64_t)m * ldy + n] = bf16_bits(acc[i]);
    else
      y[(int64_t)m * ldy + n] = acc[i];
  }
}

size_t bs_matmul_ws(int, int, int) { return 0; }

hipError_t launch_bs_matmul(const BsMatmul& a, hipStream_t s) {
  const int n_tiles = (a.N + 63) / 64;
  const dim3 grid((unsigned)((int64_t)n_tiles * ((a.M + 15) / 16)));
  const int pid = prof_begin("bs_matmul", s);
  if (a.y_dtype == X_BF16)
    QMOE_LAUNCH(bs_matmul_kernel<uint16_t>, grid, dim3(256), 0, s, a.xq, a.ldx, a.xs, a.M, a.wq, a.ws, a.N, a.K,
                (uint16_t*)a.y, a.ldy, n_tiles);
  else
    QMOE_LAUNCH(bs_matmul_kernel<float>, grid, dim3(256), 0, s, a.xq, a.ldx, a.xs, a.M, a.wq, a.ws, a.N, a.K,
                (float*)a.y, a.ldy, n_tiles);
  prof_end(pid, s);
  return hipGetLastError();
}

}  // namespace qmoe
