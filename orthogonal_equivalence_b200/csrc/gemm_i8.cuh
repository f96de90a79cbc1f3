// Int8 products of the POET-XQ weight (codes Wq [n][m], a scale per row):
//   forward   z[t][j]  = xs[t] ws[j] sum_i xq[t][i] Wq[j][i]
//   gradient  dx[t][i] = gs[t]       sum_j gq[t][j] Wq[j][i]
// with the sums exact in 32-bit integers (|code| <= 128 and at most 102400
// terms stay below 2^31).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "perm.cuh"

namespace poetx {
namespace i8 {

struct Params {
  const int8_t* a;      // [M][lda] codes of the tokens
  const int8_t* b;      // forward: [N][ldb], gradient: [K][ldb]
  const float* as;      // [M]
  const float* bs;      // [N] or NULL
  void* out;            // [M][N]
  int64_t lda, ldb;
  int M, N, K;
};

// 64 x 64 output tile, 32 bytes of K per step, 4 x 4 sums per thread by dp4a.
constexpr int TILE = 64, KB = 32;

template <typename T, bool B_KN>
__global__ void __launch_bounds__(256) product_kernel(const Params p) {
  __shared__ int as[TILE][KB / 4 + 1], bs[TILE][KB / 4 + 1];
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * TILE;
  const int n0 = blockIdx.y * TILE;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  int8_t* a8 = reinterpret_cast<int8_t*>(as);
  int8_t* b8 = reinterpret_cast<int8_t*>(bs);
  constexpr int ROW = (KB / 4 + 1) * 4;
  for (int k0 = 0; k0 < p.K; k0 += KB) {
    for (int i = threadIdx.x; i < TILE * KB; i += 256) {
      const int r = i / KB, k = i % KB;
      a8[r * ROW + k] = m0 + r < p.M && k0 + k < p.K ? p.a[(m0 + r) * p.lda + k0 + k] : int8_t(0);
    }
    for (int i = threadIdx.x; i < TILE * KB; i += 256) {
      const int r = B_KN ? i % TILE : i / KB, k = B_KN ? i / TILE : i % KB;
      int8_t v = 0;
      if (n0 + r < p.N && k0 + k < p.K)
        v = B_KN ? p.b[static_cast<int64_t>(k0 + k) * p.ldb + n0 + r] : p.b[static_cast<int64_t>(n0 + r) * p.ldb + k0 + k];
      b8[r * ROW + k] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KB / 4; ++k) {
      int av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = as[ty + 16 * i][k];
        bv[i] = bs[tx + 16 * i][k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = m0 + ty + 16 * i;
    if (r >= p.M) continue;
    const float s = p.as[r];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + tx + 16 * j;
      if (c >= p.N) continue;
      const float v = static_cast<float>(acc[i][j]) * s;
      out[r * p.N + c] = from_f32<T>(p.bs ? v * p.bs[c] : v);
    }
  }
}

}  // namespace i8
}  // namespace poetx
