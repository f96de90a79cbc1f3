// Backward of one side of an fp32 layer from an 8-bit checkpoint of its
// activation X (q8.cuh), both products of every block in one launch:
//   O_j = D_j G_j^T              tiles of TS tokens x TS rows of G_j, over b
//   part[s][j] = X_j^T D_j       tiles of TS x TS of dG_j, over the tokens of split s
// FFMA throughout (the fp32 layer's arithmetic).  A block computes one tile:
// 256 threads, (TS / 16)^2 sums each, KB terms staged in shared memory while
// the next KB are loaded into registers; X is decoded as it is loaded.  Reads
// of either operand run along its rows, whatever b is.
#pragma once

#include <cstdint>

#include "q8.cuh"

namespace poetx {
namespace bf32 {

constexpr int KB = 32, THREADS = 256;

struct Params {
  const float* D;       // [T][d]
  const float* G;       // [nblk][b][b], with O
  float* O;             // [T][d] or NULL
  const int8_t* codes;  // [T][d]
  const uint8_t* exps;  // [T][ng]
  float* part;          // [splits][nblk][b][b]
  int64_t T;
  int d, b, ng, nblk, splits;
  int tiles_b;          // tiles along b
  int64_t o_blocks;     // blocks that compute O (first in the grid)
};

// One tile: O (rows: tokens, columns: rows of G_j, K: columns of the block) or
// dG (rows and columns of dG_j, K: tokens of the split).  `id` counts the tiles
// of its kind.
template <int TS, bool WANT_O>
__device__ __forceinline__ void tile(const Params& p, int64_t id, float (*As)[TS + 1], float (*Bs)[TS + 1]) {
  constexpr int R = TS / 16;             // sums per thread and dimension
  constexpr int L = TS * KB / THREADS;   // loads per thread and operand
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int n0 = static_cast<int>(id % p.tiles_b) * TS;
  id /= p.tiles_b;
  int64_t m0 = 0;
  if constexpr (!WANT_O) {
    m0 = id % p.tiles_b * TS;
    id /= p.tiles_b;
  }
  const int j = static_cast<int>(id % p.nblk), col = j * p.b;
  const int64_t rest = id / p.nblk;      // token tile, or split
  if constexpr (WANT_O) m0 = rest * TS;
  const int64_t k_first = WANT_O ? 0 : rest * p.T / p.splits;
  const int64_t k_last = WANT_O ? p.b : (rest + 1) * p.T / p.splits;
  // this thread's elements: (tk + l * SK, ti + l * SI) of the stage
  const int tk = WANT_O ? threadIdx.x % KB : threadIdx.x / TS;
  const int ti = WANT_O ? threadIdx.x / KB : threadIdx.x % TS;
  constexpr int SK = WANT_O ? 0 : THREADS / TS, SI = WANT_O ? THREADS / KB : 0;
  float a[L], b[L];
  auto fetch = [&](int64_t k0) {
    const int64_t k = k0 + tk;
    if constexpr (WANT_O) {
      const float* d = p.D + (m0 + ti) * p.d + col + k;
      const float* g = p.G + (static_cast<int64_t>(col) + n0 + ti) * p.b + k;
#pragma unroll
      for (int l = 0; l < L; ++l) {
        a[l] = k < k_last && m0 + ti + l * SI < p.T ? d[static_cast<int64_t>(l * SI) * p.d] : 0.f;
        b[l] = k < k_last && n0 + ti + l * SI < p.b ? g[static_cast<int64_t>(l * SI) * p.b] : 0.f;
      }
    } else {
      const int ca = col + static_cast<int>(m0) + ti;
      const bool ina = m0 + ti < p.b, inb = n0 + ti < p.b;
      const int8_t* x = p.codes + k * p.d + ca;
      const uint8_t* e = p.exps + k * p.ng + ca / q8::GROUP;
      const float* d = p.D + k * p.d + col + n0 + ti;
      int8_t q[L];
      uint8_t eb[L];
#pragma unroll
      for (int l = 0; l < L; ++l) {
        const bool in = k + l * SK < k_last;
        q[l] = in && ina ? x[static_cast<int64_t>(l * SK) * p.d] : int8_t(0);
        eb[l] = in && ina ? e[static_cast<int64_t>(l * SK) * p.ng] : uint8_t(0);
        b[l] = in && inb ? d[static_cast<int64_t>(l * SK) * p.d] : 0.f;
      }
#pragma unroll
      for (int l = 0; l < L; ++l) a[l] = static_cast<float>(q[l]) * q8::exponent_value(eb[l]);
    }
  };
  float acc[R][R] = {};
  fetch(k_first);
  for (int64_t k0 = k_first; k0 < k_last; k0 += KB) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      As[tk + l * SK][ti + l * SI] = a[l];
      Bs[tk + l * SK][ti + l * SI] = b[l];
    }
    __syncthreads();
    if (k0 + KB < k_last) fetch(k0 + KB);
#pragma unroll 8
    for (int k = 0; k < KB; ++k) {
      float u[R], v[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        u[r] = As[k][ty + 16 * r];
        v[r] = Bs[k][tx + 16 * r];
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < R; ++c) acc[r][c] = fmaf(u[r], v[c], acc[r][c]);
    }
    __syncthreads();
  }
  const int64_t rows = WANT_O ? p.T : p.b, ld = WANT_O ? p.d : p.b;
  float* out = WANT_O ? p.O + col : p.part + id * p.b * static_cast<int64_t>(p.b);  // id = split * nblk + j
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t m = m0 + ty + 16 * r;
    if (m >= rows) continue;
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int n = n0 + tx + 16 * c;
      if (n < p.b) out[m * ld + n] = acc[r][c];
    }
  }
}

template <int TS>
__global__ void __launch_bounds__(THREADS) block_backward_kernel(const Params p) {
  __shared__ float As[KB][TS + 1], Bs[KB][TS + 1];
  if (blockIdx.x < p.o_blocks) tile<TS, true>(p, blockIdx.x, As, Bs);
  else tile<TS, false>(p, blockIdx.x - p.o_blocks, As, Bs);
}

}  // namespace bf32
}  // namespace poetx
