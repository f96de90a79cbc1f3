// Backward of one side of an fp32 layer from an 8-bit checkpoint of its
// activation X (q8.cuh), both products of every block in one launch:
//   O_j = D_j G_j^T              tiles of TM tokens x TS rows of G_j, over b
//   part[s][j] = X_j^T D_j       tiles of TS x TS of dG_j, over the tokens of split s
// FFMA throughout (the fp32 layer's arithmetic).  A block computes one tile; a
// thread holds 4 x 4 sums and reads four terms of either operand at once, two
// 16-byte reads of shared memory for eight packed FMA.  TS follows b, so that
// few of a tile's sums lie outside the block.  Where a TS x TS tile has fewer
// sums than the block threads, groups of threads take every GR-th token of the
// stage and are added up at the end, in order; O takes more tokens instead.  The
// next KB terms are loaded into registers while the last ones are used; X is
// decoded on its way to shared memory.  Rows of either operand are read along
// themselves, 16 bytes a thread where b is a multiple of four (VEC).
//
// 16384 x 2048, b = 64: 272-280 us, 16351 x 1920, b = 96: 454-464 us (123 and 172 us
// at 70 TFLOP/s), bound by the shared reads.  8 x 8 sums a thread spill (O 17 us less
// there, dG 20 us more, and 300 x 512 11.4 instead of 8.3 us).
#pragma once

#include <cstdint>

#include "q8.cuh"

namespace poetx {
namespace bf32 {

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

template <int TS>
struct Shape {
  static constexpr int C = TS / 4;                                       // threads along a side of the tile
  static constexpr int GR = TS == 16 ? 16 : TS == 32 ? 4 : TS == 48 ? 2 : 1;  // groups over the tokens
  static constexpr int NT = C * C * GR;                                  // 256, 256, 288, 256
  static constexpr int TM = 4 * NT / C;                                  // tokens of an O tile: 256, 128, 96, 64
  static constexpr int KBO = TS == 16 ? 16 : 32, KBG = TS == 16 ? 128 : TS == 32 ? 64 : 32;
  static constexpr int BLOCKS = TS == 64 ? 3 : 4;                        // a SM, by registers: 64 a thread; 80 for TS = 64
  static constexpr int LDM = TM + 4, LDS = TS + 4;                       // 16-byte rows, transposed stores without conflicts
  static constexpr int WORDS_O = KBO * (LDM + LDS), WORDS_G = KBG * 2 * LDS, WORDS_R = GR * TS * TS;
  static constexpr int WORDS = WORDS_O > WORDS_G ? (WORDS_O > WORDS_R ? WORDS_O : WORDS_R)
                                                 : (WORDS_G > WORDS_R ? WORDS_G : WORDS_R);
};

// Four elements from p on, those below `n`.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* p, int64_t n) {
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (VEC) {
    if (n > 0) r = *reinterpret_cast<const float4*>(p);
  } else {
    if (n > 0) r.x = p[0];
    if (n > 1) r.y = p[1];
    if (n > 2) r.z = p[2];
    if (n > 3) r.w = p[3];
  }
  return r;
}

// acc += u v^T, two sums an instruction
__device__ __forceinline__ void fma4x4(float (*acc)[4], const float* u, const float* v) {
  const float4 x = *reinterpret_cast<const float4*>(u), y = *reinterpret_cast<const float4*>(v);
  const float a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float d[2] = {a[r], a[r]};
    q8::fma2(acc[r], d, b);
    q8::fma2(acc[r] + 2, d, b + 2);
  }
}

// Rows 4 ty.. and columns 4 tx.. of a thread in a tile of C threads a row: a
// warp covers 4 x 8 threads of the widest one, so that it reads few different
// words of either operand.
template <int C>
__device__ __forceinline__ void place(int t, int& ty, int& tx) {
  if (C == 16) {
    tx = (t & 7) + 8 * (t >> 5 & 1);
    ty = (t >> 3 & 3) + 4 * (t >> 6);
  } else {
    tx = t % C;
    ty = t / C;
  }
}

template <bool VEC>
__device__ __forceinline__ void put_row(float* row, const float4& v, int n, int b) {
  if (VEC) {
    if (n < b) *reinterpret_cast<float4*>(row + n) = v;
  } else {
    if (n < b) row[n] = v.x;
    if (n + 1 < b) row[n + 1] = v.y;
    if (n + 2 < b) row[n + 2] = v.z;
    if (n + 3 < b) row[n + 3] = v.w;
  }
}

template <int TS, bool VEC>
__device__ __forceinline__ void o_tile(const Params& p, int64_t id, float* sm) {
  using S = Shape<TS>;
  float* const As = sm;                    // [KBO][LDM]: D transposed
  float* const Bs = sm + S::KBO * S::LDM;  // [KBO][LDS]: G_j transposed
  const int n0 = static_cast<int>(id % p.tiles_b) * TS;
  id /= p.tiles_b;
  const int j = static_cast<int>(id % p.nblk), col = j * p.b;
  const int64_t m0 = id / p.nblk * S::TM;
  constexpr int VA = S::TM * S::KBO / 4, VB = TS * S::KBO / 4;
  constexpr int LA = (VA + S::NT - 1) / S::NT, LB = (VB + S::NT - 1) / S::NT;
  // vector i of an operand: 32 lanes take two vectors of 16 rows, so that the
  // four transposed stores of each meet 32 different banks
  auto k_of = [](int i) { return (i >> 5) % (S::KBO / 8) * 8 + (i & 1) * 4; };
  auto m_of = [](int i) { return (i >> 5) / (S::KBO / 8) * 16 + (i >> 1 & 15); };
  float4 a[LA], b[LB];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int l = 0; l < LA; ++l) {
      const int i = threadIdx.x + l * S::NT, k = k0 + k_of(i);
      const int64_t m = m0 + m_of(i);
      a[l] = load4<VEC>(p.D + m * p.d + col + k, (VA % S::NT == 0 || i < VA) && m < p.T ? p.b - k : 0);
    }
#pragma unroll
    for (int l = 0; l < LB; ++l) {
      const int i = threadIdx.x + l * S::NT, k = k0 + k_of(i), n = n0 + m_of(i);
      b[l] = load4<VEC>(p.G + (static_cast<int64_t>(col) + n) * p.b + k,
                        (VB % S::NT == 0 || i < VB) && n < p.b ? p.b - k : 0);
    }
  };
  auto stage = [&](float* to, int ld, int i, const float4& v) {
    float* at = to + k_of(i) * ld + m_of(i);
    at[0] = v.x;
    at[ld] = v.y;
    at[2 * ld] = v.z;
    at[3 * ld] = v.w;
  };
  int ty, tx;
  place<S::C>(threadIdx.x, ty, tx);
  float acc[4][4] = {};
  fetch(0);
  for (int k0 = 0; k0 < p.b; k0 += S::KBO) {
#pragma unroll
    for (int l = 0; l < LA; ++l) {
      const int i = threadIdx.x + l * S::NT;
      if (VA % S::NT == 0 || i < VA) stage(As, S::LDM, i, a[l]);
    }
#pragma unroll
    for (int l = 0; l < LB; ++l) {
      const int i = threadIdx.x + l * S::NT;
      if (VB % S::NT == 0 || i < VB) stage(Bs, S::LDS, i, b[l]);
    }
    __syncthreads();
    if (k0 + S::KBO < p.b) fetch(k0 + S::KBO);
#pragma unroll 8
    for (int k = 0; k < S::KBO; ++k)
      fma4x4(acc, As + k * S::LDM + 4 * ty, Bs + k * S::LDS + 4 * tx);
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t m = m0 + 4 * ty + r;
    if (m < p.T)
      put_row<VEC>(p.O + m * p.d + col, make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]), n0 + 4 * tx, p.b);
  }
}

template <int TS, bool VEC>
__device__ __forceinline__ void dg_tile(const Params& p, int64_t id, float* sm) {
  using S = Shape<TS>;
  float* const As = sm;                    // [KBG][LDS]: X
  float* const Bs = sm + S::KBG * S::LDS;  // [KBG][LDS]: D
  const int n0 = static_cast<int>(id % p.tiles_b) * TS;
  id /= p.tiles_b;
  const int m0 = static_cast<int>(id % p.tiles_b) * TS;
  id /= p.tiles_b;                         // split * nblk + j
  const int j = static_cast<int>(id % p.nblk), col = j * p.b;
  const int64_t s = id / p.nblk;
  const int64_t k_first = s * p.T / p.splits, k_last = (s + 1) * p.T / p.splits;
  constexpr int V = S::KBG * TS / 4, L = (V + S::NT - 1) / S::NT;
  uint32_t q[L], eb[L];                    // four codes; their exponents
  float4 b[L];
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int i = threadIdx.x + l * S::NT, c = i % (TS / 4) * 4;
      const int64_t k = k0 + i / (TS / 4);
      const bool in = (V % S::NT == 0 || i < V) && k < k_last;
      b[l] = load4<VEC>(p.D + k * p.d + col + n0 + c, in ? p.b - n0 - c : 0);
      const int left = in ? p.b - m0 - c : 0, at = col + m0 + c;
      const int8_t* x = p.codes + k * p.d + at;
      const uint8_t* e = p.exps + k * p.ng;
      q[l] = eb[l] = 0;
      if (VEC) {
        if (left > 0) {
          q[l] = *reinterpret_cast<const uint32_t*>(x);
          eb[l] = e[at / q8::GROUP];
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (h < left) {
            q[l] |= static_cast<uint32_t>(static_cast<uint8_t>(x[h])) << 8 * h;
            eb[l] |= static_cast<uint32_t>(e[(at + h) / q8::GROUP]) << 8 * h;
          }
      }
    }
  };
  auto decode = [](uint32_t w, uint32_t ew, int h) {
    return static_cast<float>(static_cast<int8_t>(w >> 8 * h)) * q8::exponent_value(VEC ? ew : ew >> 8 * h & 0xffu);
  };
  const int g = threadIdx.x / (S::C * S::C);
  int ty, tx;
  place<S::C>(threadIdx.x % (S::C * S::C), ty, tx);
  float acc[4][4] = {};
  fetch(k_first);
  for (int64_t k0 = k_first; k0 < k_last; k0 += S::KBG) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int i = threadIdx.x + l * S::NT, at = i / (TS / 4) * S::LDS + i % (TS / 4) * 4;
      if (V % S::NT != 0 && i >= V) continue;
      *reinterpret_cast<float4*>(As + at) =
          make_float4(decode(q[l], eb[l], 0), decode(q[l], eb[l], 1), decode(q[l], eb[l], 2), decode(q[l], eb[l], 3));
      *reinterpret_cast<float4*>(Bs + at) = b[l];
    }
    __syncthreads();
    if (k0 + S::KBG < k_last) fetch(k0 + S::KBG);
#pragma unroll 8
    for (int k = 0; k < S::KBG / S::GR; ++k) {
      const int row = (k * S::GR + g) * S::LDS;
      fma4x4(acc, As + row + 4 * ty, Bs + row + 4 * tx);
    }
    __syncthreads();
  }
  float* const out = p.part + id * p.b * static_cast<int64_t>(p.b);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    *reinterpret_cast<float4*>(sm + (g * TS + 4 * ty + r) * TS + 4 * tx) =
        make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  __syncthreads();
  for (int i = threadIdx.x; i < TS * TS; i += S::NT) {
    float v = sm[i];
#pragma unroll
    for (int h = 1; h < S::GR; ++h) v += sm[h * TS * TS + i];
    const int m = m0 + i / TS, n = n0 + i % TS;
    if (m < p.b && n < p.b) out[static_cast<int64_t>(m) * p.b + n] = v;
  }
}

template <int TS, bool VEC>
__global__ void __launch_bounds__(Shape<TS>::NT, Shape<TS>::BLOCKS) block_backward_kernel(const Params p) {
  __shared__ __align__(16) float sm[Shape<TS>::WORDS];
  if (blockIdx.x < p.o_blocks) o_tile<TS, VEC>(p, blockIdx.x, sm);
  else dg_tile<TS, VEC>(p, blockIdx.x - p.o_blocks, sm);
}

}  // namespace bf32
}  // namespace poetx
