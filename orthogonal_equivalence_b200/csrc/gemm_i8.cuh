// Int8 products of the POET-XQ weight (codes Wq [n][m], a scale per row) on
// the tensor cores (tcgen05 kind::i8, 32-bit integer accumulators in TMEM):
//   forward   z[t][j]  = xs[t] ws[j] sum_i xq[t][i] Wq[j][i]
//   gradient  dx[t][i] = gs[t]       sum_j gq[t][j] Wq[j][i]
// The sums are exact (|code| <= 128 and at most 102400 terms stay below
// 2^31), so neither a split of K nor its order changes a result.
//
// Wq is stored once, [n][m]: the forward reads it K-major, the gradient
// MN-major (the contraction runs over its rows), both by TMA in 128-byte
// swizzled boxes of 128 rows.
//
//   pair kernel: 256 x 256 tiles on CTA pairs, persistent; for many tokens.
//   wide kernel: the weight's 128 rows are the M side of the tile and up to
//     128 tokens its N side, K split over a cluster whose CTAs add their
//     integer sums over distributed shared memory; for few tokens, where all
//     SMs are needed to stream the weight.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "gemm2sm.cuh"
#include "perm.cuh"

namespace poetx {
namespace i8 {

constexpr int KB = 128;          // K per stage: 128 codes = one 128-byte row
constexpr int UMMA_K = 32;
constexpr int BOX_BYTES = 128 * 128;

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 integers of a TMEM row: the accumulators as loaded by tmem_ld_32cols.
__device__ __forceinline__ int as_int(float v) { return __float_as_int(v); }

// A block of 32 columns' scales from column c on (1 where there are none or no such column).
__device__ __forceinline__ void load_scales(const float* bs, int c, int N, float* b) {
  if (bs && c + 32 <= N) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(bs + c) + q);
      b[4 * q] = f.x;
      b[4 * q + 1] = f.y;
      b[4 * q + 2] = f.z;
      b[4 * q + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) b[e] = bs && c + e < N ? __ldg(bs + c + e) : 1.f;
  }
}

// A box (32 rows of 128 bytes, swizzled) to rows of N elements that start
// anywhere, a word of the box a lane: bf16 rows on an odd element go out as the
// pairs between their words, and the elements left over singly.
template <typename T>
__device__ __forceinline__ void store_box(uint32_t box, T* out, int64_t row0, int rows, int col0, int N, int lane) {
  const int cols = min(static_cast<int>(128 / sizeof(T)), N - col0);
  T* dst = out + row0 * N + col0;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8) {
    uint32_t w[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(w[r])
                   : "r"(box + (r0 + r) * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4)
                   : "memory");
#pragma unroll
    for (int r = 0; r < 8; ++r, dst += N) {
      if constexpr (sizeof(T) == 4) {
        if (r0 + r < rows && lane < cols) dst[lane] = __uint_as_float(w[r]);
      } else {
        const int odd = (reinterpret_cast<uintptr_t>(dst) >> 1) & 1, c = 2 * lane + odd;
        const uint32_t next = __shfl_down_sync(0xffffffffu, w[r], 1);
        const uint32_t v = odd ? __funnelshift_r(w[r], next, 16) : w[r];
        if (r0 + r < rows) {
          if (c + 1 < cols) *reinterpret_cast<uint32_t*>(dst + c) = v;
          if (c + 1 == cols) dst[c] = __ushort_as_bfloat16(static_cast<unsigned short>(v));
          if (odd && lane == 0) dst[0] = __ushort_as_bfloat16(static_cast<unsigned short>(w[r]));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- many tokens
constexpr int STAGES = 6;
constexpr int STAGE_BYTES = 2 * BOX_BYTES;  // this CTA's 128 tokens and 128 columns
constexpr int EPI_BOX = 32 * 128;
constexpr int EPI_WARPS = 8;                // two a quarter of the rows, half the columns each
constexpr int EPI_BYTES = EPI_WARPS * EPI_BOX;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + 256;
constexpr int PAIR_THREADS = 64 + 32 * EPI_WARPS;

struct PairParams {
  tc2::Params g;        // sizes, raster, instruction descriptor
  const float* as;      // [M] token scales
  const float* bs;      // [N] channel scales or NULL
  void* out;            // [M][N]
  int tma_out;          // rows of out are whole 16-byte units: TMA store
};

// Warp roles, barriers and raster as in the bf16 W0 product (gemm2sm.cuh); a
// stage holds twice the K in the same bytes.  The epilogue turns 32 x 128
// bytes of output at a time (64 bf16 or 32 fp32 columns) into a swizzled box
// and stores it by TMA, or row by row when out's rows are not 16-byte units.
// With a short K it is the epilogue that bounds the product: 16384 x 96 -> 14336
// takes 165 us (72 at the copy rate) with eight warps whose scales are loaded a
// block of columns ahead, 228 with four, and 430 with four that wait for them.
// Bound by the tensor pipe and the power cap: 16384 x 4096 -> 14336 takes 619 us
// (3.1 POP/s, the pipe 84% active) in a short run and 690 to 730 in a long one,
// the gradient's product 8192 x 14336 -> 4096 294 us (91%).  Asking L2 for operands
// ahead of the stages costs 10% (the way from L2 to the SMs is nearly full too).
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmC, const PairParams pp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + EPI_BYTES);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  const tc2::Params& p = pp.g;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = tc2::cluster_rank();
  const bool leader = rank == 0;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t sEpi = smem_base + STAGES * STAGE_BYTES;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = 2 * STAGES + 2, DRAIN = 2 * STAGES + 4;
  constexpr int BM = tc2::BM, BN = tc2::BN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(FULL + s), 1);
      mbar_init(bar(EMPTY + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(TFULL + a), 1);
      mbar_init(bar(TEMPTY + a), 2 * EPI_WARPS);  // of both CTAs
    }
    mbar_init(bar(DRAIN), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(tc2::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  tc2::cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const int total = p.tiles_m * p.tiles_n;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nkb = (p.K + KB - 1) / KB;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        int mt, nt;
        tc2::decode(p, tile, mt, nt);
        const int m0 = mt * BM + rank * 128, n0 = nt * BN + rank * 128;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(bar(EMPTY + stage), phase ^ 1u, DERR_GEMM_WAIT)) { ok = false; break; }
          const uint32_t full_leader = tc2::map_to_rank(bar(FULL + stage), 0);
          if (leader) mbar_arrive_expect_tx(bar(FULL + stage), 2 * STAGE_BYTES);
          const uint32_t sa = smem_base + stage * STAGE_BYTES, sb = sa + BOX_BYTES;
          const int k = kb * KB;
          tc2::tma_load_2d_pair(sa, &tmA, full_leader, k, m0);
          if (!p.b_mn) tc2::tma_load_2d_pair(sb, &tmB, full_leader, k, n0);
          else tc2::tma_load_2d_pair(sb, &tmB, full_leader, n0, k);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 100000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      // ---------------- MMA issuer (leader CTA, for both)
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs, ++local) {
        const int acc = local & 1;
        const uint32_t acc_phase = (local >> 1) & 1;
        if (!mbar_wait(bar(TEMPTY + acc), acc_phase ^ 1u, DERR_GEMM_WAIT)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(bar(FULL + stage), phase, DERR_GEMM_WAIT)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_base + stage * STAGE_BYTES, sb = sa + BOX_BYTES;
#pragma unroll
          for (int kk = 0; kk < KB / UMMA_K; ++kk)
            mma_pair(d_tmem, smem_desc_sw128(sa + kk * UMMA_K, 16, 1024),
                     smem_desc_sw128(sb + kk * p.b_kstep, 16, 1024), p.idesc, (kb | kk) != 0 ? 1u : 0u);
          tc2::commit_pair(bar(EMPTY + stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc2::commit_pair(bar(TFULL + acc));
      }
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar(DRAIN))
                   : "memory");
      mbar_wait(bar(DRAIN), 0, DERR_GEMM_WAIT);
    }
  } else {
    // ---------------- epilogue (both CTAs): this CTA's 128 rows of each tile
    constexpr int CW = 128 / sizeof(T);  // columns of a box
    const int quarter = warp & 3, first = (warp - 2) / 4 * (BN / 2);  // rows, and columns of the tile
    const uint32_t box = sEpi + (warp - 2) * EPI_BOX;
    const uint32_t tempty_leader = tc2::map_to_rank(bar(TEMPTY), 0);
    // the scales of a tile's rows and of the next 32 columns are loaded ahead
    auto token_scale = [&](int tile) {
      int mt, nt;
      tc2::decode(p, tile, mt, nt);
      const int row = mt * BM + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      return row < p.M ? __ldg(pp.as + row) : 0.f;
    };
    auto first_col = [&](int tile) {
      int mt, nt;
      tc2::decode(p, tile, mt, nt);
      return nt * BN + first;
    };
    float as_next = 0.f, b[32];
    if (pair < total) {
      as_next = token_scale(pair);
      load_scales(pp.bs, first_col(pair), p.N, b);
    }
    int local = 0;
    for (int tile = pair; tile < total; tile += npairs, ++local) {
      int mt, nt;
      tc2::decode(p, tile, mt, nt);
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      const int row0 = mt * BM + rank * 128 + quarter * 32;
      const float as = as_next;
      const int next = tile + npairs;
      if (next < total) as_next = token_scale(next);
      const int next_col = next < total ? first_col(next) : p.N;
      bool ok = mbar_wait(bar(TFULL + acc), acc_phase, DERR_GEMM_WAIT);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const bool rows_in = row0 < p.M;
      const uint32_t tl = tmem_base + acc * BN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c0 = first; c0 < first + BN / 2; c0 += CW) {
        const int col0 = nt * BN + c0;
        uint32_t w[32];
#pragma unroll
        for (int half = 0; half < CW / 32; ++half) {
          float v[32];
          tmem_ld_32cols(tl + c0 + 32 * half, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = static_cast<float>(as_int(v[e])) * as * b[e];
          load_scales(pp.bs, c0 + 32 * half + 32 < first + BN / 2 ? col0 + 32 * half + 32 : next_col, p.N, b);
          if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[16 * half + i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
          }
        }
        if (c0 + CW == first + BN / 2) {  // this warp's part of the accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) tc2::remote_arrive(tempty_leader + 8 * acc);
        }
        if (!rows_in || col0 >= p.N) continue;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        const uint32_t rowp = box + lane * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(rowp + ((k ^ (lane & 7)) << 4)),
                       "r"(w[4 * k]), "r"(w[4 * k + 1]), "r"(w[4 * k + 2]), "r"(w[4 * k + 3])
                       : "memory");
        if (pp.tma_out) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmC, box, col0, row0);
            bulk_commit();
          }
        } else {
          __syncwarp();
          store_box<T>(box, static_cast<T*>(pp.out), row0, min(32, p.M - row0), col0, p.N, lane);
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  tc2::cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(tc2::TMEM_COLS)
                 : "memory");
  }
  tc2::cluster_sync();
}

// ---------------------------------------------------------------- few tokens
constexpr int NUM_THREADS = 192;

struct WideParams {
  const float* as;      // [T] token scales
  const float* bs;      // [N] scales of the weight's side or NULL
  void* out;            // [T][N]
  int T, N, K;
  int nt;               // tokens per tile: 16, 32, 64 or 128
  int stages;
  int w_mn;             // the weight's K is its rows (gradient)
  uint32_t idesc;
  int tmem_cols;
};

// Programmatic dependent launch: a kernel launched with that attribute may
// start, and set up its barriers and TMEM, once every CTA of the kernel before
// it has called grid_launch or ended; grid_wait returns when that kernel has
// completed and its writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Grid (S, ceil(N / 128), ceil(T / nt)), clusters of the S CTAs of one tile.
// CTA s takes the K blocks [s nkb / S, (s + 1) nkb / S), S <= nkb.  For a few
// tokens the weight's bytes bound it: 1 x 4096 -> 14336 takes 12.7 us in a graph
// and 13.3 called one after the other (9.0 at the copy rate), 48 x 14336 -> 4096
// 14.0 and 15.4 (9.2); what is left over is the launch, the first loads' way and
// the sums' exchange.  With more tokens the epilogue
// (one weight row a thread) counts, which is why the tiles stay narrow.
template <typename T>
__global__ void __launch_bounds__(NUM_THREADS)
    product_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const WideParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = BOX_BYTES + p.nt * KB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * p.stages + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  auto full = [&](int i) { return smem_u32(bars + i); };
  auto empty = [&](int i) { return smem_u32(bars + p.stages + i); };
  const uint32_t done = smem_u32(bars + 2 * p.stages);
  const int S = gridDim.x, rank = blockIdx.x;
  const int n0 = blockIdx.y * 128, t0 = blockIdx.z * p.nt;

  const int nkb = (p.K + KB - 1) / KB;
  const int k_first = static_cast<int>(int64_t(rank) * nkb / S), k_last = static_cast<int>(int64_t(rank + 1) * nkb / S);

  auto load = [&](int kb, int stage) {
    const uint32_t sw = smem_base + stage * stage_bytes;
    mbar_arrive_expect_tx(full(stage), stage_bytes);
    if (!p.w_mn) tma_load_2d(sw, &tmW, full(stage), kb * KB, n0);
    else tma_load_2d(sw, &tmW, full(stage), n0, kb * KB);
    tma_load_2d(sw + BOX_BYTES, &tmX, full(stage), kb * KB, t0);
  };
  const int k_early = min(k_last, k_first + p.stages);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    fence_async_smem();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    grid_wait();
    // the first round of loads flies while TMEM is allocated
    for (int kb = k_first; kb < k_early; ++kb) load(kb, kb - k_first);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_wait();    // before any thread reads or writes what earlier kernels of the stream do
  grid_launch();  // the next kernel may set itself up

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;  // the slot's first reader has to be done
      for (int kb = k_early; kb < k_last; ++kb) {
        if (!mbar_wait(empty(stage), phase, DERR_GEMM_WAIT)) {
          const uint64_t s0 = global_ns();
          while (global_ns() - s0 < 100000ull) {
          }
          break;
        }
        load(kb, stage);
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      const int wstep = p.w_mn ? UMMA_K * 128 : UMMA_K;
      for (int kb = k_first; kb < k_last; ++kb) {
        if (!mbar_wait(full(stage), phase, DERR_GEMM_WAIT)) break;
        tc_fence_after();
        const uint32_t sw = smem_base + stage * stage_bytes, sx = sw + BOX_BYTES;
#pragma unroll
        for (int kk = 0; kk < KB / UMMA_K; ++kk)
          mma_one(tmem_base, smem_desc_sw128(sw + kk * wstep, 16, 1024), smem_desc_sw128(sx + kk * UMMA_K, 16, 1024),
                  p.idesc, (kb != k_first || kk != 0) ? 1u : 0u);
        tc_commit(empty(stage));
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
      tc_commit(done);
    }
  }
  __syncwarp();
  const int quarter = warp & 3, row = quarter * 32 + lane;
  const int cols = min(p.nt, p.T - t0);
  const uint32_t tl = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
  T* out = static_cast<T*>(p.out) + static_cast<int64_t>(t0) * p.N + n0;
  const float* as = p.as + t0;
  const bool row_in = n0 + row < p.N;
  float bs = 1.f;
  if (warp >= 2 && p.bs && row_in) bs = p.bs[n0 + row];
  int* part = reinterpret_cast<int*>(smem);  // [cols][128], over the stages once every MMA has read them
  if (warp >= 2) {
    bool ok = mbar_wait(done, 0, DERR_GEMM_WAIT);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      for (int c0 = 0; c0 < cols; c0 += 32) {
        float v[32];
        tmem_ld_32cols(tl + c0, v);
        if (S == 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i < cols && row_in)
              out[static_cast<int64_t>(c0 + i) * p.N + row] =
                  from_f32<T>(static_cast<float>(as_int(v[i])) * __ldg(as + c0 + i) * bs);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i < cols) part[(c0 + i) * 128 + row] = as_int(v[i]);
        }
      }
      tc_fence_before();
    }
  }
  if (S > 1) {
    // add the S integer sums of the tile: this CTA the token columns rank,
    // rank + S, ..., a warp one of them at a time, four weight rows a lane; all
    // S reads of a column are in flight together
    tc2::cluster_sync();
    if (warp >= 2) {
      const int j = n0 + lane * 4;
      const bool whole = p.N % 4 == 0 && j < p.N;  // (then all four rows are inside)
      float b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = p.bs && j + e < p.N ? p.bs[j + e] : 1.f;
      const uint32_t mine = smem_u32(part) + lane * 16;
      for (int c = rank + S * (warp - 2); c < cols; c += 4 * S) {
        int v[8][4];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if (s < S)
            asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[s][0]), "=r"(v[s][1]), "=r"(v[s][2]), "=r"(v[s][3])
                         : "r"(tc2::map_to_rank(mine + c * 512, s))
                         : "memory");
          else v[s][0] = v[s][1] = v[s][2] = v[s][3] = 0;
        }
        const float a = __ldg(as + c);
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int sum = 0;
#pragma unroll
          for (int s = 0; s < 8; ++s) sum += v[s][e];
          o[e] = static_cast<float>(sum) * a * b[e];
        }
        T* dst = out + static_cast<int64_t>(c) * p.N + lane * 4;
        if (whole) {
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
          else
            *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < p.N) dst[e] = from_f32<T>(o[e]);
        }
      }
    }
    tc2::cluster_sync();  // no CTA leaves while its sums are read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// Rows of `cols` bytes copied to rows `ld` apart (ld a multiple of 16, the
// bytes behind cols unwritten), for operands whose rows are not whole 16-byte
// units and so cannot be read by TMA.  A thread builds 16 bytes from the five
// aligned words that hold them.
__global__ void __launch_bounds__(256) pad_rows_kernel(const int8_t* __restrict__ src, int64_t rows, int cols,
                                                       int8_t* __restrict__ dst, int64_t ld) {
  const int per = (cols + 15) / 16;
  const int64_t n = rows * per, size = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / per;
    const int c = static_cast<int>(i - r * per) * 16;
    const int64_t at = r * cols + c;
    uint4 w;
    uint32_t* o = reinterpret_cast<uint32_t*>(&w);
    if (at + 20 <= size) {
      const uint32_t* a = reinterpret_cast<const uint32_t*>(src + (at & ~int64_t(3)));
      const uint32_t sh = static_cast<uint32_t>(at & 3) * 8;
      uint32_t lo = a[0];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t hi = a[k + 1];
        o[k] = __funnelshift_r(lo, hi, sh);
        lo = hi;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k] = 0;
        for (int e = 0; e < 4; ++e)
          if (at + 4 * k + e < size) o[k] |= static_cast<uint32_t>(static_cast<uint8_t>(src[at + 4 * k + e])) << (8 * e);
      }
    }
    *reinterpret_cast<uint4*>(dst + r * ld + c) = w;
  }
}

}  // namespace i8
}  // namespace poetx
