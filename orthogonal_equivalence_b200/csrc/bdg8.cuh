// Backward of one side of the layer (POET-X write-up, section 1: the block
// products of R or P) from an 8-bit checkpoint of its activation, in one kernel
// on CTA pairs, for b = 256 bf16 layers:
//   O_j = D_j G_j^T
//   part[s][j] = X_j^T D_j       (over the tokens of split s)
// as in bdg2sm.cuh, except that X [T][d] is read as int8 codes with one
// exponent per 32 columns (q8.cuh): 1.03 bytes an element instead of 2, and no
// bf16 copy of X in memory.  The tensor cores have no int8 x bf16 product, so
// eight warps turn the codes into the bf16 operand tile in shared memory; code *
// 2^e is exact in bf16, so the product sees the checkpoint's own values.
//
// A pair of SMs takes a work item (block j, token split s) and walks its
// 256-token tiles; the two products of a tile and its accumulators are laid
// out as in bdg2sm.cuh.  Shared memory of a CTA: its 128 rows of G_j (64 KB,
// resident for the item), a ring of 16 KB units for D (four K-major ones for
// MMA1, four MN-major ones for MMA2 per tile), one of 8 KB slots for codes, one
// of 16 KB units for converted X, and the epilogue's boxes.
//
// Token sums: the tensor core cuts off rather than rounds what an addition
// shifts out, which biases a sum of many terms towards zero (dG of 16384 tokens,
// normal values: off by 7.0e-6 as one sum, 2.8e-6 as two, 1.1e-6 as four, 4e-7 as
// eight or nine), so a split takes about 2048 tokens at most.
//
//   warp 0: TMA producer (both CTAs)
//   warp 1: TMEM owner (both CTAs) and MMA issuer (leader only)
//   warps 2-5: epilogues (both CTAs)
//   warps 6-13: codes -> bf16 (both CTAs)
//   warp 14: producer of the codes and exponents (both CTAs)
//
// The arrivals at the leader's barriers that stand for shared-memory writes or
// TMEM reads of this SM use the plain remote arrive: after the proxy fence (or
// tcgen05 fence) the data is in place in this SM's own memory, which is the
// only place the pair's MMA reads it from, so nothing has to be released to the
// rest of the cluster.  A release at cluster scope waits for the memory system:
// with one per chunk and warp the kernel took 155 us instead of 120.
//
// The exponents come to shared memory beside their codes, copied without a
// register in between: loaded into registers, even a tile ahead, they held up
// the converting warps (16384 x 4096 without O: 63 us instead of 54).  G_j is
// released, and the next one loaded, before the last tile's dG; an item's first
// O is computed while the dG before it is written.
//
// 16384 x 4096 takes 87 us with the sum of the nine splits and 58 us without O
// (53 and 32 us at the copy rate) at 1965 MHz, and 98 to 103 us back to back for
// seconds, when the power cap (990 W drawn, sw_power_cap) holds the SMs at 1590
// MHz.  Neither HBM (50%) nor the tensor pipe (48%) is the bound, nor the conversion
// (left out: 5 us less; with four warps 9 us more): the O tiles' way through
// registers and boxes and the ends of the items are; deeper rings of any of the
// three operands change nothing.
// Every wait is bounded (ptx.cuh).  No load uses multicast.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "bdg2sm.cuh"
#include "q8.cuh"

namespace poetx {
namespace bdg8 {

using bdg2::BLK;
using bdg2::CH;
using bdg2::EPI_BOX;
using bdg2::EPI_BYTES;
using bdg2::G_BYTES;
using bdg2::HALF;
using bdg2::TILE_BYTES;
using bdg2::UMMA_K;
constexpr int UNITS = 4;                        // ring of D units (TILE_BYTES each)
constexpr int XUNITS = 2;                       // converted X
constexpr int SLOTS = 4;                        // codes
constexpr int SLOT_BYTES = CH * HALF;           // 64 tokens x 128 codes
constexpr int EXP_BYTES = CH * 4;               // and their exponents, one word a token
constexpr int SMEM_BYTES =
    (UNITS + XUNITS) * TILE_BYTES + SLOTS * (SLOT_BYTES + EXP_BYTES) + G_BYTES + EPI_BYTES + 1024 + 320;
constexpr int NUM_THREADS = 480;
constexpr int CONV_WARPS = 8;
constexpr int SPLIT_TOKENS = 2048;              // most tokens of a split (see above), about

struct Params {
  bdg2::Params g;
  const uint8_t* exps;  // [T][ng]
  int ng;               // d / 32
};

// Arrive at a barrier of either CTA of the pair (see above).
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Eight codes (two words) times s as bf16, packed.  A byte code + 128 under the
// exponent of 2^23 is the fp32 number 2^23 + 128 + code; one FMA with s and
// (2^23 + 128) s gives code * s without a rounding (two at a time), as long as
// (2^23 + 128) s is finite: FAR takes the others, 2^100 and up.
__device__ __forceinline__ uint32_t fma_pair(float x, float y, uint64_t s2, uint64_t c2) {
  uint32_t r;
  asm("{\n\t.reg .b64 v;\n\t.reg .f32 a, b;\n\t"
      "mov.b64 v, {%1, %2};\n\t"
      "fma.rn.f32x2 v, v, %3, %4;\n\t"
      "mov.b64 {a, b}, v;\n\t"
      "cvt.rn.bf16x2.f32 %0, b, a;\n\t}"
      : "=r"(r)
      : "f"(x), "f"(y), "l"(s2), "l"(c2));
  return r;
}
__device__ __forceinline__ uint64_t twice(float f) {
  const uint64_t b = __float_as_uint(f);
  return b << 32 | b;
}
template <bool FAR>
__device__ __forceinline__ uint4 expand8(uint32_t w0, uint32_t w1, float s) {
  uint32_t o[4];
  const uint64_t s2 = twice(s), c2 = twice(-8388736.f * s);
  const uint32_t b[2] = {w0 ^ 0x80808080u, w1 ^ 0x80808080u};  // code + 128
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(__byte_perm(b[i], 0x4b000000u, 0x7540 + e));
    if (FAR) {
      o[2 * i] = pack_bf16x2((f[0] - 8388736.f) * s, (f[1] - 8388736.f) * s);
      o[2 * i + 1] = pack_bf16x2((f[2] - 8388736.f) * s, (f[3] - 8388736.f) * s);
    } else {
      o[2 * i] = fma_pair(f[0], f[1], s2, c2);
      o[2 * i + 1] = fma_pair(f[2], f[3], s2, c2);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Four bytes to shared memory without a register in between, zeros if !in.
__device__ __forceinline__ void copy_word(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// An arrival at `bar` (of this CTA) once this thread's copies so far are in place.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    bdg8_pair_kernel(const __grid_constant__ CUtensorMap tmDk, const __grid_constant__ CUtensorMap tmDmn,
                     const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmPart,
                     const Params pp) {
  const bdg2::Params& p = pp.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t sX = smem_base + UNITS * TILE_BYTES;
  const uint32_t sG = sX + XUNITS * TILE_BYTES;
  const uint32_t sEpi = sG + G_BYTES;
  const uint32_t sCode = sEpi + EPI_BYTES;
  const uint32_t sExp = sCode + SLOTS * SLOT_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (sExp - smem_base) + SLOTS * EXP_BYTES);
  // full[UNITS] (leader), empty[UNITS], xfull[XUNITS] (leader), xempty[XUNITS], cfull[SLOTS],
  // cempty[SLOTS], gfull (leader), gempty, ofull, oempty (leader), afull, aempty (leader)
  constexpr int FULL = 0, EMPTY = UNITS, XFULL = 2 * UNITS, XEMPTY = XFULL + XUNITS, CFULL = XEMPTY + XUNITS,
                CEMPTY = CFULL + SLOTS, GFULL = CEMPTY + SLOTS,
                GEMPTY = GFULL + 1, OFULL = GFULL + 2, OEMPTY = GFULL + 3, AFULL = GFULL + 4, AEMPTY = GFULL + 5,
                NBARS = GFULL + 6;
  static_assert((NBARS + 1) * 8 <= 320, "barriers do not fit");
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = tc2::cluster_rank();
  const bool leader = rank == 0;
  auto bar = [&](int i) { return smem_u32(bars + i); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < UNITS; ++s) {
      mbar_init(bar(FULL + s), 1);
      mbar_init(bar(EMPTY + s), 1);
    }
    for (int s = 0; s < XUNITS; ++s) {
      mbar_init(bar(XFULL + s), 2 * CONV_WARPS);  // of both CTAs
      mbar_init(bar(XEMPTY + s), 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(bar(CFULL + s), 1 + 32);  // the codes' bytes, and each lane's exponents
      mbar_init(bar(CEMPTY + s), CONV_WARPS);
    }
    mbar_init(bar(GFULL), 1);
    mbar_init(bar(GEMPTY), 1);
    mbar_init(bar(OFULL), 1);
    mbar_init(bar(OEMPTY), 8);  // 4 epilogue warps x 2 CTAs
    mbar_init(bar(AFULL), 1);
    mbar_init(bar(AEMPTY), 8);
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  tc2::cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const int items = p.nblk * p.splits;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      prefetch_tmap(&tmDk);
      prefetch_tmap(&tmDmn);
      prefetch_tmap(&tmG);
      int unit = 0;
      uint32_t ring = 0;
      int local = 0;
      bool ok = true;
      // next unit of D, `bytes` from each CTA
      auto next_unit = [&]() -> bool {
        if (!mbar_wait(bar(EMPTY + unit), ring ^ 1u, DERR_GEMM_WAIT)) return false;
        if (leader) mbar_arrive_expect_tx(bar(FULL + unit), 2 * TILE_BYTES);
        return true;
      };
      auto advance = [&]() {
        if (++unit == UNITS) {
          unit = 0;
          ring ^= 1u;
        }
      };
      for (int item = pair; item < items && ok; item += npairs, ++local) {
        const int j = item % p.nblk, s = item / p.nblk;
        int ta, tb;
        bdg2::split_tiles(p, s, ta, tb);
        const int fcol = j * BLK + int(rank) * HALF;  // this CTA's feature columns of block j
        if (p.want_o) {
          // this CTA's rows of G_j, resident for the item
          if (!mbar_wait(bar(GEMPTY), (local & 1) ^ 1u, DERR_GEMM_WAIT)) { ok = false; break; }
          const uint32_t gfull = tc2::map_to_rank(bar(GFULL), 0);
          if (leader) mbar_arrive_expect_tx(bar(GFULL), 2 * G_BYTES);
          for (int c = 0; c < 4; ++c) tc2::tma_load_2d_pair(sG + c * TILE_BYTES, &tmG, gfull, c * CH, fcol);
        }
        for (int tile = ta; tile < tb && ok; ++tile) {
          const int tok = tile * BLK;
          if (p.want_o) {
            for (int c = 0; c < 4; ++c) {
              if (!next_unit()) { ok = false; break; }
              tc2::tma_load_2d_pair(smem_base + unit * TILE_BYTES, &tmDk, tc2::map_to_rank(bar(FULL + unit), 0),
                                    j * BLK + c * CH, tok + int(rank) * HALF);
              advance();
            }
          }
          for (int c = 0; c < 4 && ok; ++c) {
            if (!next_unit()) { ok = false; break; }
            const uint32_t full = tc2::map_to_rank(bar(FULL + unit), 0);
            const uint32_t sb = smem_base + unit * TILE_BYTES;
            const int row = tok + c * CH;
            tc2::tma_load_2d_pair(sb, &tmDmn, full, fcol, row);
            tc2::tma_load_2d_pair(sb + CH * 128, &tmDmn, full, fcol + CH, row);
            advance();
          }
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
      // ---------------- MMA issuer (leader, for both CTAs)
      const uint32_t accO = tmem_base, accG = tmem_base + BLK;
      int unit = 0, xu = 0;
      uint32_t ring = 0, xring = 0;
      int local = 0, otiles = 0;
      bool ok = true;
      for (int item = pair; item < items && ok; item += npairs, ++local) {
        const int s = item / p.nblk;
        int ta, tb;
        bdg2::split_tiles(p, s, ta, tb);
        if (p.want_o && !mbar_wait(bar(GFULL), local & 1, DERR_GEMM_WAIT)) { ok = false; break; }
        tc_fence_after();
        for (int tile = ta; tile < tb && ok; ++tile) {
          if (p.want_o) {
            if (!mbar_wait(bar(OEMPTY), (otiles & 1) ^ 1u, DERR_GEMM_WAIT)) { ok = false; break; }
            tc_fence_after();
            for (int c = 0; c < 4; ++c) {
              if (!mbar_wait(bar(FULL + unit), ring, DERR_GEMM_WAIT)) { ok = false; break; }
              tc_fence_after();
              const uint32_t sa = smem_base + unit * TILE_BYTES, sg = sG + c * TILE_BYTES;
#pragma unroll
              for (int kk = 0; kk < CH / UMMA_K; ++kk)
                tc2::mma_pair(accO, smem_desc_sw128(sa + kk * 32, 16, 1024), smem_desc_sw128(sg + kk * 32, 16, 1024),
                              p.idesc_kk, (c | kk) != 0 ? 1u : 0u);
              tc2::commit_pair(bar(EMPTY + unit));
              if (++unit == UNITS) { unit = 0; ring ^= 1u; }
            }
            if (!ok) break;
            tc2::commit_pair(bar(OFULL));
            if (tile == tb - 1) tc2::commit_pair(bar(GEMPTY));  // G_j no longer read
            ++otiles;
          }
          // the item before this one has left accG (its dG is written while this one's first O is computed)
          if (tile == ta && !mbar_wait(bar(AEMPTY), (local & 1) ^ 1u, DERR_GEMM_WAIT)) { ok = false; break; }
          for (int c = 0; c < 4; ++c) {
            if (!mbar_wait(bar(FULL + unit), ring, DERR_GEMM_WAIT)) { ok = false; break; }
            if (!mbar_wait(bar(XFULL + xu), xring, DERR_GEMM_WAIT)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = sX + xu * TILE_BYTES, sb = smem_base + unit * TILE_BYTES;
#pragma unroll
            for (int kk = 0; kk < CH / UMMA_K; ++kk)
              tc2::mma_pair(accG, smem_desc_sw128(sa + kk * (UMMA_K * 128), CH * 128, 1024),
                            smem_desc_sw128(sb + kk * (UMMA_K * 128), CH * 128, 1024), p.idesc_mnmn,
                            (tile != ta || c != 0 || kk != 0) ? 1u : 0u);
            tc2::commit_pair(bar(EMPTY + unit));
            tc2::commit_pair(bar(XEMPTY + xu));
            if (++unit == UNITS) { unit = 0; ring ^= 1u; }
            if (++xu == XUNITS) { xu = 0; xring ^= 1u; }
          }
        }
        if (!ok) break;
        tc2::commit_pair(bar(AFULL));  // every MMA of the item is done
      }
    }
  } else if (warp == 6 + CONV_WARPS) {
    // ---------------- producer of the codes (TMA) and their exponents (both CTAs)
    if (lane == 0) prefetch_tmap(&tmX);
    int slot = 0;
    uint32_t ring = 0;
    bool ok = true;
    for (int item = pair; item < items && ok; item += npairs) {
      int ta, tb;
      bdg2::split_tiles(p, item / p.nblk, ta, tb);
      const int fcol = (item % p.nblk) * BLK + int(rank) * HALF;
      for (int chunk = ta * 4; chunk < tb * 4; ++chunk) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(CEMPTY + slot), ring ^ 1u, DERR_GEMM_WAIT));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(CFULL + slot), SLOT_BYTES);
          tma_load_2d(sCode + slot * SLOT_BYTES, &tmX, bar(CFULL + slot), fcol, chunk * CH);
        }
#pragma unroll
        for (int r = lane; r < CH; r += 32) {
          const int token = chunk * CH + r;  // behind the last one: exponent 0, which reads as 0 like the codes
          const bool in = token < p.T;
          copy_word(sExp + slot * EXP_BYTES + r * 4, pp.exps + int64_t(in ? token : 0) * pp.ng + fcol / q8::GROUP, in);
        }
        copies_arrive(bar(CFULL + slot));
        if (++slot == SLOTS) { slot = 0; ring ^= 1u; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 100000ull) {
      }
    }
  } else if (warp >= 6) {
    // ---------------- codes -> bf16 (both CTAs): thread = (token of the chunk, group of 32 columns)
    const int ct = threadIdx.x - 192;
    const int row = ct & 63, group = ct >> 6;
    const uint32_t xfull_leader = tc2::map_to_rank(bar(XFULL), 0);
    int u = 0, slot = 0;
    uint32_t ring = 0, cring = 0;
    bool ok = true;
    for (int item = pair; item < items && ok; item += npairs) {
      int ta, tb;
      bdg2::split_tiles(p, item / p.nblk, ta, tb);
      for (int tile = ta; tile < tb && ok; ++tile) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ok = ok && mbar_wait(bar(CFULL + slot), cring, DERR_GEMM_WAIT) &&
               mbar_wait(bar(XEMPTY + u), ring ^ 1u, DERR_GEMM_WAIT);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            uint32_t eb;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(eb) : "r"(sExp + slot * EXP_BYTES + row * 4 + group) : "memory");
            const float sc = q8::exponent_value(static_cast<uint8_t>(eb));
            const uint32_t src = sCode + slot * SLOT_BYTES + row * 128;
            const uint32_t dst = sX + u * TILE_BYTES + (group >> 1) * (CH * 128) + row * 128;
            const int d0 = (group & 1) * 4;  // this group's first 16-byte unit in the row of 64 columns
            uint32_t w[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                           : "r"(src + (((group * 2 + i) ^ (row & 7)) << 4))
                           : "memory");
            auto put = [&](auto far) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint4 o = expand8<decltype(far)::value>(w[i][2 * h], w[i][2 * h + 1], sc);
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                   dst + (((d0 + 2 * i + h) ^ (row & 7)) << 4)),
                               "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w)
                               : "memory");
                }
            };
            if (sc >= 0x1p100f) put(std::true_type());
            else put(std::false_type());
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              arrive_pair(xfull_leader + 8 * u);
              mbar_arrive(bar(CEMPTY + slot));
            }
            if (++u == XUNITS) { u = 0; ring ^= 1u; }
            if (++slot == SLOTS) { slot = 0; cring ^= 1u; }
          }
        }
      }
    }
  } else {
    // ---------------- epilogues (both CTAs): rows quarter*32 .. +31 of this CTA's 128
    const int quarter = warp & 3;
    const uint32_t my_boxes = sEpi + (warp - 2) * 2 * EPI_BOX;
    const uint32_t oempty_leader = tc2::map_to_rank(bar(OEMPTY), 0);
    const uint32_t aempty_leader = tc2::map_to_rank(bar(AEMPTY), 0);
    const uint32_t tl = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    int buf = 0;
    int local = 0, otiles = 0;
    bool ok = true;
    for (int item = pair; item < items && ok; item += npairs, ++local) {
      const int j = item % p.nblk, s = item / p.nblk;
      int ta, tb;
      bdg2::split_tiles(p, s, ta, tb);
      if (p.want_o) {
        for (int tile = ta; tile < tb; ++tile, ++otiles) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(OFULL), otiles & 1, DERR_GEMM_WAIT));
          if (!ok) break;
          tc_fence_after();
          const int row0 = tile * BLK + int(rank) * HALF + quarter * 32;  // token rows of this warp
          const bool rows_in = row0 < p.T;
          // half a row at a time into registers (bf16 pairs) and out through the
          // boxes; the accumulator is released once the second half is read
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t w[BLK / 4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float v[32];
              tmem_ld_32cols(tl + 128 * h + 32 * g, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[16 * g + i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            }
            if (h == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_pair(oempty_leader);
            }
            if (!rows_in) continue;
#pragma unroll
            for (int c0 = 0; c0 < 2; ++c0) {
              if (lane == 0) bulk_wait_read<1>();
              __syncwarp();
              const uint32_t box = my_boxes + buf * EPI_BOX;
              const uint32_t rowp = box + lane * 128;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(rowp + ((k ^ (lane & 7)) << 4)),
                             "r"(w[32 * c0 + 4 * k]), "r"(w[32 * c0 + 4 * k + 1]), "r"(w[32 * c0 + 4 * k + 2]),
                             "r"(w[32 * c0 + 4 * k + 3])
                             : "memory");
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmO, box, j * BLK + 128 * h + 64 * c0, row0);
                bulk_commit();
              }
              buf ^= 1;
            }
          }
        }
        if (!ok) break;
      }
      // dG partial of this item: this CTA's 128 feature rows, fp32
      ok = __all_sync(0xffffffffu, mbar_wait(bar(AFULL), local & 1, DERR_GEMM_WAIT));
      if (!ok) break;
      tc_fence_after();
      const int prow = (s * p.nblk + j) * BLK + int(rank) * HALF + quarter * 32;
#pragma unroll 1
      for (int c0 = 0; c0 < BLK; c0 += 32) {
        float v[32];
        tmem_ld_32cols(tl + BLK + c0, v);
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        const uint32_t box = my_boxes + buf * EPI_BOX;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + ((k ^ (lane & 7)) << 4)),
                       "f"(v[4 * k]), "f"(v[4 * k + 1]), "f"(v[4 * k + 2]), "f"(v[4 * k + 3])
                       : "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmPart, box, c0, prow);
          bulk_commit();
        }
        buf ^= 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_pair(aempty_leader);
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc2::cluster_sync();  // every MMA into either CTA's TMEM and every remote arrive is done
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
  tc2::cluster_sync();
}

}  // namespace bdg8
}  // namespace poetx
