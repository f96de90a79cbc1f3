// Row kernels of the 8-bit path: rows quantised to int8 codes with one fp32
// scale per row, the root-mean-square norm that ends in such rows and its
// backward, and activation checkpoints (int8 codes, a shared power of two per
// 32 columns).  All of them move bytes: each reads its inputs and writes its
// outputs once, so HBM bandwidth is their floor.
//
// Quantised rows.  For a row u (fp32): scale = max|u| / 127 (fp32 division),
// code = u / scale rounded half to even.  The quotient is never formed: it is
// bracketed by u times two bounds of 1 / scale, and where the brackets round
// apart, the remainder r = u - q * scale of q = round(u * (1 / scale)) decides;
// it is exact (a multiple of ulp(scale) no larger than scale in magnitude, one
// FMA).  So the codes are those of the real quotient, whatever the order of
// any reduction.
// A row that holds an infinity or a NaN gets codes 0 and scale NaN, so it
// cannot pass for an ordinary row; a row of zeros gets codes 0 and scale 0.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>

#include "perm.cuh"

namespace poetx {
namespace q8 {

// Most threads of a row's block: two blocks of 72 registers fit a SM (rows to
// int8, and the norm up to K = 2).  The norm's backward holds more (98 at K = 2,
// 128 and spills at K = 4); it and the norm take rows of more than 7168 elements
// as K = 4, one block a SM: 16384 x 8192 bf16 174 us for the norm and 221 for its
// backward with dres (144 and 164 at the copy rate), where rows of 4096 are
// within a sixth of it.
constexpr int kRowThreads = 448;

// ---------------------------------------------------------------- loads and stores
// Eight elements of a row of d as loaded: consecutive ones from c (V = 8,
// whole 16-byte vectors), or c, c + nt, ... (V = 1, any row).  Outside the
// row: zeros.  FULL: the block's threads cover the row exactly, nothing to
// check.  V = 2: rows of a d that is no multiple of eight, taken by the array's
// own 16-byte units: a row that starts `phase` elements behind one has c =
// -phase, 8 - phase, ..., and the units it shares with its neighbours are
// loaded and stored one element at a time.  The phase, (row * d) % 8, is the same
// for all rows of a block, since the grid is a multiple of eight.
template <typename T, int V>
struct Raw8 {
  T v[8];
};
template <>
struct Raw8<__nv_bfloat16, 8> {
  uint4 v;
};
template <>
struct Raw8<float, 8> {
  float4 v[2];
};
template <>
struct Raw8<__nv_bfloat16, 2> : Raw8<__nv_bfloat16, 8> {
  __device__ __forceinline__ void from(const __nv_bfloat16* e) {
    auto two = [&](int i) {
      return static_cast<uint32_t>(__bfloat16_as_ushort(e[i])) | static_cast<uint32_t>(__bfloat16_as_ushort(e[i + 1])) << 16;
    };
    v = make_uint4(two(0), two(2), two(4), two(6));
  }
};
template <>
struct Raw8<float, 2> : Raw8<float, 8> {
  __device__ __forceinline__ void from(const float* e) {
    v[0] = make_float4(e[0], e[1], e[2], e[3]);
    v[1] = make_float4(e[4], e[5], e[6], e[7]);
  }
};

// Is the unit at c all inside the row?
__device__ __forceinline__ bool inside8(int c, int d) { return c >= 0 && c + 8 <= d; }

template <typename T, int V, bool FULL>
__device__ __forceinline__ void fetch8(Raw8<T, V>& r, const T* p, int c, int nt, int d) {
  if constexpr (V == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = c + e * nt < d ? p[c + e * nt] : from_f32<T>(0.f);
  } else if constexpr (V == 2) {
    if (inside8(c, d)) {
      fetch8<T, 8, true>(r, p, c, nt, d);
    } else {
      T v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e >= 0 && c + e < d ? p[c + e] : from_f32<T>(0.f);
      r.from(v);
    }
  } else if constexpr (std::is_same<T, float>::value) {
    const bool in = FULL || c < d;
    r.v[0] = in ? reinterpret_cast<const float4*>(p + c)[0] : make_float4(0.f, 0.f, 0.f, 0.f);
    r.v[1] = in ? reinterpret_cast<const float4*>(p + c)[1] : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    r.v = FULL || c < d ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0u, 0u, 0u, 0u);
  }
}
template <typename T, int V>
__device__ __forceinline__ void unpack8(const Raw8<T, V>& r, float* f) {
  if constexpr (V == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = to_f32<T>(r.v[e]);
  } else if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = r.v[i].x;
      f[4 * i + 1] = r.v[i].y;
      f[4 * i + 2] = r.v[i].z;
      f[4 * i + 3] = r.v[i].w;
    }
  } else {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
// f rounded to T, as loaded.
template <typename T, int V>
__device__ __forceinline__ void pack8(Raw8<T, V>& r, const float* f) {
  if constexpr (V == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = from_f32<T>(f[e]);
  } else if constexpr (std::is_same<T, float>::value) {
    r.v[0] = make_float4(f[0], f[1], f[2], f[3]);
    r.v[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&r.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}
template <typename T, int V, bool FULL>
__device__ __forceinline__ void put8(T* p, int c, int nt, int d, const Raw8<T, V>& r) {
  if constexpr (V == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e * nt < d) p[c + e * nt] = r.v[e];
  } else if (V == 2 && !inside8(c, d)) {
    float f[8];
    unpack8<T, V>(r, f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= 0 && c + e < d) p[c + e] = from_f32<T>(f[e]);
  } else if (FULL || c < d) {
    if constexpr (std::is_same<T, float>::value) {
      reinterpret_cast<float4*>(p + c)[0] = r.v[0];
      reinterpret_cast<float4*>(p + c)[1] = r.v[1];
    } else {
      *reinterpret_cast<uint4*>(p + c) = r.v;
    }
  }
}
template <typename T, int V, bool FULL>
__device__ __forceinline__ void load8(const T* p, int c, int nt, int d, float* f) {
  Raw8<T, V> r;
  fetch8<T, V, FULL>(r, p, c, nt, d);
  unpack8<T, V>(r, f);
}
template <typename T, int V, bool FULL>
__device__ __forceinline__ void store8(T* p, int c, int nt, int d, const float* f) {
  Raw8<T, V> r;
  pack8<T, V>(r, f);
  put8<T, V, FULL>(p, c, nt, d, r);
}

// V = 2: `n` floats of a row's gain (zeros outside it) as the units see them, in
// shared memory.
__device__ __forceinline__ void stage_gain(float* sm, const float* gain, int phase, int n, int d) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) sm[i] = i >= phase && i - phase < d ? gain[i - phase] : 0.f;
}
template <int V, bool FULL>
__device__ __forceinline__ void load_gain(const float* gain, const float* sm, int phase, int c, int nt, int d, float* g) {
  if constexpr (V == 2) load8<float, 8, true>(sm, c + phase, nt, d, g);
  else load8<float, V, FULL>(gain, c, nt, d, g);
}

// ---------------------------------------------------------------- two values an instruction
// Packed fp32 arithmetic (sm_100): each half rounded like the plain operation.
// It halves the norm's sums (8192 x 14336 backward: 262 -> 217 us); the gain and
// the quotients of the codes are faster plain (rows to int8, 8192 x 14336: 88 us
// packed, 78 plain), since pairs of registers cost the blocks a SM holds more
// than the instructions do.
__device__ __forceinline__ void mul2(float* a, const float* b) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a[0]), "+f"(a[1])
      : "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void add2(float* a, const float* b) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a[0]), "+f"(a[1])
      : "f"(b[0]), "f"(b[1]));
}
// c += a * b
__device__ __forceinline__ void fma2(float* c, const float* a, const float* b) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(c[0]), "+f"(c[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
// The larger of t and |a|, |b|; a NaN stays.
__device__ __forceinline__ float abs_max2(float t, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(t), "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- quantiser
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds half to even, low byte = the integer

struct RowScale {
  float s, inv, lo, hi;  // inv ~ 1 / s, lo < 1 / s < hi
  int kind;  // 0: zero row, 1: ordinary, 2: scale too small for 1 / s, 3: not finite
};

__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.s = amax / 127.f;
  r.inv = __fdividef(1.f, r.s);       // good to a few units in the last place (2^-24 each)
  r.lo = r.inv * (1.f - 0x1p-20f);
  r.hi = r.inv * (1.f + 0x1p-20f);
  r.kind = !(amax <= 3.402823466e38f) ? 3 : !(r.s > 0.f) ? 0 : r.s < 1e-36f ? 2 : 1;
  if (r.kind == 3) r.s = __uint_as_float(0x7fffffffu);
  return r;
}

// One code, slowly: rows whose scale is too small to invert (its own quotient
// in 64 bits), zero and non-finite rows.
__device__ __forceinline__ uint32_t quantise_far(float u, const RowScale& r) {
  if (r.kind != 2) return 0u;
  const double q = rint(static_cast<double>(u) / static_cast<double>(r.s));
  return static_cast<uint32_t>(static_cast<int>(fmin(fmax(q, -127.0), 127.0))) & 0xffu;
}

// One code at a border: the nearest, the even one on a tie.
__device__ __forceinline__ uint32_t quantise_border(float u, const RowScale& r) {
  const float m = fmaf(u, r.inv, kMagic), q = m - kMagic;
  const float rem = fmaf(-q, r.s, u), twice = 2.f * fabsf(rem);
  int c = static_cast<int>(q);
  if (twice > r.s || (twice == r.s && (c & 1))) c += rem > 0.f ? 1 : -1;
  return static_cast<uint32_t>(c) & 0xffu;
}

// The codes of eight values (placed as in load8).  The quotient lies between
// u * lo and u * hi; where both round to the same integer that is the code
// (two FMAs a value, one branch for all eight).
// V = 2: where the codes' rows lie like the values' (like), a unit is eight
// bytes on a boundary; rows that start on a boundary of their own take theirs
// from two neighbouring lanes (WARP: all lanes call).
template <int V, bool FULL, bool WARP>
__device__ __forceinline__ void store_codes(int8_t* p, int c, int nt, int d, const float* u, const RowScale& r,
                                            bool like, int phase) {
  uint32_t q[8];
  if (r.kind == 1) {
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = __float_as_uint(fmaf(u[i], r.lo, kMagic));
      differ |= q[i] ^ __float_as_uint(fmaf(u[i], r.hi, kMagic));
    }
    if (differ) {
      // (not rare: 127 / 2 is a border, so every u of half the row's maximum lies on one)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (q[i] != __float_as_uint(fmaf(u[i], r.hi, kMagic))) q[i] = quantise_border(u[i], r);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quantise_far(u[i], r);
  }
  if constexpr (V == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * nt < d) p[c + i * nt] = static_cast<int8_t>(q[i]);
  } else {
    uint2 w;
    w.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
    if constexpr (V == 2) {
      auto bytes = [&](uint64_t v, int at, int n) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n && at + e >= 0 && at + e < d) p[at + e] = static_cast<int8_t>(v >> 8 * e);
      };
      const uint64_t own = static_cast<uint64_t>(w.y) << 32 | w.x;
      if (like) {
        if (inside8(c, d)) *reinterpret_cast<uint2*>(p + c) = w;
        else bytes(own, c, 8);
      } else if (WARP) {
        const int lane = threadIdx.x & 31, at = c + phase;  // at: a multiple of eight
        const uint64_t next = __shfl_down_sync(0xffffffffu, own, 1);
        const uint64_t v = phase ? own >> 8 * phase | next << (64 - 8 * phase) : own;
        if (lane < 31 && at + 8 <= d) *reinterpret_cast<uint64_t*>(p + at) = v;
        else bytes(v, at, lane < 31 ? 8 : 8 - phase);
        if (lane == 0) bytes(own, c, phase);
      } else {
        bytes(own, c, 8);
      }
    } else if (FULL || c < d) {
      *reinterpret_cast<uint2*>(p + c) = w;
    }
  }
}

// max that keeps a NaN
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum of `a` (SUM) and maximum of `b` >= 0 (MAX, a NaN stays one) over a block
// of at most 16 warps; red holds 2 * 16 floats, zero beyond the block's warps,
// and is free again after the next call's barrier (callers alternate two).
struct alignas(16) BlockSums {
  float sum[16], top[16];
};
__device__ __forceinline__ void clear_sums(BlockSums* r) {
  if (threadIdx.x < 32) {
    for (int b = 0; b < 2; ++b) (threadIdx.x < 16 ? r[b].sum : r[b].top)[threadIdx.x & 15] = 0.f;
  }
  __syncthreads();
}
template <bool SUM, bool MAX>
__device__ __forceinline__ void block_reduce(float& a, float& b, BlockSums* red) {
  if (SUM) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  }
  // bits of non-negative floats are ordered as the floats, NaN above infinity
  if (MAX) b = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b) & 0x7fffffffu));
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    if (SUM) red->sum[w] = a;
    if (MAX) red->top[w] = b;
  }
  __syncthreads();
  const int n4 = (blockDim.x + 127) >> 7;  // groups of four warps
  float s = 0.f, t = 0.f;
  for (int i = 0; i < n4; ++i) {
    if (SUM) {
      const float4 v = reinterpret_cast<const float4*>(red->sum)[i];
      s += (v.x + v.y) + (v.z + v.w);
    }
    if (MAX) {
      const float4 v = reinterpret_cast<const float4*>(red->top)[i];
      t = nan_max(t, nan_max(nan_max(v.x, v.y), nan_max(v.z, v.w)));
    }
  }
  a = s;
  b = t;
}

// ---------------------------------------------------------------- rows to int8, with or without the norm
struct RowsParams {
  const void* x;          // [T][d]
  const void* residual;   // [T][d] or NULL (norm only)
  const float* gain;      // [d]: gamma (norm), column scale or NULL (plain)
  void* h;                // [T][d] or NULL: x + residual
  void* y;                // [T][d] or NULL: the normalised rows
  int8_t* codes;          // [T][ldc] or NULL
  float* scale;           // [T]
  float* rstd;            // [T] or NULL
  int64_t T;
  int64_t ldc;
  int d;
  float eps;
};

// One block per row, rows strided over the grid.  NORM: h = x + residual
// rounded to T, rstd = 1 / sqrt(mean h^2 + eps), u = h * gamma; else u = x or
// x * gain.  The codes of u and of rstd * u are the same (the factor cancels
// in u / max|u|), so one reduction gives both the sum of squares and the
// maximum, and the row is read once: a thread holds K times eight elements in
// registers, and loads its next row's before it works on this one.  K = 0:
// rows too wide for registers are read a second time (h as written; each
// thread rereads only what it wrote itself).  Bound by HBM for the norm (16384 x
// 4096 bf16 with a residual: 82 us, 72 at the copy rate; fp32 145 of 133), by the
// way through a row, loads - reduction - codes, for the rows alone (43 us of 31;
// fp32 55 of 51) and for the widest ones (4096 x 28672 bf16, read twice: 100 us of
// 54, the norm 230 of 126).
template <typename T, bool NORM, int V, int K, bool FULL>
__global__ void __launch_bounds__(NORM && K == 2 && V == 8 ? 512 : kRowThreads, NORM && (K == 4 || V == 1) ? 1 : 2)
    rows_kernel(const RowsParams p) {
  extern __shared__ __align__(16) float gain_sm[];  // V = 2
  __shared__ BlockSums red[2];
  const T* xs = static_cast<const T*>(p.x);
  const T* rs = static_cast<const T*>(p.residual);
  T* hs = static_cast<T*>(p.h);
  T* ys = static_cast<T*>(p.y);
  constexpr int KR = K > 0 ? K : 1;
  const int nt = blockDim.x, step = nt * 8, d = p.d;
  const int phase = V == 2 ? static_cast<int>(static_cast<int64_t>(blockIdx.x) * d & 7) : 0;
  const int first = V == 2 ? threadIdx.x * 8 - phase : threadIdx.x * V;
  const bool gain = NORM || p.gain, like = p.ldc == d;
  if (V == 2 && gain) stage_gain(gain_sm, p.gain, phase, K > 0 ? K * step : (d + 14) / 8 * 8, d);
  clear_sums(red);
  Raw8<T, V> nx[KR], nr[NORM ? KR : 1];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < KR; ++k) fetch8<T, V, FULL>(nx[k], xs + row * d, first + k * step, nt, d);
    if (NORM && rs) {
#pragma unroll
      for (int k = 0; k < KR; ++k) fetch8<T, V, FULL>(nr[NORM ? k : 0], rs + row * d, first + k * step, nt, d);
    }
  };
  if (K > 0 && blockIdx.x < p.T) fetch(blockIdx.x);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, buf ^= 1) {
    const int64_t base = row * d;
    float u[KR][8];
    float sum = 0.f, top = 0.f, sums[2] = {0.f, 0.f};
    // h (u so far) from x and the residual
    auto summed = [&](int c, float* v, const Raw8<T, V>& r) {
      if constexpr (NORM) {
        if (rs) {
          float f[8];
          unpack8<T, V>(r, f);
#pragma unroll
          for (int e = 0; e < 8; e += 2) add2(v + e, f + e);
          Raw8<T, V> h;
          pack8<T, V>(h, v);
          if (hs) put8<T, V, FULL>(hs + base, c, nt, d, h);
          unpack8<T, V>(h, v);
        } else if (hs) {
          store8<T, V, FULL>(hs + base, c, nt, d, v);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) fma2(sums, v + e, v + e);
      }
    };
    auto gained = [&](int c, float* v) {
      if (gain) {
        float g[8];
        load_gain<V, FULL>(p.gain, gain_sm, phase, c, nt, d, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) top = abs_max2(top, v[e], v[e + 1]);
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        unpack8<T, V>(nx[k], u[k]);
        summed(first + k * step, u[k], nr[NORM ? k : 0]);
      }
      if (row + gridDim.x < p.T) fetch(row + gridDim.x);
#pragma unroll
      for (int k = 0; k < K; ++k) gained(first + k * step, u[k]);
    } else {
      for (int c = first; c < d; c += step) {
        load8<T, V, FULL>(xs + base, c, nt, d, u[0]);
        if (NORM && rs) fetch8<T, V, FULL>(nr[0], rs + base, c, nt, d);
        summed(c, u[0], nr[0]);
        gained(c, u[0]);
      }
    }
    sum = sums[0] + sums[1];
    block_reduce<NORM, true>(sum, top, &red[buf]);
    const RowScale sc = row_scale(top);
    float rstd = 1.f;
    if constexpr (NORM) rstd = rsqrtf(sum / static_cast<float>(d) + p.eps);
    if (threadIdx.x == 0) {
      if (p.codes) p.scale[row] = sc.s * rstd;
      if (NORM && p.rstd) p.rstd[row] = rstd;
    }
    auto finish = [&](int c, float* v) {
      if (p.codes) store_codes<V, FULL, (K > 0)>(p.codes + row * p.ldc, c, nt, d, v, sc, like, phase);
      if (NORM && ys) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= rstd;
        store8<T, V, FULL>(ys + base, c, nt, d, v);
      }
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) finish(first + k * step, u[k]);
    } else {
      const T* again = NORM && hs ? hs + base : xs + base;
      for (int c = first; c < d; c += step) {
        load8<T, V, FULL>(again, c, nt, d, u[0]);
        gained(c, u[0]);
        finish(c, u[0]);
      }
    }
  }
}

// ---------------------------------------------------------------- norm backward
struct NormGradParams {
  const void* dy;
  const void* h;
  const float* gamma;
  const float* rstd;
  const void* dres;   // gradient that reaches h past the norm, or NULL
  void* dx;
  float* part;        // [gridDim.x][d] partial sums of dgamma
  int64_t T;
  int d;
};

// With p = dy * gamma: dx = rstd (p - h rstd^2 mean(p h)) + dres, and
// dgamma = sum over rows of dy h rstd.  A block walks the rows blockIdx.x,
// blockIdx.x + gridDim.x, ...; a thread keeps its columns' share of dgamma in
// registers over all of them (K > 0) or in its own words of shared memory
// (K = 0, any width), so the sum's order is fixed by the grid alone.  Bound by
// HBM: 16384 x 4096 bf16 with dres 83 us (94 in a long run), 82 at the copy rate;
// fp32 156 of 164.  Rows of more than 7168 elements do not fit two blocks a SM, and
// fp32 ones go through shared memory: 8192 x 8192 118 us of 82, fp32 221 of 164;
// 8192 x 14336 225 us of 144, fp32 430 of 287.
template <typename T, int V, int K, bool FULL>
__global__ void __launch_bounds__(kRowThreads) norm_grad_kernel(const NormGradParams p) {
  extern __shared__ __align__(16) float sm[];  // V = 2: gamma; K = 0: the share of dgamma behind it
  __shared__ BlockSums red[2];
  const T* dys = static_cast<const T*>(p.dy);
  const T* hs = static_cast<const T*>(p.h);
  const T* rs = static_cast<const T*>(p.dres);
  T* dxs = static_cast<T*>(p.dx);
  constexpr int KR = K > 0 ? K : 1;
  const int nt = blockDim.x, step = nt * 8, d = p.d;
  const int phase = V == 2 ? static_cast<int>(static_cast<int64_t>(blockIdx.x) * d & 7) : 0;
  const int first = V == 2 ? threadIdx.x * 8 - phase : threadIdx.x * V;
  const int units = K > 0 ? K * step : (d + 14) / 8 * 8;
  float* const acc_sm = V == 2 ? sm + units + phase : sm;
  constexpr int VA = V == 2 ? 8 : V;  // the share of dgamma: whole units
  float acc[KR][8];
#pragma unroll
  for (int k = 0; k < KR; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
  if constexpr (K == 0)
    for (int c = first; c < d; c += step) store8<float, VA, FULL>(acc_sm, c, nt, d, acc[0]);
  if (V == 2) stage_gain(sm, p.gamma, phase, units, d);
  clear_sums(red);
  Raw8<T, V> ny[KR], nh[KR], nr[KR];
  float next_rstd = 0.f;
  auto fetch = [&](int64_t row) {
    next_rstd = p.rstd[row];
#pragma unroll
    for (int k = 0; k < KR; ++k) {
      fetch8<T, V, FULL>(ny[k], dys + row * d, first + k * step, nt, d);
      fetch8<T, V, FULL>(nh[k], hs + row * d, first + k * step, nt, d);
    }
  };
  if (K > 0 && blockIdx.x < p.T) fetch(blockIdx.x);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, buf ^= 1) {
    const int64_t base = row * d;
    float dot = 0.f, none = 0.f, dot2[2] = {0.f, 0.f};
    float dy[KR][8], h[KR][8];
    const float rstd = K > 0 ? next_rstd : p.rstd[row];
    const float rstd2[2] = {rstd, rstd};
    auto dots = [&](int c, float* a, float* b, float* w) {
      float g[8];
      load_gain<V, FULL>(p.gamma, sm, phase, c, nt, d, g);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        mul2(b + e, rstd2);
        fma2(w + e, a + e, b + e);
        mul2(a + e, g + e);
        fma2(dot2, a + e, b + e);
      }
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        unpack8<T, V>(ny[k], dy[k]);
        unpack8<T, V>(nh[k], h[k]);
        if (rs) fetch8<T, V, FULL>(nr[k], rs + base, first + k * step, nt, d);
      }
      if (row + gridDim.x < p.T) fetch(row + gridDim.x);
#pragma unroll
      for (int k = 0; k < K; ++k) dots(first + k * step, dy[k], h[k], acc[k]);
    } else {
      for (int c = first; c < d; c += step) {
        load8<T, V, FULL>(dys + base, c, nt, d, dy[0]);
        load8<T, V, FULL>(hs + base, c, nt, d, h[0]);
        load8<float, VA, FULL>(acc_sm, c, nt, d, acc[0]);
        dots(c, dy[0], h[0], acc[0]);
        store8<float, VA, FULL>(acc_sm, c, nt, d, acc[0]);
      }
    }
    dot = dot2[0] + dot2[1];
    block_reduce<true, false>(dot, none, &red[buf]);
    const float mean = dot / static_cast<float>(d);
    const float less[2] = {-mean, -mean};
    auto finish = [&](int c, const float* a, const float* b, const Raw8<T, V>& res) {
      float o[8], r[8];
      if (rs) unpack8<T, V>(res, r);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float v[2] = {a[e], a[e + 1]};
        fma2(v, b + e, less);
        o[e] = rs ? r[e] : 0.f;
        o[e + 1] = rs ? r[e + 1] : 0.f;
        fma2(o + e, v, rstd2);
      }
      store8<T, V, FULL>(dxs + base, c, nt, d, o);
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) finish(first + k * step, dy[k], h[k], nr[k]);
    } else {
      for (int c = first; c < d; c += step) {
        float g[8];
        load8<T, V, FULL>(dys + base, c, nt, d, dy[0]);
        load8<T, V, FULL>(hs + base, c, nt, d, h[0]);
        load_gain<V, FULL>(p.gamma, sm, phase, c, nt, d, g);
        if (rs) fetch8<T, V, FULL>(nr[0], rs + base, c, nt, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dy[0][e] *= g[e];
          h[0][e] *= rstd;
        }
        finish(c, dy[0], h[0], nr[0]);
      }
    }
  }
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * d;  // (V = 2: a row like the others, blockIdx.x its number)
  if constexpr (K > 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) store8<float, V, FULL>(out, first + k * step, nt, d, acc[k]);
  } else {
    for (int c = first; c < d; c += step) {
      load8<float, VA, FULL>(acc_sm, c, nt, d, acc[0]);
      store8<float, V, FULL>(out, c, nt, d, acc[0]);
    }
  }
}

// out[c] (+)= sum of part[g][c] over g < n, in a fixed order: 32 columns per
// block, 32 slices of g summed apart and then together (with eight slices the
// norm's backward took 22 us at 3863 x 75, whose 2368 partial sums are three
// blocks' work here).
constexpr int SLICES = 32;
__global__ void __launch_bounds__(32 * SLICES) sum_partials_kernel(const float* __restrict__ part, int n, int d,
                                                           float* __restrict__ out, int accumulate) {
  __shared__ float sm[SLICES][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int g = slice; g < n; g += SLICES) s += part[static_cast<int64_t>(g) * d + c];
  sm[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < d) {
#pragma unroll
    for (int k = 1; k < SLICES; ++k) s += sm[k][lane];
    out[c] = accumulate ? out[c] + s : s;
  }
}

// out[i] (+)= sum of part[s][i] over s < splits in that order, n values each
// (any n: four at a time where the slices stay 16-byte aligned).
__global__ void add_splits_kernel(const float* __restrict__ part, int splits, int64_t n, float* __restrict__ out,
                                  int accumulate) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  if (n % 4 == 0) {
    const float4* p4 = reinterpret_cast<const float4*>(part);
    float4* o4 = reinterpret_cast<float4*>(out);
    for (int64_t i = first; i < n / 4; i += step) {
      float4 a = p4[i];
#pragma unroll 8
      for (int s = 1; s < splits; ++s) {
        const float4 v = p4[s * (n / 4) + i];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      if (accumulate) {
        const float4 o = o4[i];
        a.x += o.x;
        a.y += o.y;
        a.z += o.z;
        a.w += o.w;
      }
      o4[i] = a;
    }
  } else {
    for (int64_t i = first; i < n; i += step) {
      float a = part[i];
      for (int s = 1; s < splits; ++s) a += part[s * n + i];
      out[i] = accumulate ? out[i] + a : a;
    }
  }
}

// ---------------------------------------------------------------- activation checkpoints
// Groups of 32 columns of a row share the exponent e, the smallest with
// max|v| <= 127 * 2^e (at least -126, at most 121, where larger values are cut
// to 127 * 2^121), stored biased by 127; code = v * 2^-e rounded half to even.  Scaling by a power of two is exact, and a code has
// at most 7 bits, so code * 2^e is exact in bf16: what the backward multiplies
// is the checkpoint itself, with no second rounding.  A group that holds an
// infinity or a NaN gets exponent 255 and codes 0, and reads back as NaN.
constexpr int GROUP = 32;
constexpr uint32_t kMaxExp = 248;      // 2^121: one more and 64 * 2^122 would not be finite
constexpr uint32_t kMaxKept = 0x7f7e0000u;  // 127 * 2^121

__device__ __forceinline__ uint32_t group_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const uint32_t E = bits >> 23;
  if (E == 255u) return 255u;
  // amax = 1.M * 2^(E-127); 64 * 1.M > 127 exactly when M > 63/64
  const int eb = static_cast<int>(E) - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return eb < 1 ? 1u : eb > static_cast<int>(kMaxExp) ? kMaxExp : static_cast<uint32_t>(eb);
}
__device__ __forceinline__ float exponent_inverse(uint32_t eb) {  // 2^-e, 0 for 255
  return eb == 255u ? 0.f : __uint_as_float((254u - eb) << 23);
}
__device__ __forceinline__ float exponent_value(uint32_t eb) {    // 2^e, NaN for 255
  return __uint_as_float(eb == 255u ? 0x7fffffffu : eb << 23);
}
__device__ __forceinline__ uint32_t checkpoint_code(float v, float inv) {
  return inv == 0.f ? 0u : __float_as_uint(fmaf(v, inv, kMagic)) & 0xffu;
}
__device__ __forceinline__ float kept(float v) { return copysignf(fminf(fabsf(v), __uint_as_float(kMaxKept)), v); }

// N elements as fp32 in 16-byte units (4 fp32 or 8 bf16 each).
template <typename T, int N>
__device__ __forceinline__ void load_units(const T* p, float* f) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 a = reinterpret_cast<const float4*>(p)[i];
      f[4 * i] = a.x;
      f[4 * i + 1] = a.y;
      f[4 * i + 2] = a.z;
      f[4 * i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      Raw8<T, 8> r;
      fetch8<T, 8, true>(r, p + 8 * i, 0, 0, 0);
      unpack8<T, 8>(r, f + 8 * i);
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_units(T* p, const float* f) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) store8<T, 8, true>(p + 8 * i, 0, 0, 0, f + 8 * i);
  }
}
// N int8 codes from or to one word of N bytes (N = 4, 8 or 16).
template <int N>
__device__ __forceinline__ void load_codes(const int8_t* p, uint32_t* w) {
  if constexpr (N == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
  else if constexpr (N == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  else *w = *reinterpret_cast<const uint32_t*>(p);
}
template <int N>
__device__ __forceinline__ void write_codes(int8_t* p, const uint32_t* w) {
  if constexpr (N == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
  else if constexpr (N == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
  else *reinterpret_cast<uint32_t*>(p) = *w;
}
__device__ __forceinline__ float code_value(const uint32_t* w, int i) {
  return static_cast<float>(static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3))));
}

// The kernels below give a warp 32 * N columns of a row, N of them consecutive
// to a lane (16 or 8 bf16, 8 or 4 fp32), so that a warp's accesses are whole
// lines: at 16384 x 4096 bf16 saving takes 33 us and reading back 36 us (31 us
// is the copy rate), fp32 53 and 66 (51).  N = 1,
// for rows that are no whole vectors: a lane takes one column of each of eight
// groups.  Chunks of rows are walked without a division by the grid's shape:
// blockIdx.x and the warp give the chunk, blockIdx.y strides over the rows.
constexpr int kOddGroups = 8;
template <int N>
constexpr int chunk_cols = N == 1 ? GROUP * kOddGroups : 32 * N;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <typename T, int N>
__global__ void __launch_bounds__(128) checkpoint_save_kernel(const T* __restrict__ x, int64_t rows, int d,
                                                              int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const int lane = threadIdx.x & 31;
  const int ng = (d + GROUP - 1) / GROUP;
  const int c0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * chunk_cols<N>;
  if (c0 >= d) return;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    if constexpr (N == 1) {
      const int64_t at = row * d;
      float v[kOddGroups];
#pragma unroll
      for (int g = 0; g < kOddGroups; ++g) {
        const int c = c0 + g * GROUP + lane;
        v[g] = c < d ? to_f32<T>(x[at + c]) : 0.f;
      }
      uint32_t mine = 0;
#pragma unroll
      for (int g = 0; g < kOddGroups; ++g) {
        const int c = c0 + g * GROUP + lane;
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, magnitude(v[g])));
        const uint32_t eb = group_exponent(top);
        if (lane == g) mine = eb;
        if (c < d) codes[at + c] = static_cast<int8_t>(checkpoint_code(kept(v[g]), exponent_inverse(eb)));
      }
      if (lane < kOddGroups && c0 / GROUP + lane < ng) exps[row * ng + c0 / GROUP + lane] = static_cast<uint8_t>(mine);
    } else {
      constexpr int LG = GROUP / N;  // lanes of a group
      const int c = c0 + lane * N;
      const bool in = c < d;  // (d is a multiple of N)
      float v[N];
      uint32_t top = 0;
      if (in) {
        load_units<T, N>(x + row * d + c, v);
#pragma unroll
        for (int e = 0; e < N; ++e) top = max(top, magnitude(v[e]));
      }
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (in) {
        const uint32_t eb = group_exponent(__uint_as_float(top));
        const float inv = exponent_inverse(eb);
        if (top > kMaxKept && eb != 255u) {
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = kept(v[e]);
        }
        if (lane % LG == 0) exps[row * ng + c / GROUP] = static_cast<uint8_t>(eb);
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = __float_as_uint(fmaf(v[4 * i + e], inv, kMagic));
          w[i] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
          if (eb == 255u) w[i] = 0;
        }
        write_codes<N>(codes + row * d + c, w);
      }
    }
  }
}

// x = code * scale, the scale of a checkpoint's group (exps) or of the row
// (scale), rounded once to T (exact for a checkpoint).
template <typename T, int N>
__global__ void __launch_bounds__(128) expand_kernel(const int8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ exps,
                                                     const float* __restrict__ scale, int64_t rows, int d,
                                                     T* __restrict__ x) {
  const int lane = threadIdx.x & 31;
  const int ng = (d - 1) / GROUP + 1;
  const int c0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * chunk_cols<N>;
  if (c0 >= d) return;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int64_t at = row * d;
    if constexpr (N == 1) {
#pragma unroll
      for (int g = 0; g < kOddGroups; ++g) {
        const int c = c0 + g * GROUP + lane;
        if (c < d) {
          const float s = exps ? exponent_value(exps[row * ng + c / GROUP]) : scale[row];
          x[at + c] = from_f32<T>(static_cast<float>(codes[at + c]) * s);
        }
      }
    } else {
      const int c = c0 + lane * N;
      if (c < d) {
        uint32_t w[N / 4];
        load_codes<N>(codes + at + c, w);
        const float s = exps ? exponent_value(exps[row * ng + c / GROUP]) : scale[row];
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = code_value(w, e) * s;
        store_units<T, N>(x + at + c, v);
      }
    }
  }
}

}  // namespace q8
}  // namespace poetx
