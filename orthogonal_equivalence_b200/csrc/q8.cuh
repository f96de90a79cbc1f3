// Row kernels of the 8-bit path: rows quantised to int8 codes with one fp32
// scale per row, the root-mean-square norm that ends in such rows and its
// backward, and activation checkpoints (int8 codes, a shared power of two per
// 32 columns).  All of them move bytes: each reads its inputs and writes its
// outputs once, so HBM bandwidth is their floor.
//
// Quantised rows.  For a row u (fp32): scale = max|u| / 127 (fp32 division),
// code = u / scale rounded half to even.  The quotient is never formed: with
// q = round(u * (1 / scale)) the remainder r = u - q * scale is exact (it is a
// multiple of ulp(scale) no larger than scale in magnitude, one FMA), and
// 2|r| < scale proves q; the rare other lanes step q by one.  So the codes are
// those of the real quotient, whatever the order of any reduction.
// A row that holds an infinity or a NaN gets codes 0 and scale NaN, so it
// cannot pass for an ordinary row; a row of zeros gets codes 0 and scale 0.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>

#include "perm.cuh"

namespace poetx {
namespace q8 {

// ---------------------------------------------------------------- loads and stores
// V consecutive elements as fp32 (V = 8: 16-byte vectors; V = 1: one element).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  if constexpr (V == 1) {
    f[0] = to_f32<T>(*p);
  } else if constexpr (std::is_same<T, float>::value) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  if constexpr (V == 1) {
    *p = from_f32<T>(f[0]);
  } else if constexpr (std::is_same<T, float>::value) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint4 a;
    uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = a;
  }
}

// f rounded to T and back.
template <typename T>
__device__ __forceinline__ float round_to(float f) {
  return to_f32<T>(from_f32<T>(f));
}

// ---------------------------------------------------------------- quantiser
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds half to even, low byte = the integer

struct RowScale {
  float s, inv;
  int kind;  // 0: zero row, 1: ordinary, 2: scale too small for 1 / s, 3: not finite
};

__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.s = amax / 127.f;
  r.inv = 1.f / r.s;
  r.kind = !(amax <= 3.402823466e38f) ? 3 : !(r.s > 0.f) ? 0 : r.s < 1e-36f ? 2 : 1;
  if (r.kind == 3) r.s = __uint_as_float(0x7fffffffu);
  return r;
}

__device__ __forceinline__ int quantise_far(float u, const RowScale& r) {
  if (r.kind != 2) return 0;
  const double q = rint(static_cast<double>(u) / static_cast<double>(r.s));
  return static_cast<int>(fmin(fmax(q, -127.0), 127.0));
}

__device__ __forceinline__ int quantise(float u, const RowScale& r) {
  const float m = fmaf(u, r.inv, kMagic);
  float q = m - kMagic;
  const float rem = fmaf(-q, r.s, u);
  const float twice = 2.f * fabsf(rem);
  int code = __float_as_int(m) & 0xff;
  if (!(twice < r.s)) {  // a border: the nearest code, the even one on a tie
    const float step = copysignf(1.f, rem);
    const int qi = static_cast<int>(q);
    if (twice > r.s || (qi & 1)) code = (qi + static_cast<int>(step)) & 0xff;
  }
  return code;
}

// V codes of V values.
template <int V>
__device__ __forceinline__ void store_codes(int8_t* p, const float* u, const RowScale& r) {
  int c[V];
  if (r.kind == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = quantise(u[i], r);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = quantise_far(u[i], r);
  }
  if constexpr (V == 1) {
    *p = static_cast<int8_t>(c[0]);
  } else {
    uint2 w;
    w.x = (c[0] & 0xff) | (c[1] & 0xff) << 8 | (c[2] & 0xff) << 16 | (c[3] & 0xff) << 24;
    w.y = (c[4] & 0xff) | (c[5] & 0xff) << 8 | (c[6] & 0xff) << 16 | (c[7] & 0xff) << 24;
    *reinterpret_cast<uint2*>(p) = w;
  }
}

// max that keeps a NaN
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum of `a` and maximum of `b` over the block; red holds 2 * 32 floats and is
// free again after the next call's barrier (callers alternate two of them).
__device__ __forceinline__ void block_sum_max(float& a, float& b, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = nan_max(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  const int nw = blockDim.x >> 5, w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (l == 0) {
    red[w] = a;
    red[32 + w] = b;
  }
  __syncthreads();
  a = l < nw ? red[l] : 0.f;
  b = l < nw ? red[32 + l] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = nan_max(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
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
// maximum, and the row is read once: thread t holds elements
// (t + k * blockDim) * V + e for k < K in registers.  K = 0: rows too wide
// for that are read a second time (h as written; each thread rereads only
// what it wrote itself).
template <typename T, bool NORM, int V, int K>
__global__ void __launch_bounds__(512) rows_kernel(const RowsParams p) {
  __shared__ float red[2][64];
  const T* xs = static_cast<const T*>(p.x);
  const T* rs = static_cast<const T*>(p.residual);
  T* hs = static_cast<T*>(p.h);
  T* ys = static_cast<T*>(p.y);
  constexpr int KR = K > 0 ? K : 1;
  const int step = blockDim.x * V, first = threadIdx.x * V;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, buf ^= 1) {
    const int64_t base = row * p.d;
    float u[KR][V];
    float sum = 0.f, top = 0.f;
    auto element = [&](int c, float* v) {
      load_vec<T, V>(xs + base + c, v);
      if constexpr (NORM) {
        if (rs) {
          float r[V];
          load_vec<T, V>(rs + base + c, r);
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] = round_to<T>(v[e] + r[e]);
        }
        if (hs) store_vec<T, V>(hs + base + c, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sum = fmaf(v[e], v[e], sum);
      }
    };
    auto gained = [&](int c, float* v) {
      if (NORM || p.gain) {
        float g[V];
        load_vec<float, V>(p.gain + c, g);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= g[e];
      }
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c < p.d) element(c, u[k]);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c < p.d) {
          gained(c, u[k]);
#pragma unroll
          for (int e = 0; e < V; ++e) top = nan_max(top, fabsf(u[k][e]));
        }
      }
    } else {
      for (int c = first; c < p.d; c += step) {
        element(c, u[0]);
        gained(c, u[0]);
#pragma unroll
        for (int e = 0; e < V; ++e) top = nan_max(top, fabsf(u[0][e]));
      }
    }
    block_sum_max(sum, top, red[buf]);
    const RowScale sc = row_scale(top);
    float rstd = 1.f;
    if constexpr (NORM) rstd = 1.f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
    if (threadIdx.x == 0) {
      if (p.codes) p.scale[row] = sc.s * rstd;
      if (NORM && p.rstd) p.rstd[row] = rstd;
    }
    auto finish = [&](int c, float* v) {
      if (p.codes) store_codes<V>(p.codes + row * p.ldc + c, v, sc);
      if (NORM && ys) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= rstd;
        store_vec<T, V>(ys + base + c, v);
      }
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c < p.d) finish(c, u[k]);
      }
    } else {
      const T* again = NORM && hs ? hs : xs;
      for (int c = first; c < p.d; c += step) {
        load_vec<T, V>(again + base + c, u[0]);
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
// (K = 0, any width), so the sum's order is fixed by the grid alone.
template <typename T, int V, int K>
__global__ void __launch_bounds__(512) norm_grad_kernel(const NormGradParams p) {
  extern __shared__ float acc_sm[];
  __shared__ float red[2][64];
  const T* dys = static_cast<const T*>(p.dy);
  const T* hs = static_cast<const T*>(p.h);
  const T* rs = static_cast<const T*>(p.dres);
  T* dxs = static_cast<T*>(p.dx);
  constexpr int KR = K > 0 ? K : 1;
  const int step = blockDim.x * V, first = threadIdx.x * V;
  float acc[KR][V];
  if constexpr (K > 0) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[k][e] = 0.f;
  } else {
    for (int c = first; c < p.d; c += step)
#pragma unroll
      for (int e = 0; e < V; ++e) acc_sm[c + e] = 0.f;
  }
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, buf ^= 1) {
    const int64_t base = row * p.d;
    const float rstd = p.rstd[row];
    float dot = 0.f, none = 0.f;
    float dy[KR][V], h[KR][V];
    auto dots = [&](int c, float* a, float* b, float* w) {
      float g[V];
      load_vec<float, V>(p.gamma + c, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        b[e] *= rstd;
        w[e] = fmaf(a[e], b[e], w[e]);
        a[e] *= g[e];
        dot = fmaf(a[e], b[e], dot);
      }
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c < p.d) {
          load_vec<T, V>(dys + base + c, dy[k]);
          load_vec<T, V>(hs + base + c, h[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c < p.d) dots(c, dy[k], h[k], acc[k]);
      }
    } else {
      for (int c = first; c < p.d; c += step) {
        load_vec<T, V>(dys + base + c, dy[0]);
        load_vec<T, V>(hs + base + c, h[0]);
        dots(c, dy[0], h[0], acc_sm + c);
      }
    }
    block_sum_max(dot, none, red[buf]);
    const float mean = dot / static_cast<float>(p.d);
    auto finish = [&](int c, const float* a, const float* b) {
      float o[V];
      if (rs) load_vec<T, V>(rs + base + c, o);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = fmaf(-b[e], mean, a[e]);
        o[e] = rs ? fmaf(rstd, v, o[e]) : rstd * v;
      }
      store_vec<T, V>(dxs + base + c, o);
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = first + k * step;
        if (c < p.d) finish(c, dy[k], h[k]);
      }
    } else {
      for (int c = first; c < p.d; c += step) {
        float g[V];
        load_vec<T, V>(dys + base + c, dy[0]);
        load_vec<T, V>(hs + base + c, h[0]);
        load_vec<float, V>(p.gamma + c, g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dy[0][e] *= g[e];
          h[0][e] *= rstd;
        }
        finish(c, dy[0], h[0]);
      }
    }
  }
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.d;
  if constexpr (K > 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * step;
      if (c < p.d) store_vec<float, V>(out + c, acc[k]);
    }
  } else {
    for (int c = first; c < p.d; c += step) store_vec<float, V>(out + c, acc_sm + c);
  }
}

// out[c] (+)= sum of part[g][c] over g < n, in a fixed order: 32 columns per
// block, eight slices of g summed apart and then together.
__global__ void __launch_bounds__(256) sum_partials_kernel(const float* __restrict__ part, int n, int d,
                                                           float* __restrict__ out, int accumulate) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
    for (int g = slice; g < n; g += 8) s += part[static_cast<int64_t>(g) * d + c];
  sm[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sm[k][lane];
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

// A warp takes 32 * V columns of a row: with V = 8, four lanes hold a group.
template <typename T, int V>
__global__ void __launch_bounds__(256) checkpoint_save_kernel(const T* __restrict__ x, int64_t T_, int d,
                                                              int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const int lane = threadIdx.x & 31;
  const int ng = (d + GROUP - 1) / GROUP;
  const int chunks = (d + 32 * V - 1) / (32 * V);
  const int64_t items = T_ * chunks;
  constexpr int LG = GROUP / V;  // lanes of a group
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += nw) {
    const int64_t row = it / chunks;
    const int c = static_cast<int>(it - row * chunks) * 32 * V + lane * V;
    float v[V];
    float top = 0.f;
    if (c < d) {
      load_vec<T, V>(x + row * d + c, v);
#pragma unroll
      for (int e = 0; e < V; ++e) top = nan_max(top, fabsf(v[e]));
    }
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (c < d) {
      const uint32_t eb = group_exponent(top);
      const float inv = exponent_inverse(eb);
      if (top > __uint_as_float(kMaxKept)) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          v[e] = copysignf(fminf(fabsf(v[e]), __uint_as_float(kMaxKept)), v[e]);
      }
      if (lane % LG == 0) exps[row * ng + c / GROUP] = static_cast<uint8_t>(eb);
      if constexpr (V == 1) {
        codes[row * d + c] = static_cast<int8_t>(checkpoint_code(v[0], inv));
      } else {
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = checkpoint_code(v[e], inv);
        uint2 w;
        w.x = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
        w.y = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
        *reinterpret_cast<uint2*>(codes + row * d + c) = w;
      }
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) checkpoint_load_kernel(const int8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ exps, int64_t T_, int d,
                                                              T* __restrict__ x) {
  const int lane = threadIdx.x & 31;
  const int ng = (d + GROUP - 1) / GROUP;
  const int chunks = (d + 32 * V - 1) / (32 * V);
  const int64_t items = T_ * chunks;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += nw) {
    const int64_t row = it / chunks;
    const int c = static_cast<int>(it - row * chunks) * 32 * V + lane * V;
    if (c >= d) continue;
    const float s = exponent_value(exps[row * ng + c / GROUP]);
    float v[V];
    if constexpr (V == 1) {
      v[0] = static_cast<float>(codes[row * d + c]) * s;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(codes + row * d + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = static_cast<float>(static_cast<int8_t>(w.x >> (8 * e))) * s;
        v[4 + e] = static_cast<float>(static_cast<int8_t>(w.y >> (8 * e))) * s;
      }
    }
    store_vec<T, V>(x + row * d + c, v);
  }
}

}  // namespace q8
}  // namespace poetx
