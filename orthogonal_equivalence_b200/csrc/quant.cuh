// POET-XQ (POET-X write-up, section "POET-XQ：量化训练的额外红利"): the frozen
// base weight is stored quantized and only dequantized at run time, with no
// quantization-aware training.  The write-up fixes neither the format nor
// the granularity; the reading taken here is the plain 8-bit one it compares
// against: int8 codes, symmetric, one fp32 scale per row of the stored
// [n][m] weight (one per output feature), scale = max|row| / 127,
// code = round-half-even(w / scale) clamped to [-127, 127], w ~= code * scale.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace poetx {

template <typename T>
__device__ __forceinline__ float load_f32(const T* p, int64_t i);
template <>
__device__ __forceinline__ float load_f32<float>(const float* p, int64_t i) { return p[i]; }
template <>
__device__ __forceinline__ float load_f32<__nv_bfloat16>(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}

// One block per row: absmax by a block reduction, then the codes.  A row that
// holds an infinity or a NaN gets codes 0 and scale NaN, as in q8.cuh: the
// maximum is taken over the magnitudes' bits, which keeps a NaN above all else.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ W, int64_t rows, int cols,
                                                            int8_t* __restrict__ Wq, float* __restrict__ scale) {
  __shared__ uint32_t red[8];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* w = W + r * cols;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) top = max(top, __float_as_uint(load_f32(w, c)) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
      const uint32_t v = __reduce_max_sync(0xffffffffu, threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0u);
      if (threadIdx.x == 0) red[0] = v;
    }
    __syncthreads();
    const float amax = __uint_as_float(red[0]);
    const bool finite = amax <= 3.402823466e38f;
    const float s = finite ? amax / 127.f : __uint_as_float(0x7fffffffu);
    if (threadIdx.x == 0) scale[r] = s;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      float q = 0.f;
      if (s > 0.f) q = fminf(fmaxf(rintf(load_f32(w, c) / s), -127.f), 127.f);
      Wq[r * cols + c] = static_cast<int8_t>(q);
    }
    __syncthreads();  // red[] is reused by the next row
  }
}

// (w = code * scale, rounded once to the weight dtype, is q8::expand_kernel in
// q8.cuh, which reads any rows of codes.)

}  // namespace poetx
