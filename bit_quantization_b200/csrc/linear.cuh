// y = x W^T with NVFP4 weights as nvfp4_quantize leaves them (E2M1 codes
// [N, K/2], UE4M3 scales [N, K/16] of 16-element blocks, fp32 tensor scale)
// and few 16-bit rows x [M, K]: the projections of a generation step.
#pragma once
#include "tc.cuh"

namespace thrift {

// E2M1 code -> value.
__device__ __forceinline__ float e2m1_decode(uint32_t c) {
  const uint32_t m = c & 7u;
  const float a = m < 2 ? 0.5f * (float)m
                        : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return (c & 8u) ? -a : a;
}

constexpr int kLinMaxM = 64;

// One warp per weight row: lanes stride over its 16-blocks, the products of
// a block summed before its scale.
template <int DT>
__global__ void __launch_bounds__(256) linear_kernel(const uint16_t* __restrict__ x, int M, int K,
                                                     int N, const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales,
                                                     const float* __restrict__ gs,
                                                     uint16_t* __restrict__ y) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= N) return;
  for (int m = 0; m < M; ++m) {
    float acc = 0.0f;
    for (int kb = lane; kb < K / 16; kb += 32) {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + (int64_t)n * (K / 2)) + kb);
      const float s = ue4m3_decode(__ldg(scales + (int64_t)n * (K / 16) + kb));
      float p = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        p = fmaf(e2m1_decode((e < 8 ? c.x : c.y) >> (4 * (e & 7))),
                 h2f<DT>(__ldg(x + (int64_t)m * K + 16 * kb + e)), p);
      acc = fmaf(p, s, acc);
    }
    for (int k = lane; k < K; k += 32)  // a row holding a value that is not finite is NaN
      if (!finite_f(h2f<DT>(__ldg(x + (int64_t)m * K + k)))) acc = NAN;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) y[(int64_t)m * N + n] = f2h<DT>(acc * __ldg(gs));
  }
}

}  // namespace thrift
