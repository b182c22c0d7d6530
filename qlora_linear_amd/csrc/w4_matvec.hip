// y = x W^T for a few rows of x and a packed 4-bit group-scaled weight (gfx950).
//
// One wave per (output row, four rows of x): lanes take words of eight codes, sum
// x c and x over the word, and add s (sum x c - z sum x) in float32.
#include "device_common.h"
#include "norm_w4_launch.h"

namespace lnf4 {
namespace {

__device__ __forceinline__ float x_value(const uint16_t* p, int64_t i) { return bf16_to_f32(p[i]); }
__device__ __forceinline__ float x_value(const int8_t* p, int64_t i) { return static_cast<float>(p[i]); }
struct E4m3 {
  uint8_t v;
};
__device__ __forceinline__ float x_value(const E4m3* p, int64_t i) {
  return __builtin_amdgcn_cvt_f32_fp8(p[i].v, 0);
}

template <typename X>
__global__ __launch_bounds__(64) void w4_matvec_kernel(int64_t T, int K, int group, const X* __restrict__ x,
                                                       const float* __restrict__ x_scale, const W4Table tab,
                                                       bool y_bf16) {
  int64_t n = static_cast<int64_t>(blockIdx.x);
  int p = 0;
  while (n >= tab.row_end[p] * int64_t(16)) ++p;
  if (p > 0) n -= tab.row_end[p - 1] * int64_t(16);
  const int N = tab.N[p];
  if (n >= N) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 4;
  const int kt = (K + 127) / 128, kg = K / group;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(tab.codes[p]) + n / 16 * kt * 256;
  const int64_t sbase = n / 16 * kg;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 8 * threadIdx.x; k < K; k += 512) {
    const int c8 = (k & 127) >> 3;
    const uint32_t word = codes[(k >> 7) * 256 + 64 * (c8 & 3) + 4 * (n & 15) + (c8 >> 2)];
    const int64_t at = (sbase + k / group) * 16 + (n & 15);
    const float s = bf16_to_f32(tab.scales[p][at]);
    const float z = tab.zeros[p] == nullptr ? 8.f : static_cast<float>(tab.zeros[p][at]);
    for (int t = 0; t < 4; ++t) {
      if (t0 + t >= T) break;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sum += x_value(x, (t0 + t) * K + k + j) *
               (static_cast<float>((word >> (8 * (j & 3) + 4 * (j >> 2))) & 15u) - z);
      acc[t] += s * sum;
    }
  }
  for (int t = 0; t < 4; ++t) {
    if (t0 + t >= T) break;
    float v = acc[t];
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if (threadIdx.x == 0) {
      if (x_scale != nullptr) v *= x_scale[t0 + t];
      const int64_t at = (t0 + t) * N + n;
      if (y_bf16) static_cast<uint16_t*>(tab.y[p])[at] = to_bf16(v);
      else static_cast<float*>(tab.y[p])[at] = v;
    }
  }
}

}  // namespace

hipError_t launch_w4_matvec(int64_t T, int K, int group, int x_type, const void* x, const float* x_scale,
                            const W4Table& tab, bool y_bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(tab.row_end[tab.n - 1] * 16), static_cast<unsigned>((T + 3) / 4));
  if (x_type == kRowBf16)
    w4_matvec_kernel<<<grid, 64, 0, stream>>>(T, K, group, static_cast<const uint16_t*>(x), x_scale, tab, y_bf16);
  else if (x_type == kRowE4m3)
    w4_matvec_kernel<<<grid, 64, 0, stream>>>(T, K, group, static_cast<const E4m3*>(x), x_scale, tab, y_bf16);
  else
    w4_matvec_kernel<<<grid, 64, 0, stream>>>(T, K, group, static_cast<const int8_t*>(x), x_scale, tab, y_bf16);
  return hipGetLastError();
}

}  // namespace lnf4
