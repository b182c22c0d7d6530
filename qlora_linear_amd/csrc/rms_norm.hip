// RMS norm with the residual's addition, 8-bit output and gradient (gfx950).
//
//     h = round(x + res), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w
//     dx = dh + rstd (g - n mean(g n)),  dw = sum_t dy n,  g = dy w, n = h rstd
//
// One workgroup per row; every sum in float32.
#include "device_common.h"
#include "norm_w4_launch.h"

namespace lnf4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load1(const uint16_t* p, int64_t i) { return bf16_to_f32(p[i]); }
__device__ __forceinline__ void store1(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store1(uint16_t* p, int64_t i, float v) { p[i] = to_bf16(v); }
__device__ __forceinline__ float round_to(const float*, float v) { return v; }
__device__ __forceinline__ float round_to(const uint16_t*, float v) { return bf16_to_f32(to_bf16(v)); }

// Sum and maximum over the workgroup, the same in every thread.
__device__ __forceinline__ void block_sum_max(float& s, float& m, float (*red)[kThreads / 64]) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    m = fmaxf(m, __shfl_xor(m, o));
  }
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = s;
    red[1][threadIdx.x >> 6] = m;
  }
  __syncthreads();
  s = red[0][0] + red[0][1] + red[0][2] + red[0][3];
  m = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xFF);
}
__device__ __forceinline__ uint8_t to_i8(float v) {
  return static_cast<uint8_t>(static_cast<int>(__builtin_rintf(fminf(fmaxf(v, -127.f), 127.f))));
}

template <typename E, int OUT>
__global__ __launch_bounds__(kThreads) void rmsnorm_fwd_kernel(int d, float eps, const E* __restrict__ x,
                                                               const E* __restrict__ res, const E* __restrict__ w,
                                                               E* __restrict__ h, void* __restrict__ y,
                                                               float* __restrict__ q_scale,
                                                               float* __restrict__ rstd_out) {
  __shared__ float red[2][kThreads / 64];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * d;
  auto h_at = [&](int i) {
    const float v = load1(x, row + i);
    return res == nullptr ? v : round_to(x, v + load1(res, row + i));
  };
  float s = 0.f, m = 0.f;
  for (int i = threadIdx.x; i < d; i += kThreads) {
    const float v = h_at(i);
    s += v * v;
    m = fmaxf(m, fabsf(v * load1(w, i)));
  }
  block_sum_max(s, m, red);
  const float rstd = 1.0f / __builtin_sqrtf(s / static_cast<float>(d) + eps);
  const float scale = m * rstd / (OUT == kRowE4m3 ? 448.f : 127.f);
  for (int i = threadIdx.x; i < d; i += kThreads) {
    const float v = h_at(i);
    if (res != nullptr) store1(h, row + i, v);
    const float o = v * rstd * load1(w, i);
    if constexpr (OUT == kRowE4m3)
      static_cast<uint8_t*>(y)[row + i] = scale > 0.f ? to_e4m3(o / scale) : 0;
    else if constexpr (OUT == kRowI8)
      static_cast<uint8_t*>(y)[row + i] = scale > 0.f ? to_i8(o / scale) : 0;
    else
      store1(static_cast<E*>(y), row + i, o);
  }
  if (threadIdx.x == 0) {
    if (rstd_out != nullptr) rstd_out[blockIdx.x] = rstd;
    if (OUT == kRowE4m3 || OUT == kRowI8) q_scale[blockIdx.x] = scale;
  }
}

template <typename E>
__global__ __launch_bounds__(kThreads) void rmsnorm_bwd_kernel(int d, const E* __restrict__ dy,
                                                               const E* __restrict__ dh, const E* __restrict__ h,
                                                               const E* __restrict__ w,
                                                               const float* __restrict__ rstd_in,
                                                               E* __restrict__ dx) {
  __shared__ float red[2][kThreads / 64];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * d;
  const float rstd = rstd_in[blockIdx.x];
  float s = 0.f, m = 0.f;
  for (int i = threadIdx.x; i < d; i += kThreads)
    s += load1(dy, row + i) * load1(w, i) * (load1(h, row + i) * rstd);
  block_sum_max(s, m, red);
  const float c = s / static_cast<float>(d);
  for (int i = threadIdx.x; i < d; i += kThreads) {
    const float g = load1(dy, row + i) * load1(w, i), n = load1(h, row + i) * rstd;
    const float v = rstd * (g - n * c);
    store1(dx, row + i, dh == nullptr ? v : v + load1(dh, row + i));
  }
}

// One thread per column; consecutive rows are summed in float32 partials of 64 rows.
template <typename E>
__global__ __launch_bounds__(kThreads) void rmsnorm_dw_kernel(int64_t T, int d, const E* __restrict__ dy,
                                                              const E* __restrict__ h,
                                                              const float* __restrict__ rstd, E* __restrict__ dw) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= d) return;
  float total = 0.f;
  for (int64_t t0 = 0; t0 < T; t0 += 64) {
    float s = 0.f;
    for (int64_t t = t0; t < T && t < t0 + 64; ++t) s += load1(dy, t * d + i) * (load1(h, t * d + i) * rstd[t]);
    total += s;
  }
  store1(dw, i, total);
}

template <typename E>
__global__ __launch_bounds__(kThreads) void zero_kernel(E* __restrict__ p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i < n) p[i] = E(0);
}

template <typename E>
hipError_t fwd(int64_t T, int d, float eps, const void* x, const void* res, const void* w, void* h, int out, void* y,
               float* q_scale, float* rstd, hipStream_t stream) {
  const auto xe = static_cast<const E*>(x), re = static_cast<const E*>(res), we = static_cast<const E*>(w);
  const dim3 grid(static_cast<unsigned>(T));
  if (out == kRowE4m3)
    rmsnorm_fwd_kernel<E, kRowE4m3><<<grid, kThreads, 0, stream>>>(d, eps, xe, re, we, static_cast<E*>(h), y, q_scale, rstd);
  else if (out == kRowI8)
    rmsnorm_fwd_kernel<E, kRowI8><<<grid, kThreads, 0, stream>>>(d, eps, xe, re, we, static_cast<E*>(h), y, q_scale, rstd);
  else
    rmsnorm_fwd_kernel<E, kRowF32><<<grid, kThreads, 0, stream>>>(d, eps, xe, re, we, static_cast<E*>(h), y, q_scale, rstd);
  return hipGetLastError();
}

template <typename E>
hipError_t bwd(int64_t T, int d, const void* dy, const void* dh, const void* h, const void* w, const float* rstd,
               void* dx, void* dw, hipStream_t stream) {
  const auto dye = static_cast<const E*>(dy), he = static_cast<const E*>(h);
  rmsnorm_bwd_kernel<E><<<dim3(static_cast<unsigned>(T)), kThreads, 0, stream>>>(
      d, dye, static_cast<const E*>(dh), he, static_cast<const E*>(w), rstd, static_cast<E*>(dx));
  if (dw != nullptr)
    rmsnorm_dw_kernel<E><<<dim3((d + kThreads - 1) / kThreads), kThreads, 0, stream>>>(T, d, dye, he, rstd,
                                                                                      static_cast<E*>(dw));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(int64_t T, int d, int dtype, float eps, const void* x, const void* residual,
                              const void* w, void* h, int out, void* y, float* q_scale, float* rstd,
                              hipStream_t stream) {
  return dtype == kRowBf16 ? fwd<uint16_t>(T, d, eps, x, residual, w, h, out, y, q_scale, rstd, stream)
                           : fwd<float>(T, d, eps, x, residual, w, h, out, y, q_scale, rstd, stream);
}

size_t rmsnorm_bwd_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_rmsnorm_bwd(int64_t T, int d, int dtype, const void* dy, const void* dh, const void* h,
                              const void* w, const float* rstd, void* dx, void* dw, void*, hipStream_t stream) {
  return dtype == kRowBf16 ? bwd<uint16_t>(T, d, dy, dh, h, w, rstd, dx, dw, stream)
                           : bwd<float>(T, d, dy, dh, h, w, rstd, dx, dw, stream);
}

hipError_t launch_zero(void* p, int64_t n, int dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads));
  if (dtype == kRowBf16) zero_kernel<<<grid, kThreads, 0, stream>>>(static_cast<uint16_t*>(p), n);
  else zero_kernel<<<grid, kThreads, 0, stream>>>(static_cast<float*>(p), n);
  return hipGetLastError();
}

}  // namespace lnf4
