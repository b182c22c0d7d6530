// Internal launchers of the RMS norm and the packed 4-bit weight. Arguments are
// validated by norm_w4_api.hip; each launcher only enqueues work on `stream` and
// returns the hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lnf4 {

enum RowType { kRowF32 = 0, kRowBf16 = 1, kRowE4m3 = 2, kRowI8 = 3 };  // ln_dtype, ln_qtype

// y (of type out: bf16 / f32 as dtype, or 8 bits with q_scale) = norm of x (+ residual).
hipError_t launch_rmsnorm_fwd(int64_t T, int d, int dtype, float eps, const void* x, const void* residual,
                              const void* w, void* h, int out, void* y, float* q_scale, float* rstd,
                              hipStream_t stream);
size_t rmsnorm_bwd_bytes(int64_t T, int64_t d);
hipError_t launch_rmsnorm_bwd(int64_t T, int d, int dtype, const void* dy, const void* dh, const void* h,
                              const void* w, const float* rstd, void* dx, void* dw, void* workspace,
                              hipStream_t stream);
// n elements of dtype set to zero.
hipError_t launch_zero(void* p, int64_t n, int dtype, hipStream_t stream);

hipError_t launch_w4_quantize(const void* w, bool w_is_bf16, int64_t N, int64_t K, int group, uint8_t* codes,
                              uint16_t* scales, uint8_t* zeros, hipStream_t stream);
hipError_t launch_w4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                                int64_t K, int group, bool out_bf16, void* out, hipStream_t stream);

constexpr int kW4MaxProj = 8;
// Weights of one launch; group_end[g] (set by the launcher) = workgroups along the rows
// of weights 0 .. g.
struct W4Table {
  int n;
  int group_end[kW4MaxProj];
  int N[kW4MaxProj];
  const uint8_t* codes[kW4MaxProj];
  const uint16_t* scales[kW4MaxProj];
  const uint8_t* zeros[kW4MaxProj];
  void* y[kW4MaxProj];
};
// Bytes of float32 partial sums, where d_in is split across workgroups (else 0).
size_t w4_matvec_bytes(int64_t T, int64_t K, int n, const int* N);
hipError_t launch_w4_matvec(int64_t T, int K, int group, int x_type, const void* x, const float* x_scale,
                            const W4Table& tab, bool y_bf16, void* workspace, hipStream_t stream);

}  // namespace lnf4
