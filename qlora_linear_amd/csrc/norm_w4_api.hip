// C ABI of the RMS norm and the packed 4-bit weight (declared in include/norm_w4.h).
//
// Every entry point validates its arguments on the host before touching HIP, so
// argument errors are reported without a GPU and nothing is enqueued on error.
#include <cmath>
#include <cstdint>

#include "api_check.h"
#include "norm_w4.h"
#include "norm_w4_launch.h"

namespace {

using namespace lnf4;

bool plain_type(int t) { return t == LN_F32 || t == LN_BF16; }
size_t type_bytes(int t) { return t == LN_F32 ? 4 : t == LN_BF16 ? 2 : 1; }

int check_norm(int64_t T, int64_t d, int dtype, float eps) {
  if (T < 0 || d < 1 || !plain_type(dtype) || !std::isfinite(eps) || !(eps > 0.f)) return LN_EINVAL;
  if (T > kMaxDim || d > LN_NORM_MAX_D) return LN_ESHAPE;
  return LN_OK;
}

int norm_fwd(int64_t T, int64_t d, int dtype, float eps, const void* x, const void* residual, const void* w, void* h,
             int out_type, void* y, float* q_scale, float* rstd, void* stream) {
  if (w == nullptr) return LN_EINVAL;
  if (T != 0 && (x == nullptr || y == nullptr)) return LN_EINVAL;
  const bool quant = out_type != dtype;
  if (T != 0 && quant && q_scale == nullptr) return LN_EINVAL;
  if ((residual == nullptr) != (h == nullptr)) return LN_EINVAL;
  const int st = check_norm(T, d, dtype, eps);
  if (st != LN_OK) return st;
  if (T == 0) return LN_OK;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(h) || !aligned16(y) || !aligned16(q_scale) ||
      !aligned16(rstd))
    return LN_EALIGN;
  const size_t n = static_cast<size_t>(T) * d, e = type_bytes(dtype);
  const Span outs[4] = {{h, n * e}, {y, n * type_bytes(out_type)}, {q_scale, static_cast<size_t>(T) * 4},
                        {rstd, static_cast<size_t>(T) * 4}};
  const Span ins[3] = {{x, n * e}, {residual, n * e}, {w, static_cast<size_t>(d) * e}};
  if (any_alias(outs, 4, ins, 3)) return LN_EALIAS;
  return hip_status(launch_rmsnorm_fwd(T, static_cast<int>(d), dtype, eps, x, residual, w, h, out_type, y, q_scale,
                                       rstd, static_cast<hipStream_t>(stream)));
}

// The shape rules of a packed weight.
int check_w4(int64_t N, int64_t K, int32_t group) {
  if (N < 1 || K < 1) return LN_EINVAL;
  if (group != 32 && group != 64 && group != 128) return LN_ESHAPE;
  if (K % 64 != 0 || K % group != 0 || N > kMaxDim - 15 || K > LN_W4_MAX_D_IN) return LN_ESHAPE;
  // a launch has fewer than 2^32 threads along x: 256 a tile when packing
  if ((N + 15) / 16 * ((K + 127) / 128) >= (int64_t(1) << 24)) return LN_ESHAPE;
  return LN_OK;
}
constexpr int64_t kMaxW4Rows = int64_t(1) << 21;
constexpr int64_t kMaxW4Outputs = int64_t(1) << 35;  // of one launch (one thread to 16 of them at least)
size_t w4_code_bytes(int64_t N, int64_t K) { return static_cast<size_t>((N + 15) / 16 * ((K + 127) / 128)) * 1024; }
size_t w4_groups(int64_t N, int64_t K, int32_t group) { return static_cast<size_t>((N + 15) / 16 * (K / group)) * 16; }

}  // namespace

extern "C" {

int rmsnorm_fwd(int64_t T, int64_t d, int dtype, float eps, const void* x, const void* residual, const void* w,
                void* h, void* y, float* rstd, void* stream) {
  if (!plain_type(dtype)) return LN_EINVAL;
  return norm_fwd(T, d, dtype, eps, x, residual, w, h, dtype, y, nullptr, rstd, stream);
}

int rmsnorm_fwd_quant(int64_t T, int64_t d, int dtype, float eps, const void* x, const void* residual, const void* w,
                      void* h, int q_type, void* q, float* q_scale, void* stream) {
  if (q_type != LN_E4M3 && q_type != LN_I8) return LN_EINVAL;
  return norm_fwd(T, d, dtype, eps, x, residual, w, h, q_type, q, q_scale, nullptr, stream);
}

size_t rmsnorm_bwd_workspace_bytes(int64_t T, int64_t d) {
  if (T == 0 || check_norm(T, d, LN_F32, 1.f) != LN_OK) return 0;
  return rmsnorm_bwd_bytes(T, d);
}

int rmsnorm_bwd(int64_t T, int64_t d, int dtype, const void* dy, const void* dh, const void* h, const void* w,
                const float* rstd, void* dx, void* dw, void* workspace, size_t workspace_bytes, void* stream) {
  if (w == nullptr) return LN_EINVAL;
  if (T != 0 && (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr)) return LN_EINVAL;
  const int st = check_norm(T, d, dtype, 1.f);
  if (st != LN_OK) return st;
  if (!aligned16(dw)) return LN_EALIGN;
  const auto hs = static_cast<hipStream_t>(stream);
  if (T == 0) return dw == nullptr ? LN_OK : hip_status(launch_zero(dw, d, dtype, hs));
  if (!aligned16(dy) || !aligned16(dh) || !aligned16(h) || !aligned16(w) || !aligned16(rstd) || !aligned16(dx))
    return LN_EALIGN;
  const size_t need = dw == nullptr ? 0 : rmsnorm_bwd_bytes(T, d);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return LN_EWORKSPACE;
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LN_EALIGN;
  const size_t n = static_cast<size_t>(T) * d, e = type_bytes(dtype);
  const Span outs[3] = {{dx, n * e}, {dw, static_cast<size_t>(d) * e}, {need > 0 ? workspace : nullptr, need}};
  const Span ins[5] = {{dy, n * e}, {dh, n * e}, {h, n * e}, {w, static_cast<size_t>(d) * e},
                       {rstd, static_cast<size_t>(T) * 4}};
  if (any_alias(outs, 3, ins, 5)) return LN_EALIAS;
  return hip_status(launch_rmsnorm_bwd(T, static_cast<int>(d), dtype, dy, dh, h, w, rstd, dx, dw, workspace, hs));
}

int w4_quantize(const void* w, int w_dtype, int64_t d_out, int64_t d_in, int32_t group, uint8_t* codes,
                uint16_t* scales, uint8_t* zeros, void* stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr || !plain_type(w_dtype)) return LN_EINVAL;
  const int st = check_w4(d_out, d_in, group);
  if (st != LN_OK) return st;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros)) return LN_EALIGN;
  const size_t gs = w4_groups(d_out, d_in, group);
  const Span outs[3] = {{codes, w4_code_bytes(d_out, d_in)}, {scales, gs * 2}, {zeros, gs}};
  const Span ins[1] = {{w, static_cast<size_t>(d_out) * d_in * type_bytes(w_dtype)}};
  if (any_alias(outs, 3, ins, 1)) return LN_EALIAS;
  return hip_status(launch_w4_quantize(w, w_dtype == LN_BF16, d_out, d_in, group, codes, scales, zeros,
                                       static_cast<hipStream_t>(stream)));
}

int w4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t d_out, int64_t d_in,
                  int32_t group, int out_dtype, void* out, void* stream) {
  if (codes == nullptr || scales == nullptr || out == nullptr || !plain_type(out_dtype)) return LN_EINVAL;
  const int st = check_w4(d_out, d_in, group);
  if (st != LN_OK) return st;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(zeros) || !aligned16(out)) return LN_EALIGN;
  const size_t gs = w4_groups(d_out, d_in, group);
  const Span outs[1] = {{out, static_cast<size_t>(d_out) * d_in * type_bytes(out_dtype)}};
  const Span ins[3] = {{codes, w4_code_bytes(d_out, d_in)}, {scales, gs * 2}, {zeros, gs}};
  if (any_alias(outs, 1, ins, 3)) return LN_EALIAS;
  return hip_status(launch_w4_dequantize(codes, scales, zeros, d_out, d_in, group, out_dtype == LN_BF16, out,
                                         static_cast<hipStream_t>(stream)));
}

size_t w4_matvec_multi_workspace_bytes(int64_t T, int64_t d_in, int32_t n_proj, const int64_t* d_out) {
  if (T < 1 || T > kMaxW4Rows || n_proj < 1 || n_proj > LN_MAX_PROJ || d_out == nullptr) return 0;
  int N[LN_MAX_PROJ];
  for (int g = 0; g < n_proj; ++g) {
    if (check_w4(d_out[g], d_in, 32) != LN_OK) return 0;
    N[g] = static_cast<int>(d_out[g]);
  }
  return w4_matvec_bytes(T, d_in, n_proj, N);
}

size_t w4_matvec_workspace_bytes(int64_t T, int64_t d_in, int64_t d_out) {
  return w4_matvec_multi_workspace_bytes(T, d_in, 1, &d_out);
}

int w4_matvec_multi(int64_t T, int64_t d_in, int32_t n_proj, const int64_t* d_out, int32_t group, int x_dtype,
                    const void* x, const float* x_scale, const uint8_t* const* codes, const uint16_t* const* scales,
                    const uint8_t* const* zeros, int y_dtype, void* const* y, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (n_proj < 1 || n_proj > LN_MAX_PROJ || T < 0) return LN_EINVAL;
  if (d_out == nullptr || codes == nullptr || scales == nullptr || y == nullptr) return LN_EINVAL;
  if (T != 0 && x == nullptr) return LN_EINVAL;
  if ((x_dtype != LN_BF16 && x_dtype != LN_E4M3 && x_dtype != LN_I8) || !plain_type(y_dtype)) return LN_EINVAL;
  static_assert(LN_MAX_PROJ <= kW4MaxProj, "table size");
  W4Table tab{};
  Span outs[LN_MAX_PROJ + 1], ins[3 * LN_MAX_PROJ + 2];
  int n_in = 0;
  int64_t tiles = 0;
  const size_t t = static_cast<size_t>(T);
  tab.n = n_proj;
  for (int g = 0; g < n_proj; ++g) {
    if (codes[g] == nullptr || scales[g] == nullptr || (zeros != nullptr && zeros[g] == nullptr)) return LN_EINVAL;
    if (T != 0 && y[g] == nullptr) return LN_EINVAL;
    const int st = check_w4(d_out[g], d_in, group);
    if (st != LN_OK) return st;
    const uint8_t* z = zeros == nullptr ? nullptr : zeros[g];
    if (!aligned16(codes[g]) || !aligned16(scales[g]) || !aligned16(z) || !aligned16(y[g])) return LN_EALIGN;
    tiles += (d_out[g] + 15) / 16;
    if (tiles >= (int64_t(1) << 24)) return LN_ESHAPE;
    tab.N[g] = static_cast<int>(d_out[g]);
    tab.codes[g] = codes[g];
    tab.scales[g] = scales[g];
    tab.zeros[g] = z;
    tab.y[g] = y[g];
    const size_t gs = w4_groups(d_out[g], d_in, group);
    outs[g] = {y[g], t * static_cast<size_t>(d_out[g]) * type_bytes(y_dtype)};
    ins[n_in++] = {codes[g], w4_code_bytes(d_out[g], d_in)};
    ins[n_in++] = {scales[g], gs * 2};
    ins[n_in++] = {z, gs};
  }
  if (T > kMaxW4Rows || T * 16 * tiles > kMaxW4Outputs) return LN_ESHAPE;
  if (T == 0) return LN_OK;
  if (!aligned16(x) || !aligned16(x_scale)) return LN_EALIGN;
  const size_t need = w4_matvec_bytes(T, d_in, n_proj, tab.N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return LN_EWORKSPACE;
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LN_EALIGN;
  outs[n_proj] = {need > 0 ? workspace : nullptr, need};
  ins[n_in++] = {x, t * static_cast<size_t>(d_in) * type_bytes(x_dtype)};
  ins[n_in++] = {x_scale, t * 4};
  if (any_alias(outs, n_proj + 1, ins, n_in)) return LN_EALIAS;
  return hip_status(launch_w4_matvec(T, static_cast<int>(d_in), group, x_dtype, x, x_scale, tab, y_dtype == LN_BF16,
                                     workspace, static_cast<hipStream_t>(stream)));
}

int w4_matvec(int64_t T, int64_t d_in, int64_t d_out, int32_t group, int x_dtype, const void* x, const float* x_scale,
              const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int y_dtype, void* y,
              void* workspace, size_t workspace_bytes, void* stream) {
  return w4_matvec_multi(T, d_in, 1, &d_out, group, x_dtype, x, x_scale, &codes, &scales,
                         zeros == nullptr ? nullptr : &zeros, y_dtype, &y, workspace, workspace_bytes, stream);
}

}  // extern "C"
