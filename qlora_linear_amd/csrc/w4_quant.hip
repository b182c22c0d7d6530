// Packing of the 4-bit group-scaled weight and its way back (gfx950).
//
// Layout (norm_w4.h): tiles of 16 rows x 128 columns, 1024 bytes; byte
// 256 g + 16 r + 4 q + i holds row r, columns 32 q + 8 g + i (low nibble) and
// 32 q + 8 g + i + 4 (high nibble). One thread owns one 4-byte word: the eight
// consecutive columns 32 q + 8 g .. + 7 of its row.
#include "device_common.h"
#include "norm_w4_launch.h"

namespace lnf4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
}

// rint of the float32 quotient v / s, |v / s| <= 16. The product with the reciprocal
// (1 ulp: off by less than 16 * 2^-22) decides all but the quotients near a half, where it
// may lie on the other side; those (a lane in eight of a wave, for bf16 weights) are
// divided, as are all of a scale whose reciprocal overflows (the comparison is then false).
__device__ __forceinline__ float rint_quotient(float v, float s, float inv) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's last bit is 1
  float n = __builtin_fmaf(v, inv, kMagic) - kMagic;
  if (!(fabsf(__builtin_fmaf(v, inv, -n)) < 0.5f - 0x1p-16f)) n = __builtin_rintf(__fdiv_rn(v, s));
  return n;
}

// The float32 quotient r / d for d = 7 or 15, r >= 0 finite: the product with the rounded
// reciprocal c and one correction by its exact remainder. The correctly rounded quotient
// for every such r (compared with the division for all 2^31 of them, subnormal ones too); the
// product alone moves one scale in 10^5 by a bf16 step where the quotient is next to a tie.
__device__ __forceinline__ float quotient_of(float r, float d, float c) {
  const float p = r * c;
  return __builtin_fmaf(__builtin_fmaf(-p, d, r), c, p);
}

// Minimum and maximum over the 4, 8 or 16 consecutive lanes of a group, by lane moves
// inside a row of 16: neighbours, then pairs, are exchanged; after that quads hold one
// value each and mirrors join them.
template <int CTRL>
__device__ __forceinline__ void join_extrema(float& lo, float& hi) {
  auto moved = [](float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  };
  lo = fminf(lo, moved(lo));
  hi = fmaxf(hi, moved(hi));
}
__device__ __forceinline__ void group_extrema(int group, float& lo, float& hi) {
  join_extrema<0xB1>(lo, hi);                     // quad_perm 1 0 3 2
  join_extrema<0x4E>(lo, hi);                     // quad_perm 2 3 0 1
  if (group >= 64) join_extrema<0x141>(lo, hi);   // row_half_mirror
  if (group >= 128) join_extrema<0x140>(lo, hi);  // row_mirror
}

// One 256-thread workgroup per tile. Thread t: row t >> 4, columns 8 (t & 15) .. + 7,
// so a group is G / 8 consecutive lanes. Bound by its arithmetic rather than by HBM
// (27 vector instructions an element by the counter, which keep the vector units busy all of
// the time, 13.6 us of 4-cycle issues at 2 GHz): no division as a rule, the codes put together as
// floats (sums of multiples of powers of 16 below 2^16 are exact), two conversions a word.
// 4096 x 4096 bf16 13.8 us, 3.1 TB/s.
template <typename In>
__global__ __launch_bounds__(kThreads) void w4_quantize_kernel(const In* __restrict__ w, int64_t N, int64_t K,
                                                               int kt, int group, uint32_t* __restrict__ codes,
                                                               uint16_t* __restrict__ scales,
                                                               uint8_t* __restrict__ zeros) {
  const int64_t tile = blockIdx.x;
  const int64_t n0 = tile / kt * 16;
  const int64_t k0 = (tile % kt) * 128;
  const int r = threadIdx.x >> 4, c8 = threadIdx.x & 15;
  const int64_t n = n0 + r, k = k0 + 8 * c8;
  const bool in_k = k < K, ok = n < N && in_k;  // K is a multiple of 64: eight columns exist or none
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (ok) load8(w + n * K + k, v);
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, v[j]);
    hi = fmaxf(hi, v[j]);
  }
  group_extrema(group, lo, hi);
  const bool asym = zeros != nullptr;
  const uint16_t sb = to_bf16(asym ? quotient_of(hi - lo, 15.f, 1.f / 15.f) : quotient_of(fmaxf(-lo, hi), 7.f, 1.f / 7.f));
  const float s = bf16_to_f32(sb);
  const float inv = __builtin_amdgcn_rcpf(s);
  float z = 8.f;
  if (asym) z = s > 0.f ? fminf(fmaxf(rint_quotient(-lo, s, inv), 0.f), 15.f) : 0.f;
  float half[2] = {0.f, 0.f};  // the word's two halves
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float n = s > 0.f ? rint_quotient(v[j], s, inv) : 0.f;
    const float c = __builtin_amdgcn_fmed3f(n + z, 0.f, 15.f);
    half[(j & 3) >> 1] += c * static_cast<float>(1 << (8 * (j & 1) + 4 * (j >> 2)));
  }
  uint32_t word = static_cast<uint32_t>(half[0]) | static_cast<uint32_t>(half[1]) << 16;
  if (!ok) word = 0;
  const int q = c8 >> 2, g = c8 & 3;
  codes[tile * 256 + 64 * g + 4 * r + q] = word;
  if ((c8 & (group / 8 - 1)) == 0 && in_k) {
    const int64_t at = (n0 / 16 * (K / group) + k / group) * 16 + r;
    scales[at] = ok ? sb : uint16_t(0);
    if (asym) zeros[at] = ok ? static_cast<uint8_t>(z) : uint8_t(0);
  }
}

// The same split on the way back, bound by HBM: 4096 x 4096 to bf16 10 us, 4.2 TB/s.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void w4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                 const uint16_t* __restrict__ scales,
                                                                 const uint8_t* __restrict__ zeros, int64_t N,
                                                                 int64_t K, int kt, int group,
                                                                 void* __restrict__ out) {
  const int64_t tile = blockIdx.x;
  const int64_t n0 = tile / kt * 16;
  const int64_t k0 = (tile % kt) * 128;
  const int r = threadIdx.x >> 4, c8 = threadIdx.x & 15;
  const int64_t n = n0 + r, k = k0 + 8 * c8;
  if (n >= N || k >= K) return;
  const uint32_t word = codes[tile * 256 + 64 * (c8 & 3) + 4 * r + (c8 >> 2)];
  const int64_t at = (n0 / 16 * (K / group) + k / group) * 16 + r;
  const float s = bf16_to_f32(scales[at]), z = zeros == nullptr ? 8.f : static_cast<float>(zeros[at]);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = (static_cast<float>((word >> (8 * (j & 3) + 4 * (j >> 2))) & 15u) - z) * s;
  const int64_t o = n * K + k;
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) =
        uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace

hipError_t launch_w4_quantize(const void* w, bool w_is_bf16, int64_t N, int64_t K, int group, uint8_t* codes,
                              uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  const int64_t kt = (K + 127) / 128, tiles = (N + 15) / 16 * kt;
  const dim3 grid(static_cast<unsigned>(tiles));
  if (w_is_bf16)
    w4_quantize_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const uint16_t*>(w), N, K, static_cast<int>(kt),
                                                      group, reinterpret_cast<uint32_t*>(codes), scales, zeros);
  else
    w4_quantize_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const float*>(w), N, K, static_cast<int>(kt), group,
                                                      reinterpret_cast<uint32_t*>(codes), scales, zeros);
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                                int64_t K, int group, bool out_bf16, void* out, hipStream_t stream) {
  const int64_t kt = (K + 127) / 128, tiles = (N + 15) / 16 * kt;
  const dim3 grid(static_cast<unsigned>(tiles));
  const auto c = reinterpret_cast<const uint32_t*>(codes);
  if (out_bf16)
    w4_dequantize_kernel<true><<<grid, kThreads, 0, stream>>>(c, scales, zeros, N, K, static_cast<int>(kt), group, out);
  else
    w4_dequantize_kernel<false><<<grid, kThreads, 0, stream>>>(c, scales, zeros, N, K, static_cast<int>(kt), group, out);
  return hipGetLastError();
}

}  // namespace lnf4
