// y = x W^T for a few rows of x and a packed 4-bit group-scaled weight (gfx950).
//
//     y[t][n] = x_scale[t] sum_g s[n][g] ( sum_{k in g} x[t][k] c[n][k] - z[n][g] sum_{k in g} x[t][k] )
//
// Bound by reading the packed weight once (half a byte an element) up to a few dozen
// rows of x. A workgroup owns R tiles of 16 weight rows over all of d_in; its W waves
// take the 128-column chunks w, w + W, ... independently, with no barrier until their
// sums meet in LDS. In a chunk
//   * a lane's 16 bytes of codes are four matrix-instruction operands (32 columns each)
//     in place: a wave reads 1024 consecutive bytes per tile, D chunks ahead;
//   * codes become operands in registers: bytes for int8 rows (3 instructions per eight
//     codes), and for the others bf16 by the E4M3 conversion with scale 2^9, as a byte c of
//     0 .. 15 is c 2^-9 in E4M3, whose subnormals and first binade are equidistant (7).
//     E4M3 rows widen to bf16 (exactly) as well: the E4M3 matrix instruction would take the
//     nibbles as they are, but its sums lose bits (single products of 32 columns 5e-6 to
//     1.4e-5 off, bf16 ones below 1e-8), as do f16 products with subnormal codes;
//   * the matrix instruction multiplies codes, not weights: the group's scale and zero
//     point are applied to its 16 x 16 sums. The zero point needs sum x over the group,
//     one more instruction with a constant operand, shared by the R tiles;
//   * x operands come straight from global memory (L2) in operand layout, 16 rows x 64
//     (8-bit: 32) bytes a load, as many chunks ahead as the codes: the counter that
//     loads retire by is in order, a shallower x ring would wait for the codes behind it.
// Sums over waves run in a fixed order: results do not depend on the run.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "norm_w4_launch.h"

namespace lnf4 {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint2 buf_load8(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, static_cast<int>(voff),
                                                                       static_cast<int>(soff), 0));
}
__device__ __forceinline__ uint32_t buf_load2(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff) {
  return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, static_cast<int>(voff),
                                                                    static_cast<int>(soff), 0));
}
__device__ __forceinline__ uint32_t buf_load1(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff) {
  return static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(rs, static_cast<int>(voff),
                                                                  static_cast<int>(soff), 0));
}

// Bytes 0, 1 or 2, 3 of v as E4M3 values times a power of two, as two bf16 (exact).
template <bool UPPER>
__device__ __forceinline__ uint32_t bf16_of_e4m3(uint32_t v, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, UPPER));
}

// The rows' type: operand registers, products, and what turns a group's sums into float.
template <int XT>
struct Rows;
template <>
struct Rows<kRowBf16> {
  typedef uint4 Op;    // 8 elements as loaded
  typedef uint4 Wide;  // 8 elements as multiplied
  typedef f32x4_t Acc;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ Op load(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t s) {
    return buf_load16(rs, at, s);
  }
  static __device__ __forceinline__ Wide widen(const Op& x) { return x; }
  static __device__ __forceinline__ Wide codes(uint32_t w) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    return Wide{bf16_of_e4m3<false>(lo, 512.f), bf16_of_e4m3<true>(lo, 512.f), bf16_of_e4m3<false>(hi, 512.f),
                bf16_of_e4m3<true>(hi, 512.f)};
  }
  static __device__ __forceinline__ Wide minus(bool eight) {
    const uint32_t v = eight ? 0xC100C100u : 0xBF80BF80u;  // -8 or -1
    return Wide{v, v, v, v};
  }
  static __device__ __forceinline__ Acc mma(const Wide& x, const Wide& w, const Acc& c) { return mfma16(x, w, c); }
};
template <>
struct Rows<kRowE4m3> : Rows<kRowBf16> {
  typedef uint2 Op;
  static constexpr int kBytes = 1;
  static __device__ __forceinline__ Op load(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t s) {
    return buf_load8(rs, at, s);
  }
  static __device__ __forceinline__ Wide widen(const Op& x) {
    return Wide{bf16_of_e4m3<false>(x.x, 1.f), bf16_of_e4m3<true>(x.x, 1.f), bf16_of_e4m3<false>(x.y, 1.f),
                bf16_of_e4m3<true>(x.y, 1.f)};
  }
};
template <>
struct Rows<kRowI8> {
  typedef uint2 Op;
  typedef uint2 Wide;
  typedef i32x4_t Acc;
  static constexpr int kBytes = 1;
  static __device__ __forceinline__ Op load(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t s) {
    return buf_load8(rs, at, s);
  }
  static __device__ __forceinline__ Wide widen(const Op& x) { return x; }
  static __device__ __forceinline__ Wide codes(uint32_t w) { return Wide{w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu}; }
  static __device__ __forceinline__ Wide minus(bool eight) {
    const uint32_t v = eight ? 0xF8F8F8F8u : 0xFFFFFFFFu;
    return Wide{v, v};
  }
  static __device__ __forceinline__ Acc mma(const Wide& x, const Wide& w, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, x), __builtin_bit_cast(long, w), c, 0, 0, 0);
  }
};

// v of lane 16 j + (lane & 15) in every lane, for a v that differs between the four
// lane rows (GP = 4) or the two lane halves (GP = 2): j = 0 .. GP - 1.
template <int GP>
__device__ __forceinline__ void spread(uint32_t v, uint32_t (&o)[GP]) {
  if constexpr (GP == 1) {
    o[0] = v;
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    if constexpr (GP == 2) {
      o[0] = h[0], o[1] = h[1];
    } else {
      const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
      const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
      o[0] = a[0], o[1] = a[1], o[2] = b[0], o[3] = b[1];
    }
  }
}

// TB: 16-row blocks of x; R: tiles a workgroup; W: waves; D: chunks in flight; G: group.
template <int XT, int TB, int R, int W, int D, int G, bool ZERO>
__global__ __launch_bounds__(W * 64) void w4_matvec_kernel(int64_t T, int K, const uint8_t* __restrict__ x,
                                                           const float* __restrict__ x_scale, const W4Table tab,
                                                           int t_blocks, bool y_bf16) {
  using X = Rows<XT>;
  using Op = typename X::Op;
  using Acc = typename X::Acc;
  constexpr int GP = 128 / G;
  __shared__ float red[W][R * TB * 4][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x % t_blocks) * (16 * TB);
  int group = blockIdx.x / t_blocks, p = 0;
  while (group >= tab.group_end[p]) ++p;
  if (p > 0) group -= tab.group_end[p - 1];
  const int N = tab.N[p], nt = (N + 15) / 16, kt = (K + 127) / 128, kg = K / G;
  // Buffer resources: one per tile, so every load's row offset is a lane constant and its
  // chunk a scalar. No load leaves its operand (none relies on the range check).
  __amdgpu_buffer_rsrc_t code_rs[R], scale_rs[R], zero_rs[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t tile = min(group * R + r, nt - 1);  // a tile past the end reads the last one
    code_rs[r] = make_rsrc(tab.codes[p] + tile * kt * 1024, kt * 1024);
    scale_rs[r] = make_rsrc(tab.scales[p] + tile * kg * 16, kg * 32);
    if constexpr (ZERO) zero_rs[r] = make_rsrc(tab.zeros[p] + tile * kg * 16, kg * 16);
  }
  // the block's rows of x; a row past T reads the last one (its sums are not stored)
  const int rows = static_cast<int>(min(T - t0, static_cast<int64_t>(16 * TB)));
  const auto x_rs = make_rsrc(x + t0 * K * X::kBytes, static_cast<uint32_t>(rows) * K * X::kBytes);
  uint32_t x_at[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) x_at[b] = (static_cast<uint32_t>(min(16 * b + l16, rows - 1)) * K + 8 * g) * X::kBytes;
  // the lane's group of a chunk; where only the first half exists, a group of that
  const uint32_t group_at = (GP == 1 ? 0 : GP == 2 ? g >> 1 : g) * 16 + l16;
  const uint32_t group_at_half = (GP == 4 ? g & 1 : 0) * 16 + l16;

  struct Chunk {
    uint4 codes[R];
    uint32_t scale[R], zero[R];
    Op x[TB][4];
  };
  Chunk ring[D];
  const int nw = kt > wave ? (kt - wave + W - 1) / W : 0;  // chunks of this wave
  auto load = [&](int i, Chunk& c) {
    const int at = wave + W * i;
    const bool half = GP > 1 && at * 128 + 64 == K;  // (a group of 128 fills its chunk)
    const uint32_t ga = half ? group_at_half : group_at;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c.codes[r] = buf_load16(code_rs[r], lane * 16, at * 1024);
      c.scale[r] = buf_load2(scale_rs[r], ga * 2, at * (GP * 32));
      if constexpr (ZERO) c.zero[r] = buf_load1(zero_rs[r], ga, at * (GP * 16));
    }
    // (in place of a half that does not exist the first one is read; the step clears it)
    const uint32_t x0 = at * 128 * X::kBytes, x1 = x0 + (half ? 0 : 64 * X::kBytes);
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) c.x[b][q] = X::load(x_rs, x_at[b] + 32 * (q & 1) * X::kBytes, q < 2 ? x0 : x1);
  };

  float tot[R][TB][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) tot[r][b][j] = 0.f;
  const typename X::Wide minus = X::minus(!ZERO);
  auto step = [&](int i, Chunk& c) {
    if (GP > 1 && (wave + W * i) * 128 + 64 == K) {
#pragma unroll
      for (int b = 0; b < TB; ++b) c.x[b][2] = c.x[b][3] = Op{};
    }
    float s[R][GP], z[R][GP];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t v[GP];
      spread<GP>(c.scale[r] | (ZERO ? c.zero[r] << 16 : 0u), v);
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        s[r][j] = __uint_as_float(v[j] << 16);
        if constexpr (ZERO) z[r][j] = static_cast<float>(v[j] >> 16);
      }
    }
    Acc acc[R][TB], xs[TB];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool first = q * 32 % G == 0;
      typename X::Wide xq[TB];
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        xq[b] = X::widen(c.x[b][q]);
        xs[b] = X::mma(xq[b], minus, first ? Acc{} : xs[b]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t words[4] = {c.codes[r].x, c.codes[r].y, c.codes[r].z, c.codes[r].w};
        const typename X::Wide w = X::codes(words[q]);
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[r][b] = X::mma(xq[b], w, first ? Acc{} : acc[r][b]);
      }
      if ((q + 1) * 32 % G == 0) {
        const int j = q * 32 / G;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float u;
              if constexpr (ZERO)
                u = static_cast<float>(acc[r][b][e]) + z[r][j] * static_cast<float>(xs[b][e]);
              else
                u = static_cast<float>(acc[r][b][e] + xs[b][e]);
              tot[r][b][e] += s[r][j] * u;
            }
      }
    }
  };
  if (nw > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < nw) load(d, ring[d]);
    for (int i = 0; i < nw; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i + d < nw) step(i + d, ring[d]);
        if (i + d + D < nw) load(i + d + D, ring[d]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][(r * TB + b) * 4 + e][lane] = tot[r][b][e];
  __syncthreads();
  for (int o = threadIdx.x; o < R * TB * 256; o += W * 64) {
    const int e = o >> 6, ln = o & 63;
    const int64_t t = t0 + e / 4 % TB * 16 + 4 * (ln >> 4) + e % 4;
    const int n = (group * R + e / (4 * TB)) * 16 + (ln & 15);
    if (t >= T || n >= N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[w][e][ln];
    if (x_scale != nullptr) v *= x_scale[t];
    const int64_t at = t * N + n;
    if (y_bf16) static_cast<uint16_t*>(tab.y[p])[at] = to_bf16(v);
    else static_cast<float*>(tab.y[p])[at] = v;
  }
}

// One launch of the kernel <XT, TB, R, W, D> for the table's group size and zero points.
template <int XT, int TB, int R, int W, int D>
hipError_t run(int64_t T, int K, int group, const void* x, const float* x_scale, W4Table tab, bool y_bf16,
               hipStream_t stream) {
  int groups = 0;
  for (int p = 0; p < tab.n; ++p) {
    groups += ((tab.N[p] + 15) / 16 + R - 1) / R;
    tab.group_end[p] = groups;
  }
  const int t_blocks = static_cast<int>((T + 16 * TB - 1) / (16 * TB));
  const dim3 grid(static_cast<unsigned>(groups) * static_cast<unsigned>(t_blocks));
  const auto xb = static_cast<const uint8_t*>(x);
  auto go = [&](auto g, auto zero) {
    w4_matvec_kernel<XT, TB, R, W, D, decltype(g)::value, decltype(zero)::value>
        <<<grid, W * 64, 0, stream>>>(T, K, xb, x_scale, tab, t_blocks, y_bf16);
  };
  auto with = [&](auto zero) {
    if (group == 32) go(std::integral_constant<int, 32>{}, zero);
    else if (group == 64) go(std::integral_constant<int, 64>{}, zero);
    else go(std::integral_constant<int, 128>{}, zero);
  };
  if (tab.zeros[0] != nullptr) with(std::true_type{});
  else with(std::false_type{});
  return hipGetLastError();
}

template <int XT>
hipError_t pick(int64_t T, int K, int group, const void* x, const float* x_scale, const W4Table& tab, bool y_bf16,
                hipStream_t stream) {
  int tiles = 0;
  for (int p = 0; p < tab.n; ++p) tiles += (tab.N[p] + 15) / 16;
  if (T <= 16) {
    if (tiles <= 256) return run<XT, 1, 1, 16, 2>(T, K, group, x, x_scale, tab, y_bf16, stream);
    if (tiles <= 768) return run<XT, 1, 2, 8, 2>(T, K, group, x, x_scale, tab, y_bf16, stream);
    return run<XT, 1, 4, 8, 1>(T, K, group, x, x_scale, tab, y_bf16, stream);
  }
  if (T <= 32) return run<XT, 2, 4, 8, 1>(T, K, group, x, x_scale, tab, y_bf16, stream);
  return run<XT, 4, 4, 4, 1>(T, K, group, x, x_scale, tab, y_bf16, stream);
}

}  // namespace

hipError_t launch_w4_matvec(int64_t T, int K, int group, int x_type, const void* x, const float* x_scale,
                            const W4Table& tab, bool y_bf16, hipStream_t stream) {
  if (x_type == kRowBf16) return pick<kRowBf16>(T, K, group, x, x_scale, tab, y_bf16, stream);
  if (x_type == kRowE4m3) return pick<kRowE4m3>(T, K, group, x, x_scale, tab, y_bf16, stream);
  return pick<kRowI8>(T, K, group, x, x_scale, tab, y_bf16, stream);
}

}  // namespace lnf4
