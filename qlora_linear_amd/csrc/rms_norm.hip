// RMS norm with the residual's addition, 8-bit output and gradient (gfx950).
//
//     h = round(x + res), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w
//     dx = dh + rstd (g - n mean(g n)),  dw = sum_t dy n,  g = dy w, n = h rstd
//
// Bound by HBM: every operand is read once and every result written once. A row stays
// in registers between its reduction and its output: TPR threads hold it, NV 16-byte
// vectors each (thread i: vectors i, i + TPR, ...), so all loads of a row are in flight
// together. The 8-bit scale needs max |h w| rstd, which the same reduction finds. All
// statistics and sums are float32.
//
// Rows need not be 16-byte aligned (d of any size): vectors are loaded with the
// alignment of an element, which the hardware allows for global memory, and only the
// last, partial vector of a row goes element by element.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "norm_w4_launch.h"

namespace lnf4 {
namespace {

template <typename E>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
};

// 16 bytes with the alignment of their elements.
template <typename E>
struct Raw;
template <>
struct Raw<uint16_t> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Raw<float> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
typedef uint32_t raw8_t __attribute__((ext_vector_type(2), aligned(1)));

template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return to_bf16(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// A vector of a row as it lies in memory; elements past the row's end are zero.
template <typename E>
struct Held {
  uint32_t u[4];
};
template <typename E>
__device__ __forceinline__ Held<E> load_vec(const E* p, int left) {
  constexpr int kN = Vec<E>::kN;
  Held<E> o{{0u, 0u, 0u, 0u}};
  if (left >= kN) {
    const auto v = *reinterpret_cast<const typename Raw<E>::type*>(p);
    o.u[0] = v.x, o.u[1] = v.y, o.u[2] = v.z, o.u[3] = v.w;
  } else if (left > 0) {
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (j < left) {
        if constexpr (sizeof(E) == 4) o.u[j] = __float_as_uint(p[j]);
        else o.u[j / 2] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
      }
  }
  return o;
}
template <typename E>
__device__ __forceinline__ float elem(const Held<E>& v, int j) {
  if constexpr (sizeof(E) == 4) return __uint_as_float(v.u[j]);
  else return __uint_as_float((j & 1) ? (v.u[j / 2] & 0xFFFF0000u) : (v.u[j / 2] << 16));
}
template <typename E>
__device__ __forceinline__ Held<E> hold(const float (&f)[Vec<E>::kN]) {
  Held<E> o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(E) == 4) o.u[j] = __float_as_uint(f[j]);
    else o.u[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
  }
  return o;
}
template <typename E>
__device__ __forceinline__ void store_vec(E* p, int left, const Held<E>& v) {
  constexpr int kN = Vec<E>::kN;
  if (left >= kN) {
    *reinterpret_cast<typename Raw<E>::type*>(p) = typename Raw<E>::type{v.u[0], v.u[1], v.u[2], v.u[3]};
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (j < left) p[j] = from_f32<E>(elem(v, j));
  }
}

// 8-bit levels of four values (byte j = value j); |v| is at most the format's largest
// up to a float32 rounding.
template <int OUT>
__device__ __forceinline__ uint32_t levels4(const float* v) {
  if constexpr (OUT == kRowE4m3) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true));
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w |= (static_cast<uint32_t>(static_cast<int>(__builtin_rintf(v[j]))) & 0xFFu) << (8 * j);
    return w;
  }
}

// A vector of values as levels at p, `left` of the row left from there.
template <int OUT, int N>
__device__ __forceinline__ void store_levels(uint8_t* p, int left, const float (&f)[N]) {
  uint32_t lv[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) lv[j] = levels4<OUT>(f + 4 * j);
  if (left >= N) {
    if constexpr (N == 8) *reinterpret_cast<raw8_t*>(p) = raw8_t{lv[0], lv[1]};
    else __builtin_memcpy(p, lv, 4);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < left) p[j] = static_cast<uint8_t>(lv[j / 4] >> (8 * (j & 3)));
  }
}

// The values as packed, not as unpacked for the reduction, stay in registers after it
// (the compiler would keep both: twice the registers, half the rows in flight).
template <typename E>
__device__ __forceinline__ void repack(Held<E>& v) {
  if constexpr (sizeof(E) == 2) asm volatile("" : "+v"(v.u[0]), "+v"(v.u[1]), "+v"(v.u[2]), "+v"(v.u[3]));
}

// Sum and maximum over the TPR threads of a row, the same bits in each. The threads of
// a row are consecutive; red has a pair per wave of the workgroup.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& s, float& m, float2* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    m = fmaxf(m, __shfl_xor(m, o));
  }
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = make_float2(s, m);
    __syncthreads();
    const float2* r = red + wave / kWaves * kWaves;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      s += r[i].x;
      m = fmaxf(m, r[i].y);
    }
  }
}

// Workgroups of one row (or a few) each: a launch has fewer than 2^32 threads along x, so
// many rows spread over y as well.
constexpr int64_t kGridX = 1 << 20;
dim3 row_grid(int64_t n) {
  return n <= kGridX ? dim3(static_cast<unsigned>(n))
                     : dim3(static_cast<unsigned>(kGridX), static_cast<unsigned>((n + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t row_block() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }

// A row's 8-bit scale and what turns its values into levels. With m = max |h w|, which the
// reduction of the sum of squares finds beside it, the scale is m rstd / top level and the level
// of y is the nearest to h w (top level / m): rstd cancels. The factor is held in two parts, so
// that the quotient is off by its last rounding only; with bf16 rows, whose h w is exact, a
// quotient in the middle of two levels (1 in 10^4, as bf16 quotients have few bits) comes out
// as that and goes to the even one.
// h w may leave float32's normal range where y does not: near its ends (and in rows of zeros)
// the largest y is found again, from y, and levels are y times a reciprocal of it.
constexpr float kTiny = 0x1p-100f, kUp = 0x1p48f, kHuge = 0x1p127f;
__device__ __forceinline__ bool far_row(float m, float top) {
  return __builtin_expect(!(fminf(m, top) >= kTiny && top <= kHuge), 0);
}
struct Levels {
  float scale, first, inv, low;  // level = f inv + f low of f = h first w
  template <int N>
  __device__ __forceinline__ void apply(float (&f)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = __builtin_fmaf(f[j], inv, f[j] * low);
  }
};
template <int OUT>
constexpr float kTopLevel = OUT == kRowE4m3 ? 448.f : 127.f;
template <int OUT>
__device__ __forceinline__ Levels row_levels(float m, float top) {
  constexpr float kTop = kTopLevel<OUT>;
  const float inv = kTop / m;
  return Levels{top / kTop, 1.f, inv, __builtin_fmaf(-inv, m, kTop) * (inv * (1.f / kTop))};
}
// The same from top = max |y|, any. Rows so small that the reciprocal would overflow are scaled
// up first (exactly; rstd, at most 2^75 for the least eps, does not overflow by it). A subnormal scale has few bits: it is rounded up, so that no level passes
// the top one, and the levels are those of the scale as it is then.
template <int OUT>
__device__ __forceinline__ Levels far_levels(float top, float rstd) {
  constexpr float kTop = kTopLevel<OUT>;
  const float up = top < kTiny ? kUp : 1.f;
  Levels l{top / kTop, rstd * up, 0.f, 0.f};
  float over = kTop, under = top * up;
  if (l.scale < 0x1p-126f) {
    if (l.scale * kTop < top) l.scale = __uint_as_float(__float_as_uint(l.scale) + 1u);
    over = 1.f, under = l.scale * kUp;
  }
  if (l.scale > 0.f) l.inv = over / under;  // (not of zeros, not NaN)
  return l;
}

// ---- forward ---------------------------------------------------------------------------
// 8192 x 4096 bf16 with residual 44 us, 6.1 TB/s; 1 x 4096 to E4M3 3 us, a launch and two
// latencies. (Times here are over three sets of rows in turn, more than the memory-side
// cache holds where the sizes are large.)
template <typename E, int OUT, int TPR, int NV>
__global__ __launch_bounds__((TPR < 256 ? 256 : TPR)) void rmsnorm_fwd_kernel(
    int64_t T, int d, float eps, const E* __restrict__ x, const E* __restrict__ res, const E* __restrict__ w,
    E* __restrict__ h, void* __restrict__ y, float* __restrict__ q_scale, float* __restrict__ rstd_out) {
  constexpr int kN = Vec<E>::kN, kBlock = TPR < 256 ? 256 : TPR;
  static_assert(TPR == 64 || TPR == kBlock, "a barrier runs in workgroups of one row only");
  constexpr bool kQuant = OUT == kRowE4m3 || OUT == kRowI8;
  __shared__ float2 red[kBlock / 64];
  const int64_t t = row_block() * (kBlock / TPR) + threadIdx.x / TPR;
  const int i0 = threadIdx.x % TPR;
  if (t >= T) return;  // (whole rows; a workgroup with a barrier ahead has one row)
  const int64_t row = t * d;
  // (at 8 vectors a thread the weight is read a second time rather than kept)
  constexpr bool kKeep = NV <= 4;
  Held<E> hv[NV], wv[kKeep ? NV : 1];
  auto weight = [&](int v) {
    const int at = (i0 + v * TPR) * kN;
    return kKeep ? wv[kKeep ? v : 0] : load_vec(w + at, d - at);
  };
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (i0 + v * TPR) * kN;
    hv[v] = load_vec(x + row + at, d - at);
  }
  if (res != nullptr) {
    Held<E> rv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (i0 + v * TPR) * kN;
      rv[v] = load_vec(res + row + at, d - at);
    }
#pragma unroll
    for (int v = 0; kKeep && v < NV; ++v) {
      const int at = (i0 + v * TPR) * kN;
      wv[kKeep ? v : 0] = load_vec(w + at, d - at);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (i0 + v * TPR) * kN;
      float f[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) f[j] = elem(hv[v], j) + elem(rv[v], j);
      hv[v] = hold<E>(f);
      store_vec(h + row + at, d - at, hv[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; kKeep && v < NV; ++v) {
      const int at = (i0 + v * TPR) * kN;
      wv[kKeep ? v : 0] = load_vec(w + at, d - at);
    }
  }
  float s = 0.f, m = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    Held<E> wt{};
    if constexpr (kQuant) wt = weight(v);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const float f = elem(hv[v], j);
      s += f * f;
      if constexpr (kQuant) m = fmaxf(m, fabsf(f * elem(wt, j)));
    }
  }
  row_reduce<TPR>(s, m, red);
  const float rstd = 1.0f / __builtin_sqrtf(s / static_cast<float>(d) + eps);
  if (i0 == 0 && rstd_out != nullptr) rstd_out[t] = rstd;
  Levels to{};
  if constexpr (kQuant) {
    const float top = m * rstd;
    to = row_levels<OUT>(m, top);
    if (far_row(m, top)) {  // (the same in all threads of a row, and so of a workgroup with barriers)
      float unused = 0.f, far = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        Held<E> wt = weight(v);
        repack(hv[v]);
        repack(wt);
#pragma unroll
        for (int j = 0; j < kN; ++j) far = fmaxf(far, fabsf(elem(hv[v], j) * rstd * elem(wt, j)));
      }
      if constexpr (TPR > 64) __syncthreads();  // red has been read
      row_reduce<TPR>(unused, far, red);
      to = far_levels<OUT>(top == top ? far : top, rstd);
    }
    if (i0 == 0) q_scale[t] = to.scale;
  }
  const float first = kQuant ? to.first : rstd;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (i0 + v * TPR) * kN, left = d - at;
    Held<E> wt = weight(v);
    repack(hv[v]);
    repack(wt);
    float f[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) f[j] = elem(hv[v], j) * first * elem(wt, j);
    if constexpr (kQuant) {
      to.apply(f);
      store_levels<OUT>(static_cast<uint8_t*>(y) + row + at, left, f);
    } else if (left > 0) {
      store_vec(static_cast<E*>(y) + row + at, left, hold<E>(f));
    }
  }
}

// Rows wider than the registers of a workgroup hold: the row is read twice, the second
// time mostly from L2 (h is formed again from x and the residual). 512 x 40000 bf16 20 us,
// 4.2 TB/s.
constexpr int kLoop = 1024;
template <typename E, int OUT>
__global__ __launch_bounds__(kLoop) void rmsnorm_fwd_loop_kernel(int64_t T, int d, float eps, const E* __restrict__ x,
                                                                 const E* __restrict__ res,
                                                                 const E* __restrict__ w, E* __restrict__ h,
                                                                 void* __restrict__ y,
                                                                 float* __restrict__ q_scale,
                                                                 float* __restrict__ rstd_out) {
  __shared__ float2 red[kLoop / 64];
  const int64_t t = row_block(), row = t * d;
  if (t >= T) return;
  constexpr int kN = Vec<E>::kN;
  constexpr bool kQuant = OUT == kRowE4m3 || OUT == kRowI8;
  auto h_at = [&](int at) {
    Held<E> v = load_vec(x + row + at, d - at);
    if (res == nullptr) return v;
    const Held<E> r = load_vec(res + row + at, d - at);
    float f[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) f[j] = elem(v, j) + elem(r, j);
    return hold<E>(f);
  };
  float s = 0.f, m = 0.f;
  for (int at = threadIdx.x * kN; at < d; at += kLoop * kN) {
    const Held<E> v = h_at(at), wt = load_vec(w + at, d - at);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const float f = elem(v, j);
      s += f * f;
      m = fmaxf(m, fabsf(f * elem(wt, j)));
    }
  }
  row_reduce<kLoop>(s, m, red);
  const float rstd = 1.0f / __builtin_sqrtf(s / static_cast<float>(d) + eps);
  Levels to{};
  if constexpr (kQuant) {
    const float top = m * rstd;
    to = row_levels<OUT>(m, top);
    if (far_row(m, top)) {
      float unused = 0.f, far = 0.f;
      for (int at = threadIdx.x * kN; at < d; at += kLoop * kN) {
        const Held<E> v = h_at(at), wt = load_vec(w + at, d - at);
#pragma unroll
        for (int j = 0; j < kN; ++j) far = fmaxf(far, fabsf(elem(v, j) * rstd * elem(wt, j)));
      }
      __syncthreads();  // red has been read
      row_reduce<kLoop>(unused, far, red);
      to = far_levels<OUT>(top == top ? far : top, rstd);
    }
  }
  const float first = kQuant ? to.first : rstd;
  for (int at = threadIdx.x * kN; at < d; at += kLoop * kN) {
    const int left = d - at;
    const Held<E> v = h_at(at), wt = load_vec(w + at, left);
    if (res != nullptr) store_vec(h + row + at, left, v);
    float f[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) f[j] = elem(v, j) * first * elem(wt, j);
    if constexpr (kQuant) {
      to.apply(f);
      store_levels<OUT>(static_cast<uint8_t*>(y) + row + at, left, f);
    } else {
      store_vec(static_cast<E*>(y) + row + at, left, hold<E>(f));
    }
  }
  if (threadIdx.x == 0) {
    if (rstd_out != nullptr) rstd_out[t] = rstd;
    if constexpr (kQuant) q_scale[t] = to.scale;
  }
}

// ---- backward --------------------------------------------------------------------------
// BLOCK / TPR rows at a time (the workgroup's slots), the workgroup strides over all
// rows; with DW every thread also sums dy n of its columns over its rows, the slots'
// sums are added in LDS in a fixed order, and part[workgroup][d] holds the result.
// 8192 x 4096 bf16 with dh and dw 53 us, 5.1 TB/s; 333 x 1001 float32 without dw 3.5 us.
template <typename E, int TPR, int NV, int BLOCK, bool DW>
__global__ __launch_bounds__(BLOCK) void rmsnorm_bwd_kernel(int64_t T, int d, const E* __restrict__ dy,
                                                            const E* __restrict__ dh, const E* __restrict__ h,
                                                            const E* __restrict__ w,
                                                            const float* __restrict__ rstd_in,
                                                            E* __restrict__ dx, float* __restrict__ part) {
  constexpr int kN = Vec<E>::kN, kSlots = BLOCK / TPR;
  static_assert(TPR % 64 == 0 && BLOCK % TPR == 0, "whole waves a row, whole rows a workgroup");
  __shared__ float2 red[BLOCK / 64];
  const int i0 = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  Held<E> wv[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (i0 + v * TPR) * kN;
    wv[v] = load_vec(w + at, d - at);
  }
  float acc[DW ? NV * kN : 1];
#pragma unroll
  for (int j = 0; j < (DW ? NV * kN : 1); ++j) acc[j] = 0.f;
  // every slot runs as often as the workgroup's first (barriers); one past the end has
  // vectors of length 0: it loads zeros and stores nothing
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kSlots; t0 < T; t0 += static_cast<int64_t>(gridDim.x) * kSlots) {
    const bool ok = t0 + slot < T;
    const int64_t t = ok ? t0 + slot : t0;
    const int64_t row = t * d;
    const int dd = ok ? d : 0;
    Held<E> hv[NV], gv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (i0 + v * TPR) * kN;
      hv[v] = load_vec(h + row + at, dd - at);
      gv[v] = load_vec(dy + row + at, dd - at);
    }
    const float rstd = rstd_in[t];
    float s = 0.f, unused = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Held<E> wt = wv[v];
      repack(wt);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const float n = elem(hv[v], j) * rstd, g = elem(gv[v], j);
        if constexpr (DW) acc[v * kN + j] += g * n;
        s += g * elem(wt, j) * n;
      }
    }
    if constexpr (TPR > 64) __syncthreads();  // the last row's red has been read
    row_reduce<TPR>(s, unused, red);
    const float c = s / static_cast<float>(d);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (i0 + v * TPR) * kN, left = dd - at;
      repack(hv[v]);
      repack(gv[v]);
      Held<E> wt = wv[v];
      repack(wt);
      float f[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const float n = elem(hv[v], j) * rstd;
        f[j] = rstd * (elem(gv[v], j) * elem(wt, j) - n * c);
      }
      if (dh != nullptr) {
        const Held<E> e = load_vec(dh + row + at, left);
#pragma unroll
        for (int j = 0; j < kN; ++j) f[j] += elem(e, j);
      }
      if (left > 0) store_vec(dx + row + at, left, hold<E>(f));
    }
  }
  if constexpr (DW) {
    float* out = part + static_cast<int64_t>(blockIdx.x) * d;
    if constexpr (kSlots > 1) {
      __shared__ float sum[NV * TPR * kN];  // [v][j][thread]: lanes side by side, no bank conflicts
      for (int k = 0; k < kSlots; ++k) {
        if (slot == k) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              float* p = sum + (v * kN + j) * TPR + i0;
              *p = k == 0 ? acc[v * kN + j] : *p + acc[v * kN + j];
            }
        }
        __syncthreads();
      }
      for (int i = threadIdx.x; i < d; i += BLOCK) {
        const int vec = i / kN;
        out[i] = sum[(vec / TPR * kN + i % kN) * TPR + vec % TPR];
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const int i = (i0 + v * TPR) * kN + j;
          if (i < d) out[i] = acc[v * kN + j];
        }
    }
  }
}

// Rows wider than the registers hold: read twice (512 x 40000 bf16 30 us, 4.1 TB/s).
template <typename E>
__global__ __launch_bounds__(kLoop) void rmsnorm_bwd_loop_kernel(int64_t T, int d, const E* __restrict__ dy,
                                                                 const E* __restrict__ dh,
                                                                 const E* __restrict__ h, const E* __restrict__ w,
                                                                 const float* __restrict__ rstd_in,
                                                                 E* __restrict__ dx) {
  __shared__ float2 red[kLoop / 64];
  const int64_t t = row_block(), row = t * d;
  if (t >= T) return;
  const float rstd = rstd_in[t];
  float s = 0.f, unused = 0.f;
  constexpr int kN = Vec<E>::kN;
  for (int at = threadIdx.x * kN; at < d; at += kLoop * kN) {
    const Held<E> g = load_vec(dy + row + at, d - at), v = load_vec(h + row + at, d - at), wt = load_vec(w + at, d - at);
#pragma unroll
    for (int j = 0; j < kN; ++j) s += elem(g, j) * elem(wt, j) * (elem(v, j) * rstd);
  }
  row_reduce<kLoop>(s, unused, red);
  const float c = s / static_cast<float>(d);
  for (int at = threadIdx.x * kN; at < d; at += kLoop * kN) {
    const int left = d - at;
    const Held<E> g = load_vec(dy + row + at, left), v = load_vec(h + row + at, left), wt = load_vec(w + at, left);
    float f[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) f[j] = rstd * (elem(g, j) * elem(wt, j) - elem(v, j) * rstd * c);
    if (dh != nullptr) {
      const Held<E> e = load_vec(dh + row + at, left);
#pragma unroll
      for (int j = 0; j < kN; ++j) f[j] += elem(e, j);
    }
    store_vec(dx + row + at, left, hold<E>(f));
  }
}

// part[b][i] = sum of dy n over the rows b, b + blocks, ... of column i; one vector of
// columns a thread. With the join 25 us for 512 x 40000 bf16, 3.2 TB/s.
template <typename E>
__global__ __launch_bounds__(256) void rmsnorm_dw_part_kernel(int64_t T, int d, const E* __restrict__ dy,
                                                              const E* __restrict__ h,
                                                              const float* __restrict__ rstd,
                                                              float* __restrict__ part) {
  constexpr int kN = Vec<E>::kN;
  const int at = (blockIdx.x * 256 + threadIdx.x) * kN;
  if (at >= d) return;
  float s[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) s[j] = 0.f;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const Held<E> g = load_vec(dy + t * d + at, d - at), v = load_vec(h + t * d + at, d - at);
    const float r = rstd[t];
#pragma unroll
    for (int j = 0; j < kN; ++j) s[j] += elem(g, j) * (elem(v, j) * r);
  }
  float* const out = part + static_cast<int64_t>(blockIdx.y) * d + at;
#pragma unroll
  for (int j = 0; j < kN; ++j)
    if (at + j < d) out[j] = s[j];
}

// dw[i] = sum over blocks of part[block][i]: 32 columns a workgroup, 32 threads a
// column over the blocks, joined in LDS in a fixed order. 512 x 4096 4.8 us, mostly latency.
template <typename E>
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(int blocks, int d, const float* __restrict__ part,
                                                          E* __restrict__ dw) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5, i = blockIdx.x * 32 + c;
  float s = 0.f;
  if (i < d) {
    int b = k;
    for (; b + 7 * 32 < blocks; b += 8 * 32) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = part[static_cast<int64_t>(b + 32 * j) * d + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * d + i];
  }
  red[k][c] = s;
  __syncthreads();
  if (k == 0 && i < d) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) v += red[j][c];
    dw[i] = from_f32<E>(v);
  }
}

template <typename E>
__global__ __launch_bounds__(256) void zero_kernel(E* __restrict__ p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = E(0);
}

// Threads and vectors a thread of a row of `vecs` vectors: up to two vectors a thread, from
// one wave, 4 or 16, as long as 16 waves of two hold the row. Measured in one sweep of
// launches back to back, each with its gap (bf16 forward with residual, us): 8192 x 4096 at 256 threads of two 47, 1024 of one 49, 64 of eight 55; 1 x
// 4096 at 256 of two 2.9, 64 of eight 5.3; 8192 x 1024 at 64 of two 11.1, 256 of one 12.9;
// but 400 x 1024 at 256 of one 2.9, 64 of two 4.2 (few rows leave the GPU idle whatever
// is chosen, and one vector a thread has the shorter way from its loads to its stores).
// most: the most vectors of 1024 threads.
constexpr int kFewRows = 512;
struct RowShape {
  int tpr, nv;  // tpr 0: does not fit
};
RowShape row_shape(int64_t T, int64_t vecs, int most) {
  if (vecs <= 64) return {64, 1};
  if (vecs <= 128 && T > kFewRows) return {64, 2};
  if (vecs <= 256) return {256, 1};
  if (vecs <= 512) return {256, 2};
  for (int nv = 1; nv <= most; nv *= 2)
    if (vecs <= 1024 * nv) return {1024, nv};
  return {0, 0};
}
// go(threads, vectors) of a shape, as compile-time constants.
template <int MOST, class Go>
void with_shape(const RowShape& sh, Go&& go) {
  using std::integral_constant;
  const integral_constant<int, 64> t64;
  const integral_constant<int, 256> t256;
  const integral_constant<int, 1024> t1024;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  if (sh.tpr == 64) sh.nv == 1 ? go(t64, one) : go(t64, two);
  else if (sh.tpr == 256) sh.nv == 1 ? go(t256, one) : go(t256, two);
  else if (sh.nv == 1) go(t1024, one);
  else if (sh.nv == 2) go(t1024, two);
  else if constexpr (MOST >= 4) {
    if (sh.nv == 4) go(t1024, integral_constant<int, 4>{});
    else if constexpr (MOST >= 8) go(t1024, integral_constant<int, 8>{});
  }
}

template <typename E, int OUT>
hipError_t fwd(int64_t T, int d, float eps, const void* xv, const void* rv, const void* wv, void* hv, void* y,
               float* q_scale, float* rstd, hipStream_t stream) {
  const auto x = static_cast<const E*>(xv), res = static_cast<const E*>(rv), w = static_cast<const E*>(wv);
  const auto h = static_cast<E*>(hv);
  // Up to 32768 values of a row in registers (1 x 28672 float32 5.3 us, 2048 x 20000 68, with the
  // residual 129; the loop 7.4, 84 and 163), but 16384 of bf16 rows with levels, whose arithmetic
  // does not fit beside more of them (78 x 20856 6.8 us, 2048 x 20000 48; the loop 5.9 and 34).
  constexpr int kMost = (Vec<E>::kN == 8 && (OUT == kRowE4m3 || OUT == kRowI8) ? 16 : 32) / Vec<E>::kN;
  const RowShape sh = row_shape(T, (d + Vec<E>::kN - 1) / Vec<E>::kN, kMost);
  if (sh.tpr == 0)
    rmsnorm_fwd_loop_kernel<E, OUT><<<row_grid(T), kLoop, 0, stream>>>(T, d, eps, x, res, w, h, y, q_scale, rstd);
  else
    with_shape<kMost>(sh, [&](auto tpr, auto nv) {
      constexpr int kTpr = decltype(tpr)::value, kNv = decltype(nv)::value, kRows = kTpr < 256 ? 256 / kTpr : 1;
      rmsnorm_fwd_kernel<E, OUT, kTpr, kNv><<<row_grid((T + kRows - 1) / kRows), kTpr * kRows, 0, stream>>>(
          T, d, eps, x, res, w, h, y, q_scale, rstd);
    });
  return hipGetLastError();
}

template <typename E>
hipError_t fwd_out(int64_t T, int d, float eps, const void* x, const void* res, const void* w, void* h, int out,
                   void* y, float* q_scale, float* rstd, hipStream_t stream) {
  if (out == kRowE4m3) return fwd<E, kRowE4m3>(T, d, eps, x, res, w, h, y, q_scale, rstd, stream);
  if (out == kRowI8) return fwd<E, kRowI8>(T, d, eps, x, res, w, h, y, q_scale, rstd, stream);
  return fwd<E, kRowF32>(T, d, eps, x, res, w, h, y, q_scale, rstd, stream);  // E itself
}

// Workgroups of the backward, each with one row of float32 partial sums of dw: two or
// more a CU, few enough that the partial sums stay small beside the rows.
constexpr int kBwdBlocks = 512;
constexpr int kBwdThreads = 512;
int bwd_blocks(int64_t T) { return static_cast<int>(T < kBwdBlocks ? T : kBwdBlocks); }

template <typename E>
hipError_t bwd(int64_t T, int d, const void* dyv, const void* dhv, const void* hv, const void* wv, const float* rstd,
               void* dxv, void* dwv, void* workspace, hipStream_t stream) {
  const auto dy = static_cast<const E*>(dyv), dh = static_cast<const E*>(dhv), h = static_cast<const E*>(hv);
  const auto w = static_cast<const E*>(wv);
  const auto dx = static_cast<E*>(dxv), dw = static_cast<E*>(dwv);
  const auto part = static_cast<float*>(workspace);
  // dw's sums take a register an element: 16 elements a thread leave four waves a SIMD. Wider
  // rows are read twice, and have their dw in a pass of its own (78 x 20856 without dw 5.8 us,
  // in registers 6.9; many rows about alike, 2048 x 20000 with dh 62 and 63, float32 126 and 129;
  // with the sums too they spill).
  constexpr int kMost = 16 / Vec<E>::kN;
  const int64_t vecs = (d + Vec<E>::kN - 1) / Vec<E>::kN;
  const RowShape sh = row_shape(T, vecs, kMost);
  const bool both = dw != nullptr && sh.tpr != 0;
  int blocks = bwd_blocks(T);
  if (sh.tpr == 0)
    rmsnorm_bwd_loop_kernel<E><<<row_grid(T), kLoop, 0, stream>>>(T, d, dy, dh, h, w, rstd, dx);
  else
    with_shape<kMost>(sh, [&](auto tpr, auto nv) {
      constexpr int kTpr = decltype(tpr)::value, kNv = decltype(nv)::value;
      constexpr int kBlock = kTpr < kBwdThreads ? kBwdThreads : kTpr, kSlots = kBlock / kTpr;
      const int n = static_cast<int>(std::min<int64_t>((T + kSlots - 1) / kSlots, blocks));
      if (both) {
        blocks = n;
        rmsnorm_bwd_kernel<E, kTpr, kNv, kBlock, true><<<dim3(n), kBlock, 0, stream>>>(T, d, dy, dh, h, w, rstd, dx, part);
      } else {
        rmsnorm_bwd_kernel<E, kTpr, kNv, kBlock, false><<<dim3(n), kBlock, 0, stream>>>(T, d, dy, dh, h, w, rstd, dx, part);
      }
    });
  if (dw != nullptr && !both) {
    blocks = std::min(blocks, 64);
    rmsnorm_dw_part_kernel<E><<<dim3(static_cast<unsigned>((vecs + 255) / 256), blocks), 256, 0, stream>>>(T, d, dy, h, rstd, part);
  }
  if (dw != nullptr) rmsnorm_dw_kernel<E><<<dim3((d + 31) / 32), 1024, 0, stream>>>(blocks, d, part, dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(int64_t T, int d, int dtype, float eps, const void* x, const void* residual,
                              const void* w, void* h, int out, void* y, float* q_scale, float* rstd,
                              hipStream_t stream) {
  return dtype == kRowBf16 ? fwd_out<uint16_t>(T, d, eps, x, residual, w, h, out, y, q_scale, rstd, stream)
                           : fwd_out<float>(T, d, eps, x, residual, w, h, out, y, q_scale, rstd, stream);
}

size_t rmsnorm_bwd_bytes(int64_t T, int64_t d) {
  return (static_cast<size_t>(bwd_blocks(T)) * d * 4 + 255) / 256 * 256;
}

hipError_t launch_rmsnorm_bwd(int64_t T, int d, int dtype, const void* dy, const void* dh, const void* h,
                              const void* w, const float* rstd, void* dx, void* dw, void* workspace,
                              hipStream_t stream) {
  return dtype == kRowBf16 ? bwd<uint16_t>(T, d, dy, dh, h, w, rstd, dx, dw, workspace, stream)
                           : bwd<float>(T, d, dy, dh, h, w, rstd, dx, dw, workspace, stream);
}

hipError_t launch_zero(void* p, int64_t n, int dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  if (dtype == kRowBf16) zero_kernel<<<grid, 256, 0, stream>>>(static_cast<uint16_t*>(p), n);
  else zero_kernel<<<grid, 256, 0, stream>>>(static_cast<float*>(p), n);
  return hipGetLastError();
}

}  // namespace lnf4
