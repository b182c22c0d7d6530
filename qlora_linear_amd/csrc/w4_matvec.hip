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
//   * codes become operands in registers. bf16 and E4M3 rows: bf16 by the E4M3 conversion
//     with scale 2^9, as a byte c of 0 .. 15 is c 2^-9 in E4M3, whose subnormals and first
//     binade are equidistant (7 instructions per eight codes). E4M3 rows widen to bf16
//     (exactly) as well: the E4M3 matrix instruction would take the nibbles as they are, but
//     its sums lose bits (single products of 32 columns 5e-6 to 1.4e-5 off, bf16 ones below
//     1e-8), as do f16 products with subnormal codes. int8 rows: bytes c - z (5 and 7);
//   * the matrix instruction multiplies codes, not weights: the group's scale, and with
//     bf16 codes the zero point, are applied to its 16 x 16 sums. That zero point needs
//     sum x over the group, one more instruction with a constant operand, shared by the R
//     tiles; int8 rows do without (5120 -> 32003 at 64 rows, groups of 64: 44 -> 38 us);
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
  static constexpr bool kBiased = true;  // codes are multiplied as they are, 0 .. 15
  static __device__ __forceinline__ Op load(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t s) {
    return buf_load16(rs, at, s);
  }
  static __device__ __forceinline__ Wide widen(const Op& x) { return x; }
  template <bool ZERO>
  static __device__ __forceinline__ Wide codes(uint32_t w, uint32_t) {
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
  // Codes less their zero point (z in every byte of zeros), as two's complement bytes: with
  // bit 7 set first no byte borrows from the next. Without zero points 16 (c - 8), which is
  // the nibble in the byte's upper half with the sign turned.
  static constexpr bool kBiased = false;
  template <bool ZERO>
  static __device__ __forceinline__ Wide codes(uint32_t w, uint32_t zeros) {
    constexpr uint32_t kSign = 0x80808080u;
    if constexpr (!ZERO) return Wide{((w << 4) & 0xF0F0F0F0u) ^ kSign, (w & 0xF0F0F0F0u) ^ kSign};
    const uint32_t lo = (w & 0x0F0F0F0Fu) | kSign, hi = ((w >> 4) & 0x0F0F0F0Fu) | kSign;
    return Wide{(lo - zeros) ^ kSign, (hi - zeros) ^ kSign};
  }
  static __device__ __forceinline__ Acc mma(const Wide& x, const Wide& w, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, x), __builtin_bit_cast(long, w), c, 0, 0, 0);
  }
};

// Nothing is moved across: the counted waits rely on the order that loads are issued in.
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

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

// Scales and zero points of a chunk's groups from the lane's raw ones, the zero points
// as floats or, where they are taken off the codes, in every byte of a word.
template <class X, int GP, bool ZERO>
__device__ __forceinline__ void group_factors(uint32_t scale, uint32_t zero, float (&s)[GP], uint32_t (&z)[GP]) {
  uint32_t v[GP];
  spread<GP>(scale | zero << 16, v);
#pragma unroll
  for (int j = 0; j < GP; ++j) {
    s[j] = __uint_as_float(v[j] << 16);
    if (X::kBiased) z[j] = ZERO ? __float_as_uint(static_cast<float>(v[j] >> 16)) : 0u;
    else if (ZERO) z[j] = (v[j] >> 16) * 0x01010101u;
    else s[j] *= 0.0625f, z[j] = 0u;
  }
}

// tot += s (acc + z xs) of a 16 x 16 block, xs holding -sum x (without zero points
// -8 sum x, and z is not used); tot += s acc where the codes have no bias.
template <class X, bool ZERO>
__device__ __forceinline__ void add_group(const typename X::Acc& acc, const typename X::Acc& xs, float s, uint32_t z,
                                          float (&tot)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float u = static_cast<float>(acc[e]);
    if constexpr (X::kBiased) u = ZERO ? u + __uint_as_float(z) * xs[e] : u + xs[e];
    tot[e] += s * u;
  }
}

// Up to 16 rows of x. R: tiles a workgroup; W: waves; D: chunks in flight; G: group.
// 8192 -> 28672 at 1 row 26 us, 4.6 TB/s; 4096 -> 1024 4.4 us, a launch and the loads' latency.
template <int XT, int R, int W, int D, int G, bool ZERO>
__global__ __launch_bounds__(W * 64) void w4_matvec_kernel(int T, int K, const uint8_t* __restrict__ x,
                                                           const float* __restrict__ x_scale, const W4Table tab,
                                                           bool y_bf16) {
  using X = Rows<XT>;
  using Op = typename X::Op;
  using Acc = typename X::Acc;
  constexpr int GP = 128 / G;
  __shared__ float red[W][R * 4][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int group = blockIdx.x, p = 0;
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
  // (a row past T reads the last one; its sums are not stored)
  const auto x_rs = make_rsrc(x, static_cast<uint32_t>(T) * K * X::kBytes);
  const uint32_t x_at = (static_cast<uint32_t>(min(l16, T - 1)) * K + 8 * g) * X::kBytes;
  // the lane's group of a chunk; where only the first half exists, a group of that
  const uint32_t group_at = (GP == 1 ? 0 : GP == 2 ? g >> 1 : g) * 16 + l16;
  const uint32_t group_at_half = (GP == 4 ? g & 1 : 0) * 16 + l16;

  struct Chunk {
    uint4 codes[R];
    uint32_t scale[R], zero[R];
    Op x[4];
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
    // (in place of a half that does not exist the first one is read; its scales become 0)
    const uint32_t x0 = at * 128 * X::kBytes, x1 = x0 + (half ? 0 : 64 * X::kBytes);
#pragma unroll
    for (int q = 0; q < 4; ++q) c.x[q] = X::load(x_rs, x_at + 32 * (q & 1) * X::kBytes, q < 2 ? x0 : x1);
  };

  float tot[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) tot[r][e] = 0.f;
  typename X::Wide minus{};
  if constexpr (X::kBiased) minus = X::minus(!ZERO);
  auto step = [&](int i, const Chunk& c) {
    const bool absent = GP > 1 && (wave + W * i) * 128 + 64 == K && g >= 2;  // the lane's group
    float s[R][GP];
    uint32_t z[R][GP];
#pragma unroll
    for (int r = 0; r < R; ++r) group_factors<X, GP, ZERO>(absent ? 0u : c.scale[r], ZERO ? c.zero[r] : 0u, s[r], z[r]);
    Acc acc[R], xs;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool first = q * 32 % G == 0;
      const typename X::Wide xq = X::widen(c.x[q]);
      if constexpr (X::kBiased) xs = X::mma(xq, minus, first ? Acc{} : xs);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t words[4] = {c.codes[r].x, c.codes[r].y, c.codes[r].z, c.codes[r].w};
        acc[r] = X::mma(xq, X::template codes<ZERO>(words[q], z[r][q * 32 / G]), first ? Acc{} : acc[r]);
      }
      if ((q + 1) * 32 % G == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) add_group<X, ZERO>(acc[r], xs, s[r][q * 32 / G], z[r][q * 32 / G], tot[r]);
      }
    }
  };
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
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][r * 4 + e][lane] = tot[r][e];
  __syncthreads();
  for (int o = threadIdx.x; o < R * 256; o += W * 64) {
    const int e = o >> 6, ln = o & 63;
    const int t = 4 * (ln >> 4) + e % 4;
    const int n = (group * R + e / 4) * 16 + (ln & 15);
    if (t >= T || n >= N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[w][e][ln];
    if (x_scale != nullptr) v *= x_scale[t];
    const int64_t at = static_cast<int64_t>(t) * N + n;
    if (y_bf16) static_cast<uint16_t*>(tab.y[p])[at] = to_bf16(v);
    else static_cast<float*>(tab.y[p])[at] = v;
  }
}

// More rows of x: the x operands of a chunk, 16 TB rows, outweigh its codes, so the
// waves of a workgroup share them through LDS. RW x KW waves: each row wave owns R
// tiles, the KW waves of a row wave take the chunks of a step (KW chunks) in turn. x of
// a step is copied straight to LDS (a ring of NS steps, one barrier a step; 16-byte
// pieces XOR-swizzled by row so that operand reads spread over the banks), codes run NS
// steps ahead in registers. Every load is issued whether its step exists or not (the
// last step's again past the end), so the counts that the waits rely on are constant.
// The ring's slots are arrays of their own: with one array the compiler lets operand
// reads of one slot wait for the copies in flight to the others.
// 28672 -> 8192 at 16 rows of bf16 32 us, 4.1 TB/s of codes, scales and x once, bound by
// reading x again in every split; 5120 -> 32003 at 64 rows with zero points 42 us, bound by
// the instructions on the groups' sums (without any 33 us).
template <int XT, int TB, int R, int RW, int KW, int NS, int G, bool ZERO>
__global__ __launch_bounds__(RW * KW * 64) void w4_matvec_shared_kernel(int64_t T, int K, const uint8_t* __restrict__ x,
                                                                        const float* __restrict__ x_scale,
                                                                        const W4Table tab, int t_blocks, bool y_bf16,
                                                                        int splits, float* __restrict__ part) {
  using X = Rows<XT>;
  using Op = typename X::Op;
  using Acc = typename X::Acc;
  constexpr int GP = 128 / G, kWaves = RW * KW;
  constexpr int kRowBytes = 128 * X::kBytes, kChunk = 16 * TB * kRowBytes, kStage = KW * kChunk;
  constexpr int kCopies = kStage / 1024, kPer = (kCopies + kWaves - 1) / kWaves;  // 1 KB copies, and a wave's share
  constexpr int kPieces = kRowBytes / 16, kCopyRows = 64 / kPieces;
  static_assert(NS == 3, "one array a slot");
  __shared__ __align__(1024) unsigned char slot0[kStage];
  __shared__ __align__(1024) unsigned char slot1[kStage];
  __shared__ __align__(1024) unsigned char slot2[kStage];
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rw = wave % RW, kw = wave / RW;
  // When the last step is over the chunk waves' sums meet in the slots: value i of a wave
  // (64 lanes) beside those of the other row waves.
  constexpr int kSumsOf = kStage / 4 / (RW * 64);  // values a slot holds
  static_assert((KW - 1) * R * TB * 4 <= NS * kSumsOf, "sums fit the slots");
  auto sums = [&](int i) -> float& {
    unsigned char* const slot = i / kSumsOf == 0 ? slot0 : i / kSumsOf == 1 ? slot1 : slot2;
    return reinterpret_cast<float*>(slot)[(i % kSumsOf * RW + rw) * 64 + lane];
  };
  const int sp = blockIdx.x % splits;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / splits % t_blocks) * (16 * TB);
  int group = blockIdx.x / splits / t_blocks, p = 0;
  while (group >= tab.group_end[p]) ++p;
  if (p > 0) group -= tab.group_end[p - 1];
  const int N = tab.N[p], nt = (N + 15) / 16, kt = (K + 127) / 128, kg = K / G;
  // this workgroup's steps of KW chunks (the launcher leaves no split empty)
  const int all_steps = (kt + KW - 1) / KW, per = (all_steps + splits - 1) / splits;
  const int step0 = sp * per, steps = min(per, all_steps - step0);
  const int tile0 = (group * RW + rw) * R;
  __amdgpu_buffer_rsrc_t code_rs[R], scale_rs[R], zero_rs[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t tile = min(tile0 + r, nt - 1);
    code_rs[r] = make_rsrc(tab.codes[p] + tile * kt * 1024, kt * 1024);
    scale_rs[r] = make_rsrc(tab.scales[p] + tile * kg * 16, kg * 32);
    if constexpr (ZERO) zero_rs[r] = make_rsrc(tab.zeros[p] + tile * kg * 16, kg * 16);
  }
  const int rows = static_cast<int>(min(T - t0, static_cast<int64_t>(16 * TB)));
  const auto x_rs = make_rsrc(x + t0 * K * X::kBytes, static_cast<uint32_t>(rows) * K * X::kBytes);
  const uint32_t group_at = (GP == 1 ? 0 : GP == 2 ? g >> 1 : g) * 16 + l16;
  const uint32_t group_at_half = (GP == 4 ? g & 1 : 0) * 16 + l16;
  // Copy c of a stage fills its bytes 1024 c ..: rows kCopyRows c .. of a chunk, lane L the
  // physical piece L % kPieces of row L / kPieces, which holds the logical piece
  // (physical ^ row) (mod kPieces).
  int copy_c[kPer];
  uint32_t copy_at[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    copy_c[i] = (wave + kWaves * i) % kCopies;
    const int row = copy_c[i] * kCopyRows % (16 * TB) + lane / kPieces;
    const int piece = (lane ^ row) & (kPieces - 1);
    copy_at[i] = static_cast<uint32_t>(min(row, rows - 1)) * K * X::kBytes + 16 * piece;
  }
  const bool has_half = GP > 1 && (K & 64) != 0;
  auto load_x = [&](int i, unsigned char* stage) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = min((step0 + i) * KW + copy_c[j] * 1024 / kChunk, kt - 1);
      uint32_t off = copy_at[j];
      // (in place of the half that a last chunk lacks, the first one; its scales become 0)
      if (has_half && at == kt - 1) off -= ((lane ^ (copy_c[j] * kCopyRows + lane / kPieces)) & (kPieces / 2)) * 16;
      buf_load16_lds(x_rs, stage + copy_c[j] * 1024, off, at * kRowBytes);
    }
  };
  struct Chunk {
    uint4 codes[R];
    uint32_t scale[R], zero[R];
  };
  Chunk ring[NS];
  auto load_w = [&](int i, Chunk& c) {
    const int at = min((step0 + i) * KW + kw, kt - 1);
    const uint32_t ga = has_half && at == kt - 1 ? group_at_half : group_at;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c.codes[r] = buf_load16(code_rs[r], lane * 16, at * 1024);
      c.scale[r] = buf_load2(scale_rs[r], ga * 2, at * (GP * 32));
      if constexpr (ZERO) c.zero[r] = buf_load1(zero_rs[r], ga, at * (GP * 16));
    }
  };
  float tot[R][TB][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) tot[r][b][j] = 0.f;
  typename X::Wide minus{};
  if constexpr (X::kBiased) minus = X::minus(!ZERO);
  // operand q of row block b: 8 elements at 32 q + 8 g of row 16 b + l16
  auto x_op = [&](const unsigned char* chunk, int b, int q) {
    const int row = 16 * b + l16, byte = (32 * q + 8 * g) * X::kBytes;
    const int piece = ((byte >> 4) ^ row) & (kPieces - 1);
    return *reinterpret_cast<const Op*>(chunk + row * kRowBytes + 16 * piece + (byte & 15));
  };
  auto step = [&](int i, const Chunk& c, const unsigned char* stage) {
    const int at = (step0 + i) * KW + kw;
    if (at >= kt) return;  // the last step may lack a chunk
    const bool absent = has_half && at == kt - 1 && g >= 2;  // the lane's group
    const unsigned char* const chunk = stage + kw * kChunk;
    float s[R][GP];
    uint32_t z[R][GP];
#pragma unroll
    for (int r = 0; r < R; ++r) group_factors<X, GP, ZERO>(absent ? 0u : c.scale[r], ZERO ? c.zero[r] : 0u, s[r], z[r]);
    Acc acc[R][TB], xs[TB];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool first = q * 32 % G == 0;
      typename X::Wide xq[TB];
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        xq[b] = X::widen(x_op(chunk, b, q));
        if constexpr (X::kBiased) xs[b] = X::mma(xq[b], minus, first ? Acc{} : xs[b]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t words[4] = {c.codes[r].x, c.codes[r].y, c.codes[r].z, c.codes[r].w};
        const typename X::Wide w = X::template codes<ZERO>(words[q], z[r][q * 32 / G]);
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[r][b] = X::mma(xq[b], w, first ? Acc{} : acc[r][b]);
      }
      if ((q + 1) * 32 % G == 0) {
        const int j = q * 32 / G;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int b = 0; b < TB; ++b) add_group<X, ZERO>(acc[r][b], xs[b], s[r][j], z[r][j], tot[r][b]);
      }
    }
  };
  // Order of a wave's loads: x of steps 0 .. NS - 2, codes of steps 0 .. NS - 1; then in
  // step i x of step i + NS - 1 and codes of step i + NS. Loads retire in order, so the x
  // of step i has landed when at most as many loads are outstanding as were issued after
  // it: x of NS - 2 steps and codes of NS - 1 (more at the start).
  constexpr int kCodes = R * (ZERO ? 3 : 2);
  constexpr int kWait = (NS - 2) * kPer + (NS - 1) * kCodes;
  static_assert(kWait < 64, "load counter");
  load_x(0, slot0);
  load_x(1, slot1);
  keep_order();
#pragma unroll
  for (int d = 0; d < NS; ++d) {
    load_w(d, ring[d]);
    keep_order();
  }
  auto turn = [&](int i, Chunk& c, const unsigned char* mine, unsigned char* next) {
    wait_vmem_upto<kWait>();
    __syncthreads();  // x of this step is whole, and the step that used `next` is over
    load_x(i + NS - 1, next);
    keep_order();
    step(i, c, mine);
    keep_order();
    load_w(i + NS, c);
    keep_order();
  };
  for (int i = 0; i < steps; i += NS) {
    turn(i, ring[0], slot0, slot2);
    if (i + 1 < steps) turn(i + 1, ring[1], slot1, slot0);
    if (i + 2 < steps) turn(i + 2, ring[2], slot2, slot1);
  }
  wait_vmem();  // run-ahead copies land before their slots are used again or given back
  if constexpr (KW > 1) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KW - 1; ++k) {
      if (kw != k + 1) continue;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) sums((k * R * TB + r * TB + b) * 4 + e) = tot[r][b][e];
    }
    __syncthreads();
    if (kw > 0) return;
  }
  float factor[TB][4];
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t t = min(t0 + 16 * b + 4 * g + e, T - 1);
      factor[b][e] = x_scale != nullptr && splits == 1 ? x_scale[t] : 1.f;
    }
  auto finish = [&](auto* y, int64_t stride) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int n = (tile0 + r) * 16 + l16;
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t t = t0 + 16 * b + 4 * g + e;
          float v = tot[r][b][e];
          if constexpr (KW > 1)
#pragma unroll
            for (int k = 0; k < KW - 1; ++k) v += sums((k * R * TB + r * TB + b) * 4 + e);
          v *= factor[b][e];
          if (t < T && n < N) {
            if constexpr (sizeof(*y) == 2) y[t * stride + n] = to_bf16(v);
            else y[t * stride + n] = v;
          }
        }
    }
  };
  if (splits > 1) {
    int64_t all = 0, before = 0;
    for (int i = 0; i < tab.n; ++i) {
      before = i == p ? all : before;
      all += tab.N[i];
    }
    finish(part + sp * T * all + before, all);
  } else if (y_bf16) {
    finish(static_cast<uint16_t*>(tab.y[p]), N);
  } else {
    finish(static_cast<float*>(tab.y[p]), N);
  }
}

// y = x_scale sum over splits of part [splits][T][all outputs side by side], in order;
// blockIdx.y: the row of x. 4 us for 16 rows of 8192, mostly latency.
constexpr int kMaxSplits = 16;
__global__ __launch_bounds__(256) void w4_matvec_join_kernel(int64_t all, int splits, const float* __restrict__ part,
                                                             const float* __restrict__ x_scale, const W4Table tab,
                                                             bool y_bf16) {
  const int64_t t = blockIdx.y, stride = gridDim.y * all;
  int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n >= all) return;
  const float* const at = part + t * all + n;
  float w[kMaxSplits];
#pragma unroll
  for (int k = 0; k < kMaxSplits; ++k) w[k] = k < splits ? at[k * stride] : 0.f;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxSplits; ++k) v += w[k];
  if (x_scale != nullptr) v *= x_scale[t];
  int p = 0;
  while (n >= tab.N[p]) n -= tab.N[p++];
  const int64_t o = t * tab.N[p] + n;
  if (y_bf16) static_cast<uint16_t*>(tab.y[p])[o] = to_bf16(v);
  else static_cast<float*>(tab.y[p])[o] = v;
}

// A call's arguments, as the launchers pass them on.
struct Call {
  int64_t T;
  int K, group;
  const void* x;
  const float* x_scale;
  W4Table tab;
  bool y_bf16;
  int splits;
  float* part;
  hipStream_t stream;
};

// The launch for the call's group size and zero points.
template <class Go>
void with_group(const Call& c, Go&& go) {
  auto with = [&](auto zero) {
    if (c.group == 32) go(std::integral_constant<int, 32>{}, zero);
    else if (c.group == 64) go(std::integral_constant<int, 64>{}, zero);
    else go(std::integral_constant<int, 128>{}, zero);
  };
  if (c.tab.zeros[0] != nullptr) with(std::true_type{});
  else with(std::false_type{});
}

// Workgroups along the rows of all weights, `tiles` tiles each.
int set_groups(W4Table& tab, int tiles) {
  int groups = 0;
  for (int p = 0; p < tab.n; ++p) {
    groups += ((tab.N[p] + 15) / 16 + tiles - 1) / tiles;
    tab.group_end[p] = groups;
  }
  return groups;
}

template <int XT, int R, int W, int D>
hipError_t run(Call c) {
  const dim3 grid(static_cast<unsigned>(set_groups(c.tab, R)));
  with_group(c, [&](auto g, auto zero) {
    constexpr int kG = decltype(g)::value;
    constexpr bool kZero = decltype(zero)::value;
    // 16 waves of two tiles have 128 registers each: bf16 rows with four groups a chunk and
    // zero points would spill at two chunks in flight (4096 -> 6144 at 4 rows 9.7 us, with one 5.5)
    constexpr int kD = XT == kRowBf16 && kG == 32 && kZero && R * W > 16 ? 1 : D;
    w4_matvec_kernel<XT, R, W, kD, kG, kZero><<<grid, W * 64, 0, c.stream>>>(
        static_cast<int>(c.T), c.K, static_cast<const uint8_t*>(c.x), c.x_scale, c.tab, c.y_bf16);
  });
  return hipGetLastError();
}

template <int XT, int TB, int R, int RW, int KW>
hipError_t run_shared(Call c) {
  const int t_blocks = static_cast<int>((c.T + 16 * TB - 1) / (16 * TB));
  const dim3 grid(static_cast<unsigned>(set_groups(c.tab, R * RW)) * static_cast<unsigned>(t_blocks) *
                  static_cast<unsigned>(c.splits));
  with_group(c, [&](auto g, auto zero) {
    w4_matvec_shared_kernel<XT, TB, R, RW, KW, 3, decltype(g)::value, decltype(zero)::value>
        <<<grid, RW * KW * 64, 0, c.stream>>>(c.T, c.K, static_cast<const uint8_t*>(c.x), c.x_scale, c.tab, t_blocks,
                                              c.y_bf16, c.splits, c.part);
  });
  if (c.splits > 1) {
    int64_t all = 0;
    for (int p = 0; p < c.tab.n; ++p) all += c.tab.N[p];
    w4_matvec_join_kernel<<<dim3(static_cast<unsigned>((all + 255) / 256), static_cast<unsigned>(c.T)), 256, 0, c.stream>>>(
        all, c.splits, c.part, c.x_scale, c.tab, c.y_bf16);
  }
  return hipGetLastError();
}

// Which kernel, and over how many workgroups d_in is split (their float32 sums meet in
// the workspace and a second launch of 4 to 5 us joins them). Measured, it included (us):
//   * up to 16 rows. Over 768 tiles there are workgroups enough: four tiles each (8192 ->
//     28672 at 1 row 26; two tiles and 16 waves 32). Fewer tiles at a usual depth: two tiles
//     over 16 waves (4096 -> 6144 at 4 rows 5.9; one tile 6.9), one tile below 257 (4096 ->
//     1024 at 1 row 4.2; two 4.9). From 96 chunks with few tiles, x in LDS and d_in split
//     (28672 -> 8192 at 16 rows 33, 28672 -> 1024 at 16 rows 14; two tiles over 16 waves 40
//     and 18).
//   * more rows. 32 or 64 in one block where 8-tile workgroups fill the GPU (5120 -> 32003
//     at 64 rows 40; blocks of 32 rows 50), otherwise blocks of 32 rows, 4-tile workgroups
//     and d_in split (28672 -> 2048 at 64 rows 24; 8-tile workgroups of 64 rows, split as
//     often, 32; unsplit 59).
enum Kind { kOneTile, kTwoTiles, kFourTiles, kDeep, kWide32, kWide64, kNarrow };
struct Plan {
  Kind kind;
  int splits;
};
Plan plan(int64_t T, int64_t K, int n, const int* N) {
  int64_t tiles = 0, groups4 = 0, groups8 = 0;
  for (int p = 0; p < n; ++p) {
    const int64_t t = (N[p] + 15) / 16;
    tiles += t;
    groups4 += (t + 3) / 4;
    groups8 += (t + 7) / 8;
  }
  const int64_t chunks = (K + 127) / 128;
  // as many splits as give two workgroups a CU, each with four steps of kw chunks at least
  auto split = [&](Kind kind, int64_t groups, int64_t kw) {
    const int64_t steps = (chunks + kw - 1) / kw;
    int64_t s = std::min<int64_t>({512 / groups, steps / 4, kMaxSplits});
    if (s < 2) return Plan{kind, 1};
    const int64_t per = (steps + s - 1) / s;
    return Plan{kind, static_cast<int>((steps + per - 1) / per)};  // none empty
  };
  if (T <= 16) {
    if (tiles > 768) return {kFourTiles, 1};
    if (chunks >= 96) return split(kDeep, groups4, 4);
    return {tiles > 256 ? kTwoTiles : kOneTile, 1};
  }
  const int64_t blocks32 = (T + 31) / 32, blocks64 = (T + 63) / 64;
  if (T > 32 && groups8 * blocks64 >= 192) return {kWide64, 1};
  if (groups8 * blocks32 >= 192) return {kWide32, 1};
  return split(kNarrow, groups4 * blocks32, 2);
}

template <int XT>
hipError_t pick(Kind kind, const Call& c) {
  switch (kind) {
    case kOneTile: return run<XT, 1, 16, 2>(c);
    case kTwoTiles: return run<XT, 2, 16, 2>(c);
    case kFourTiles: return run<XT, 4, 8, 1>(c);
    case kDeep: return run_shared<XT, 1, 1, 4, 4>(c);
    // (16 waves where the ring is half as wide: 8192 -> 28672 at 32 int8 rows 39 us, with 8 44;
    // bf16 rows 38 with 8, 36 to 47 with 16, where an instance spills)
    case kWide32: return run_shared<XT, 2, 2, 4, XT == kRowBf16 ? 2 : 4>(c);
    case kWide64: return run_shared<XT, 4, 2, 4, 2>(c);
    case kNarrow: return run_shared<XT, 2, 1, 4, 2>(c);
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t w4_matvec_bytes(int64_t T, int64_t K, int n, const int* N) {
  const Plan p = plan(T, K, n, N);
  if (p.splits == 1) return 0;
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += N[i];
  return (static_cast<size_t>(p.splits) * T * all * 4 + 255) / 256 * 256;
}

hipError_t launch_w4_matvec(int64_t T, int K, int group, int x_type, const void* x, const float* x_scale,
                            const W4Table& tab, bool y_bf16, void* workspace, hipStream_t stream) {
  const Plan p = plan(T, K, tab.n, tab.N);
  const Call c{T, K, group, x, x_scale, tab, y_bf16, p.splits, static_cast<float*>(workspace), stream};
  if (x_type == kRowBf16) return pick<kRowBf16>(p.kind, c);
  if (x_type == kRowE4m3) return pick<kRowE4m3>(p.kind, c);
  return pick<kRowI8>(p.kind, c);
}

}  // namespace lnf4
