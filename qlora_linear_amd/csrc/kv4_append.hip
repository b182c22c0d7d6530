// New tokens into the paged 4-bit cache, with the rotation of queries and keys on the way,
// and rows of the cache read back (gfx950). Layout and definitions: kv4.h.
//
// One thread owns eight consecutive elements of a head: a group is 4, 8 or 16 consecutive
// lanes, the eight codes of a key are one 4-byte word of its row, those of a value four
// bytes that lie between the same bytes of its three neighbouring tokens.
#include <type_traits>

#include "device_common.h"
#include "group_code.h"
#include "kv4_launch.h"

namespace lnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 16;  // tokens of a workgroup

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// The code of d = f32(x - lo) >= 0 for a step s > 0: the integer nearest to the exact quotient,
// halves to even. The product with the reciprocal (1 ulp) decides all but the quotients near a
// half; for those the remainder d - n s, which is exact (both are multiples of the smaller's
// last bit and it is below s), is compared with s / 2. A step whose reciprocal
// overflows goes that way too (the comparison is then false).
__device__ __forceinline__ float code_of(float d, float s, float inv) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's last bit is 1
  float n = __builtin_fmaf(d, inv, kMagic) - kMagic;
  if (!(fabsf(__builtin_fmaf(d, inv, -n)) < 0.5f - 0x1p-16f)) {
    n = __builtin_rintf(__fdiv_rn(d, s));
    const float r2 = 2.f * __builtin_fmaf(-n, s, d);
    const bool odd = (static_cast<int>(n) & 1) != 0;
    if (r2 > s || (r2 == s && odd)) n += 1.f;
    if (-r2 > s || (-r2 == s && odd)) n -= 1.f;
  }
  return fminf(n, 15.f);
}

// The eight elements from d0 on of a head rotated: x holds them, row is the head's first element.
// A product of the two float32 (or narrower) factors is exact in float64, so that the sum is
// rounded once there, whether fused or not. rot_dim is a multiple of 16: the eight elements
// are all rotated or none, and all first or all second ones of their pairs.
template <typename In>
__device__ __forceinline__ void rotate8(const In* row, int d0, int rot, bool interleaved, const float* cos,
                                        const float* sin, float (&x)[8]) {
  if (interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(cos + d0 / 2), s = *reinterpret_cast<const float4*>(sin + d0 / 2);
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double a = x[2 * i], b = x[2 * i + 1], ci = cs[i], si = sn[i];
      x[2 * i] = static_cast<float>(a * ci - b * si);
      x[2 * i + 1] = static_cast<float>(b * ci + a * si);
    }
    return;
  }
  const int half = rot >> 1;
  const bool second = d0 >= half;
  const int i0 = second ? d0 - half : d0;
  float other[8], cs[8], sn[8];
  load8(row + (second ? i0 : d0 + half), other);
  load8(cos + i0, cs);
  load8(sin + i0, sn);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double a = x[i], b = other[i], ci = cs[i], si = second ? sn[i] : -sn[i];
    x[i] = static_cast<float>(a * ci + b * si);
  }
}

// A workgroup takes `tile` tokens (the last tile's may not exist) and 2^head_bits of the
// n_q + 2 n_kv heads: queries, keys, values in this order.
template <int D, typename In>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Kv4Append a, ln_kv4_cache c, int tile, int head_bits) {
  constexpr int kPieces = D / 8;
  __shared__ int64_t slot_of[kMaxTile];
  __shared__ int dropped;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile;
  const int head0 = static_cast<int>(blockIdx.y) << head_bits;
  const int n_q = a.q == nullptr ? 0 : a.n_q, heads = n_q + 2 * c.n_kv;
  const int tid = threadIdx.x;

  if (head0 + (1 << head_bits) > n_q) {
    // Which tokens go into the cache: of those with the same slot the last, so that every later
    // token's slot is compared, with the range of the tile's slots first (a prompt's are
    // neighbours; with all of them one by one 8192 tokens took 88 us, not 52)
    const int64_t n_slots = c.n_pages * c.page_size;
    auto kept = [&](int64_t t, int64_t slot) {
      if (slot < 0 || slot >= n_slots) return false;
      return a.rot_dim == 0 || (a.positions[t] >= 0 && a.positions[t] < a.n_pos);
    };
    if (tid < tile) {
      const int64_t slot = t0 + tid < a.T ? a.slots[t0 + tid] : -1;
      slot_of[tid] = kept(t0 + tid, slot) ? slot : -1;
    }
    if (tid == 0) dropped = 0;
    __syncthreads();
    int64_t least = n_slots, most = -1;
    for (int i = 0; i < tile; ++i) {
      const int64_t slot = slot_of[i];
      most = max(most, slot);
      least = min(least, slot < 0 ? n_slots : slot);
    }
    const uint64_t range = static_cast<uint64_t>(most - least);
    auto compare = [&](int64_t t, int64_t slot) {
      if (static_cast<uint64_t>(slot - least) > range) return;
      int same = 0;
      for (int i = 0; i < tile; ++i) same |= (slot == slot_of[i] && t > t0 + i) << i;
      if (same != 0 && kept(t, slot)) atomicOr(&dropped, same);
    };
    if (most >= 0) {
      int64_t t = t0 + 1 + tid;
      for (; t + 3 * kThreads < a.T; t += 4 * kThreads) {
        int64_t slot[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) slot[i] = a.slots[t + i * kThreads];
#pragma unroll
        for (int i = 0; i < 4; ++i) compare(t + i * kThreads, slot[i]);
      }
      for (; t < a.T; t += kThreads) compare(t, a.slots[t]);
    }
    __syncthreads();
  }

  for (int u = tid; u < (tile << head_bits) * kPieces; u += kThreads) {
    const int piece = u % kPieces, rest = u / kPieces;
    const int head = head0 + (rest & ((1 << head_bits) - 1)), i = rest >> head_bits;
    const int64_t t = t0 + i;
    if (head >= heads || t >= a.T) continue;
    const int d0 = 8 * piece;
    const int64_t pos = a.rot_dim == 0 ? 0 : a.positions[t];
    const bool placed = a.rot_dim == 0 || (pos >= 0 && pos < a.n_pos);
    const bool is_q = head < n_q, is_k = !is_q && head < n_q + c.n_kv;
    const int h = is_q ? head : is_k ? head - n_q : head - n_q - c.n_kv;
    const In* row = is_q   ? static_cast<const In*>(a.q) + t * a.q_stride
                    : is_k ? static_cast<const In*>(a.k) + t * a.k_stride
                           : static_cast<const In*>(a.v) + t * a.v_stride;
    row += h * D;
    float x[8];
    load8(row + d0, x);
    if ((is_q || is_k) && d0 < a.rot_dim && placed) {
      const int64_t at = pos * (a.rot_dim >> 1);
      rotate8(row, d0, a.rot_dim, a.interleaved, a.cos + at, a.sin + at, x);
    }
    uint4 b = pack8(x);
    if (is_q) {
      if (!placed) b = uint4{0, 0, 0, 0};
      *reinterpret_cast<uint4*>(a.q_out + (t * n_q + h) * D + d0) = b;
      continue;
    }
    const int64_t slot = (dropped >> i) & 1 ? -1 : slot_of[i];
    if (slot < 0) continue;  // (a group's lanes share their token)

    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) lo = fminf(lo, x[j]), hi = fmaxf(hi, x[j]);
    group_extrema(c.group, lo, hi);
    const uint16_t sb = to_bf16(quotient_of(hi - lo, 15.f, 1.f / 15.f));
    const float s = bf16_to_f32(sb), inv = __builtin_amdgcn_rcpf(s);
    uint32_t code[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) code[j] = s > 0.f ? static_cast<uint32_t>(code_of(x[j] - lo, s, inv)) : 0u;

    const int64_t page = slot / c.page_size;
    const int tok = static_cast<int>(slot - page * c.page_size);
    const int64_t ph = page * c.n_kv + h;
    if (d0 % c.group == 0) {
      const int64_t at = (ph * (D / c.group) + d0 / c.group) * c.page_size + tok;
      reinterpret_cast<uint32_t*>(is_k ? c.k_scales : c.v_scales)[at] = sb | (static_cast<uint32_t>(to_bf16(lo)) << 16);
    }
    const int chunk = d0 / 32, seg = d0 % 32 / 8;
    if (is_k) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) word |= (code[j] | (code[4 + j] << 4)) << (8 * j);
      *reinterpret_cast<uint32_t*>(c.k_codes + (ph * c.page_size + tok) * (D / 2) + seg * (D / 8) + 4 * chunk) = word;
    } else {
      uint8_t* at = c.v_codes + (ph * c.page_size + tok / 4 * 4) * (D / 2) + 4 * seg * (D / 8) + 4 * chunk + tok % 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) at[j * (D / 8)] = static_cast<uint8_t>(code[2 * j] | (code[2 * j + 1] << 4));
    }
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) { *reinterpret_cast<uint4*>(p) = pack8(v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = float4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<float4*>(p)[1] = float4{v[4], v[5], v[6], v[7]};
}

// One thread to eight elements of a slot's key and value of head blockIdx.y.
template <int D, typename Out>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(int64_t T, const int64_t* slots, ln_kv4_cache c, Out* k,
                                                            Out* v) {
  constexpr int kPieces = D / 8;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int piece = static_cast<int>(u % kPieces), h = blockIdx.y;
  const int64_t t = u / kPieces, row = t * c.n_kv + h;
  if (t >= T) return;
  const int d0 = 8 * piece, chunk = d0 / 32, seg = d0 % 32 / 8;
  const int64_t slot = slots[t];
  float xk[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, xv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (slot >= 0 && slot < c.n_pages * c.page_size) {
    const int64_t page = slot / c.page_size;
    const int tok = static_cast<int>(slot - page * c.page_size);
    const int64_t ph = page * c.n_kv + h, at = (ph * (D / c.group) + d0 / c.group) * c.page_size + tok;
    if (k != nullptr) {
      const uint32_t p = reinterpret_cast<const uint32_t*>(c.k_scales)[at];
      const float s = __uint_as_float(p << 16), lo = __uint_as_float(p & 0xFFFF0000u);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(c.k_codes + (ph * c.page_size + tok) * (D / 2) +
                                                            seg * (D / 8) + 4 * chunk);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xk[j] = s * static_cast<float>((w >> (8 * j)) & 15u) + lo;
        xk[4 + j] = s * static_cast<float>((w >> (8 * j + 4)) & 15u) + lo;
      }
    }
    if (v != nullptr) {
      const uint32_t p = reinterpret_cast<const uint32_t*>(c.v_scales)[at];
      const float s = __uint_as_float(p << 16), lo = __uint_as_float(p & 0xFFFF0000u);
      const uint8_t* from = c.v_codes + (ph * c.page_size + tok / 4 * 4) * (D / 2) + 4 * seg * (D / 8) + 4 * chunk + tok % 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b = from[j * (D / 8)];
        xv[2 * j] = s * static_cast<float>(b & 15u) + lo;
        xv[2 * j + 1] = s * static_cast<float>(b >> 4) + lo;
      }
    }
  }
  if (k != nullptr) store8(k + row * D + d0, xk);
  if (v != nullptr) store8(v + row * D + d0, xv);
}

// f(integral_constant of the head's width)
template <class F>
hipError_t with_dim(int d, F&& f) {
  if (d == 64) return f(std::integral_constant<int, 64>{});
  if (d == 128) return f(std::integral_constant<int, 128>{});
  return f(std::integral_constant<int, 256>{});
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Append& a, bool bf16, const ln_kv4_cache& c, hipStream_t stream) {
  // A few tokens: one unit a thread and as many workgroups as that takes. A prompt: sixteen
  // tokens a workgroup, so that later slots are compared by fewer of them.
  const int heads = (a.q == nullptr ? 0 : a.n_q) + 2 * c.n_kv;
  const int tile = a.T >= 512 ? kMaxTile : 1;
  int head_bits = 0;
  while ((tile << head_bits) * (c.head_dim / 8) < (tile == 1 ? kThreads : 4 * kThreads)) ++head_bits;
  const dim3 grid(static_cast<unsigned>((a.T + tile - 1) / tile),
                  static_cast<unsigned>((heads + (1 << head_bits) - 1) >> head_bits));
  return with_dim(c.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (bf16)
      kv4_append_kernel<D, uint16_t><<<grid, kThreads, 0, stream>>>(a, c, tile, head_bits);
    else
      kv4_append_kernel<D, float><<<grid, kThreads, 0, stream>>>(a, c, tile, head_bits);
    return hipGetLastError();
  });
}

hipError_t launch_kv4_read(int64_t T, const int64_t* slots, const ln_kv4_cache& c, bool bf16, void* k, void* v,
                           hipStream_t stream) {
  return with_dim(c.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const dim3 grid(static_cast<unsigned>((T * (D / 8) + kThreads - 1) / kThreads), static_cast<unsigned>(c.n_kv));
    if (bf16)
      kv4_read_kernel<D, uint16_t><<<grid, kThreads, 0, stream>>>(T, slots, c, static_cast<uint16_t*>(k),
                                                                  static_cast<uint16_t*>(v));
    else
      kv4_read_kernel<D, float><<<grid, kThreads, 0, stream>>>(T, slots, c, static_cast<float*>(k),
                                                               static_cast<float*>(v));
    return hipGetLastError();
  });
}

}  // namespace lnf4
