// New tokens into the paged 4-bit cache, with the rotation of queries and keys on the way,
// and rows of the cache read back (gfx950). Layout and definitions: kv4.h.
//
// One thread owns eight consecutive elements of a head: a group is 4, 8 or 16 consecutive lanes,
// the eight codes of a key are one 4-byte word of its row, those of a value four bytes that lie
// between the same bytes of its three neighbouring tokens.
#include <type_traits>

#include "device_common.h"
#include "group_code.h"
#include "kv4_launch.h"

namespace lnf4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

__device__ __forceinline__ void unpack8(const uint4& b, float (&x)[8]) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
}

// The code of d = f32(x - lo) >= 0 for a step s below any that its reciprocal is good for: the
// integer nearest to the exact quotient, halves to even.
__device__ __forceinline__ uint32_t code_by_division(float d, float s) {
  if (!(s > 0.f)) return 0u;
  float n = __builtin_rintf(__fdiv_rn(d, s));
  const float r2 = 2.f * __builtin_fmaf(-n, s, d);
  const bool odd = (static_cast<int>(n) & 1) != 0;
  if (r2 > s || (r2 == s && odd)) n += 1.f;
  if (-r2 > s || (-r2 == s && odd)) n -= 1.f;
  return static_cast<uint32_t>(fminf(n, 15.f));
}

// The codes of eight elements of a group as a word: those of elements 0 .. 3 (EVERY 1) or 0, 2, 4, 6
// (EVERY 2) in the low nibbles of its bytes, the others in the high ones.
// The product with the step's reciprocal is off by less than 2^-18; raised by twice that it
// gives the integer above where the quotient is at or next to a half (of bf16 rows one in a
// hundred is at one, so there is no branch for them). The remainder d - n s is exact (both are
// multiples of the smaller's last bit and it is at most s), and so is its sum with s / 2 near
// -s / 2: below zero the integer below is the nearest, at zero the even one of the two.
template <int EVERY>
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float lo, float s) {
  constexpr float kMagic = 12582912.f;  // 1.5 2^23: the sum's last bits are the integer's
  const float inv = __builtin_amdgcn_rcpf(s), half = 0.5f * s;
  uint32_t n[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = x[j] - lo, f = __builtin_fmaf(d, inv, 0x1p-17f) + kMagic;
    const float over = __builtin_fmaf(kMagic - f, s, d) + half;
    const uint32_t bits = __float_as_uint(f);
    n[j] = bits + static_cast<uint32_t>((static_cast<int>(__float_as_uint(over)) - static_cast<int>(bits & 1u)) >> 31);
  }
  if (!(s > 0x1p-120f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = code_by_division(x[j] - lo, s);
  }
  constexpr int A = EVERY, B = EVERY == 1 ? 4 : 1;  // step of the low nibbles, first of the high ones
  auto bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u),
                                 0x05040100u);
  };
  return bytes(n[0], n[A], n[2 * A], n[3 * A]) | (bytes(n[B], n[B + A], n[B + 2 * A], n[B + 3 * A]) << 4);
}

// x c + y s of eight elements as bf16, as float64 sums that are rounded to float32 and then to
// bf16 (a product of two float32 is exact there). The float32 sum is off by less than e, its
// two roundings and the product's; where bf16 has the same neighbour for both ends, that is the one,
// else (in a wave in five) the eight are summed in float64.
__device__ __forceinline__ uint4 rotated8(const float (&x)[8], const float (&y)[8], const float (&c)[8],
                                          const float (&s)[8]) {
  uint32_t lo[4], hi[4], unlike = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float r[2], e[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p = y[2 * j + i] * s[2 * j + i];
      r[i] = __builtin_fmaf(x[2 * j + i], c[2 * j + i], p);
      e[i] = __builtin_fmaf(__builtin_fmaf(fabsf(x[2 * j + i]), fabsf(c[2 * j + i]), fabsf(p)), 0x1p-22f, 0x1p-146f);
    }
    lo[j] = pack_bf16x2(r[0] - e[0], r[1] - e[1]);
    hi[j] = pack_bf16x2(r[0] + e[0], r[1] + e[1]);
    unlike |= lo[j] ^ hi[j];
  }
  if (unlike != 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float r[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const double a = x[2 * j + i], b = y[2 * j + i], ci = c[2 * j + i], si = s[2 * j + i];
        r[i] = static_cast<float>(a * ci + b * si);
        asm volatile("" : "+v"(r[i]));  // (the compiler else rounds the float64 to bf16 at once)
      }
      lo[j] = pack_bf16x2(r[0], r[1]);
    }
  }
  return uint4{lo[0], lo[1], lo[2], lo[3]};
}

// Eight elements as they lie in memory.
struct Raw16 {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void widen(float (&x)[8]) const { unpack8(v, x); }
};
struct Raw32 {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// Heads of a workgroup, and tokens, where a thread has N rows.
constexpr int heads_of(int D, int N) { return N == 1 ? 2048 / D : D == 64 ? 8 : 4; }
constexpr int tokens_of(int D, int N) { return N == 1 ? 1 : D == 256 ? 8 : 16; }

// Which of a workgroup's TILE tokens go into the cache, by their slots (else -1): of those with
// the same slot the last, so that every later slot of the launch is compared, with the range of
// the tile's slots first (a prompt's are neighbours; one by one 8192 tokens took 23 us more).
template <int TILE>
__device__ __forceinline__ void find_slots(const Kv4Append& a, const ln_kv4_cache& c, int64_t t0, int64_t* slot_of,
                                           int* dropped) {
  const int tid = threadIdx.x;
  const int64_t n_slots = c.n_pages * c.page_size;
  auto kept = [&](int64_t t, int64_t slot) {
    if (slot < 0 || slot >= n_slots) return false;
    return a.rot_dim == 0 || (a.positions[t] >= 0 && a.positions[t] < a.n_pos);
  };
  if (tid < TILE) {
    const int64_t slot = t0 + tid < a.T ? a.slots[t0 + tid] : -1;
    slot_of[tid] = kept(t0 + tid, slot) ? slot : -1;
  }
  if (tid == 0) *dropped = 0;
  __syncthreads();
  int64_t least = n_slots, most = -1;
#pragma unroll
  for (int i = 0; i < TILE; ++i) {
    const int64_t slot = slot_of[i];
    most = max(most, slot);
    least = min(least, slot < 0 ? n_slots : slot);
  }
  const uint64_t range = static_cast<uint64_t>(most - least);
  auto compare = [&](int64_t t, int64_t slot) {
    if (static_cast<uint64_t>(slot - least) > range) return;
    int same = 0;
    for (int i = 0; i < TILE; ++i) same |= (slot == slot_of[i] && t > t0 + i) << i;
    if (same != 0 && kept(t, slot)) atomicOr(dropped, same);
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
  if (tid < TILE && ((*dropped >> tid) & 1)) slot_of[tid] = -1;
  __syncthreads();
}

// Codes of eight elements from d0 on, in bf16, of a slot's row of head h, and the group's scales.
template <int D, int EVERY>
__device__ __forceinline__ uint32_t coded8(const ln_kv4_cache& c, const uint4& b, int d0, int64_t ph, int tok,
                                           uint16_t* scales) {
  float x[8];
  unpack8(b, x);
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) lo = fminf(lo, x[j]), hi = fmaxf(hi, x[j]);
  group_extrema(c.group, lo, hi);
  const uint16_t sb = to_bf16(quotient_of(hi - lo, 15.f, 1.f / 15.f));
  if (d0 % c.group == 0) {
    const int64_t at = (ph * (D / c.group) + d0 / c.group) * c.page_size + tok;
    reinterpret_cast<uint32_t*>(scales)[at] = sb | (static_cast<uint32_t>(to_bf16(lo)) << 16);
  }
  return codes8<EVERY>(x, lo, bf16_to_f32(sb));
}

// The first `turned` workgroups along y take queries and keys, which are rotated: a thread one
// token of N heads, which share their angles (half of the kernel's loads where each row
// fetches its own). The others take values: a thread N tokens of a head, whose codes are whole
// words where the tokens fill four places that lie together. N is 1 for fewer than 512 tokens, so
// that there are as many workgroups as can be, or 4.
// 8192 tokens of 32 and 8 heads of 128 (187 MB) take 53 us, the vector units issuing in 71 % of the CUs'
// cycles; 2047 tokens of 40 and 40 heads, groups of 32 (99 MB), 37 us, 81 %. With the chunks of a tile's heads
// as the grid's fastest index the first took 57.
template <int D, typename In, int N>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Kv4Append a, ln_kv4_cache c, int turned) {
  constexpr int kPieces = D / 8, kTile = tokens_of(D, N), kHeads = heads_of(D, N);
  typedef std::conditional_t<sizeof(In) == 2, Raw16, Raw32> Raw;
  __shared__ int64_t slot_of[kTile];
  __shared__ int dropped;
  const int tile = blockIdx.x, part = blockIdx.y;
  const int64_t t0 = static_cast<int64_t>(tile) * kTile;
  const int piece = threadIdx.x % kPieces, rest = threadIdx.x / kPieces, d0 = 8 * piece;
  const int chunk = d0 / 32, seg = d0 % 32 / 8;

  if (part < turned) {
    const int n_q = a.q == nullptr ? 0 : a.n_q, heads = n_q + c.n_kv;
    const int i = rest % kTile, head0 = part * kHeads + rest / kTile * N;
    const int64_t t = min(t0 + i, a.T - 1);
    const int half = a.rot_dim >> 1;
    const bool turn = d0 < a.rot_dim, second = !a.interleaved && d0 >= half;
    int64_t pos = a.rot_dim == 0 ? 0 : a.positions[t];
    const bool placed = a.rot_dim == 0 || (pos >= 0 && pos < a.n_pos);
    if (!placed) pos = 0;
    Raw raw[N], other[N];
    float cs[8], sn[8];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int head = min(head0 + n, heads - 1);
      const In* row = head < n_q ? static_cast<const In*>(a.q) + t * a.q_stride + head * D
                                 : static_cast<const In*>(a.k) + t * a.k_stride + (head - n_q) * D;
      raw[n].load(row + d0);
      if (turn && !a.interleaved) other[n].load(row + d0 + (second ? -half : half));
    }
    if (turn) {
      const float *cos = a.cos + pos * half, *sin = a.sin + pos * half;
      if (a.interleaved) {
        const float4 c4 = *reinterpret_cast<const float4*>(cos + d0 / 2), s4 = *reinterpret_cast<const float4*>(sin + d0 / 2);
        const float c1[4] = {c4.x, c4.y, c4.z, c4.w}, s1[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) cs[2 * j] = cs[2 * j + 1] = c1[j], sn[2 * j] = -s1[j], sn[2 * j + 1] = s1[j];
      } else {
        load8(cos + (second ? d0 - half : d0), cs);
        load8(sin + (second ? d0 - half : d0), sn);
#pragma unroll
        for (int j = 0; j < 8; ++j) sn[j] = second ? sn[j] : -sn[j];
      }
    }
    if ((part + 1) * kHeads > n_q) find_slots<kTile>(a, c, t0, slot_of, &dropped);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int head = head0 + n;
      if (head >= heads || t0 + i >= a.T) continue;
      float x[8], y[8];
      raw[n].widen(x);
      uint4 b;
      if (turn && placed) {
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
        } else {
          other[n].widen(y);
        }
        b = rotated8(x, y, cs, sn);
      } else {
        b = pack8(x);
      }
      if (head < n_q) {
        if (!placed) b = uint4{0, 0, 0, 0};
        *reinterpret_cast<uint4*>(a.q_out + (t * n_q + head) * D + d0) = b;
        continue;
      }
      const int64_t slot = slot_of[i];
      if (slot < 0) continue;  // (a group's lanes share their token)
      const int64_t page = slot / c.page_size, ph = page * c.n_kv + head - n_q;
      const int tok = static_cast<int>(slot - page * c.page_size);
      *reinterpret_cast<uint32_t*>(c.k_codes + (ph * c.page_size + tok) * (D / 2) + seg * (D / 8) + 4 * chunk) =
          coded8<D, 1>(c, b, d0, ph, tok, c.k_scales);
    }
    return;
  }

  const int head = (part - turned) * kHeads + rest % kHeads, i0 = rest / kHeads * N;
  Raw raw[N];
#pragma unroll
  for (int n = 0; n < N; ++n)
    raw[n].load(static_cast<const In*>(a.v) + min(t0 + i0 + n, a.T - 1) * a.v_stride + min(head, c.n_kv - 1) * D + d0);
  find_slots<kTile>(a, c, t0, slot_of, &dropped);
  if (head >= c.n_kv) return;
  // byte j of a token's word is its among the four bytes of elements 2 j, 2 j + 1
  uint32_t word[N];
  uint8_t* at[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int64_t slot = slot_of[i0 + n];
    if (slot < 0) continue;
    float x[8];
    raw[n].widen(x);
    const int64_t page = slot / c.page_size, ph = page * c.n_kv + head;
    const int tok = static_cast<int>(slot - page * c.page_size);
    word[n] = coded8<D, 2>(c, pack8(x), d0, ph, tok, c.v_scales);
    at[n] = c.v_codes + (ph * c.page_size + tok / 4 * 4) * (D / 2) + 4 * seg * (D / 8) + 4 * chunk + tok % 4;
  }
  if constexpr (N == 4) {
    const int64_t s = slot_of[i0];
    if (s >= 0 && s % 4 == 0 && slot_of[i0 + 1] == s + 1 && slot_of[i0 + 2] == s + 2 && slot_of[i0 + 3] == s + 3) {
      // 4 x 4 bytes transposed: whole words
      const uint32_t a01 = __builtin_amdgcn_perm(word[1], word[0], 0x05010400u), a23 = __builtin_amdgcn_perm(word[1], word[0], 0x07030602u);
      const uint32_t b01 = __builtin_amdgcn_perm(word[3], word[2], 0x05010400u), b23 = __builtin_amdgcn_perm(word[3], word[2], 0x07030602u);
      *reinterpret_cast<uint32_t*>(at[0]) = __builtin_amdgcn_perm(b01, a01, 0x05040100u);
      *reinterpret_cast<uint32_t*>(at[0] + D / 8) = __builtin_amdgcn_perm(b01, a01, 0x07060302u);
      *reinterpret_cast<uint32_t*>(at[0] + 2 * (D / 8)) = __builtin_amdgcn_perm(b23, a23, 0x05040100u);
      *reinterpret_cast<uint32_t*>(at[0] + 3 * (D / 8)) = __builtin_amdgcn_perm(b23, a23, 0x07060302u);
      return;
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (slot_of[i0 + n] < 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) at[n][j * (D / 8)] = static_cast<uint8_t>(word[n] >> (8 * j));
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

// Tokens of a launch at most. Each tile of a launch compares its slots with all later ones of the launch, and
// a later launch writes over an earlier one's, which also keeps the last. 65536 tokens of 32 and 8 heads of
// 128: 419 us, in launches of 16384 444, of 4096 472, in one 591.
constexpr int64_t kAtOnce = 8192;

hipError_t launch_kv4_append(const Kv4Append& all, bool bf16, const ln_kv4_cache& c, hipStream_t stream) {
  const int heads = (all.q == nullptr ? 0 : all.n_q) + c.n_kv;
  const int64_t e = bf16 ? 2 : 4;
  auto from = [](const void* p, int64_t bytes) -> const void* { return p == nullptr ? p : static_cast<const char*>(p) + bytes; };
  return with_dim(c.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    Kv4Append a = all;
    auto run = [&](auto in, auto rows) {
      constexpr int N = decltype(rows)::value, kTile = tokens_of(D, N), kHeads = heads_of(D, N);
      const int turned = (heads + kHeads - 1) / kHeads;
      const dim3 grid(static_cast<unsigned>((a.T + kTile - 1) / kTile),
                      static_cast<unsigned>(turned + (c.n_kv + kHeads - 1) / kHeads));
      kv4_append_kernel<D, decltype(in), N><<<grid, kThreads, 0, stream>>>(a, c, turned);
    };
    for (int64_t t0 = 0; t0 < all.T; t0 += kAtOnce) {
      a.T = all.T - t0 < kAtOnce ? all.T - t0 : kAtOnce;
      a.q = from(all.q, t0 * all.q_stride * e), a.k = from(all.k, t0 * all.k_stride * e);
      a.v = from(all.v, t0 * all.v_stride * e), a.slots = all.slots + t0;
      a.positions = all.positions == nullptr ? nullptr : all.positions + t0;
      a.q_out = all.q_out == nullptr ? nullptr : all.q_out + t0 * all.n_q * D;
      const bool many = a.T >= 512;
      if (bf16 && many)
        run(uint16_t{}, std::integral_constant<int, 4>{});
      else if (bf16)
        run(uint16_t{}, std::integral_constant<int, 1>{});
      else if (many)
        run(float{}, std::integral_constant<int, 4>{});
      else
        run(float{}, std::integral_constant<int, 1>{});
    }
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
