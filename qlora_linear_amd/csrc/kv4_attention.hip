// Attention over the paged 4-bit cache (gfx950). Layout and definitions: kv4.h.
//
//     y = sum_t p_t v_t / sum_t p_t,   p_t = 2^(c q.k_t - m),   c = scale log2 e
// in one pass over the keys with a running maximum m. The matrix instruction multiplies codes,
// which widen to bf16 exactly; steps and least values are applied to its 16 x 16 results:
//     q.k_t  = sum_g s_tg (q_g . c_tg) + lo_tg sum(q_g)
//     y_g    = sum_t (p_t s_tg) (c_tg - 8) + sum_t p_t (lo_tg + 8 s_tg)
// (around 8 the rounding of p s to bf16 multiplies the deviation from the middle of the range,
// not the value; sum_t p_t s_tg over the rounded products is one more instruction against ones).
//
// A wave works on tiles of 32 keys, alone: keys are the rows of the first product and queries
// its columns (16 a tile: the tokens of a sequence times the query heads of a key head), so that
// a lane's results are eight keys of one query. That is the operand of the second product as it
// is, whose rows are elements of the head: nothing moves between lanes in a tile, and codes
// reach the lanes that multiply them straight from global memory, 16 rows of a key tile at a
// time. The maximum is raised only when a score passes it by 2^8 (a vote); p then stays below
// 2^8, which costs no accuracy, and the cross-lane maximum and the rescaling drop out of most tiles.
//
// The four waves of a workgroup take every fourth tile of a row block (up to 16 NQ rows of one
// sequence and key head) and join in LDS. Row blocks and their key tiles, in steps of four, are
// laid end to end, and each workgroup takes an equal share of that line, whatever the sequences'
// lengths: a row block that is cut is written as float32 parts, which a second launch joins in
// order.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "kv4_launch.h"

namespace lnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 32;             // keys of a wave's tile
constexpr float kLowest = -3.0e38f;   // the maximum of no keys
constexpr int kListed = 1024;         // sequences whose steps are summed in LDS

struct Plan {
  int wgs;           // workgroups that share the steps
  int items;         // row blocks at most
  bool per_sequence; // one row block a sequence: workgroups sum the steps themselves
  int nq;            // 16-row tiles of a row block
  int join_rows;     // rows of one at most
};

// The row block that begins in a workgroup's share and goes on in others', the last of them
// `last` (0: there is none).
struct alignas(32) Cut {
  int last, head, c0, row0, rows;
};

struct Args {
  Kv4Attention a;
  ln_kv4_cache c;
  int heads;          // query heads of a key head
  int rows;           // of a row block, 16 NQ
  int tiles_per_page;
  uint32_t page_inv;  // 2^32 / tiles_per_page, rounded up
  float scale2;       // scale log2 e
  int wgs, items, per_sequence;
  // workspace: first[b] = row blocks before sequence b, before[i] = steps before row block i of
  // one key head, before[n] all of them, seq[i] its sequence; the parts; a workgroup's cut
  int *count, *first, *before, *seq;
  float *part_o, *part_ml;
  Cut* cut;
};

// A row block: rows [row0, row0 + rows) of a sequence's n_b heads rows, keys [lo, hi) that any
// of them sees.
struct Block {
  int b, c0, n, len, row0, rows, lo, hi;
  __device__ __forceinline__ int steps() const {
    return max(1, ((hi + kTile - 1) / kTile - lo / kTile + kWaves - 1) / kWaves);
  }
};

__device__ __forceinline__ void seq_rows(const Kv4Attention& a, int b, int& c0, int& n) {
  if (a.cu_q == nullptr) {
    c0 = b, n = 1;
  } else {
    c0 = min(max(a.cu_q[b], 0), a.T);
    n = min(max(a.cu_q[b + 1], c0), a.T) - c0;
  }
}

__device__ __forceinline__ Block make_block(const Args& g, int b, int rb) {
  Block k;
  k.b = b;
  seq_rows(g.a, b, k.c0, k.n);
  k.len = min(max(g.a.lens[b], 0), g.a.max_pages * g.c.page_size);
  k.row0 = rb * g.rows;
  k.rows = min(g.rows, k.n * g.heads - k.row0);
  const int j0 = k.row0 / g.heads, j1 = (k.row0 + max(k.rows, 1) - 1) / g.heads;
  k.hi = max(k.len - k.n + j1 + 1, 0);
  k.lo = g.a.window > 0 ? max(k.len - k.n + j0 + 1 - g.a.window, 0) : 0;
  if (k.rows <= 0 || k.lo >= k.hi) k.lo = k.hi = 0;
  return k;
}

// (sums above 2^30 come of a cu_q that does not rise only)
constexpr int kMostSteps = 1 << 30;
__device__ __forceinline__ int wave_scan(int v, int most) {
  const int lane = threadIdx.x & 63;
  v = min(v, most);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v = min(v + o, most);
  }
  return v;
}

// Inclusive sum of v over the workgroup's threads, all the sum, both held at `most`. part: one
// int a wave.
template <int WAVES>
__device__ __forceinline__ int block_scan(int v, int* part, int& all, int most) {
  const int wave = threadIdx.x >> 6;
  v = wave_scan(v, most);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) part[wave] = v;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before = min(before + (w < wave ? part[w] : 0), most);
    all = min(all + part[w], most);
  }
  return min(v + before, most);
}

// The number of entries of the rising list at[0 .. n) that are <= x, less one.
__device__ __forceinline__ int place_of(const int* at, int n, int64_t x, int64_t times) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] * times <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Workgroup w's share begins at step_of(w) of all steps; the workgroup that has step x.
__device__ __forceinline__ int64_t step_of(int w, int64_t steps, int wgs) { return w * steps / wgs; }
__device__ __forceinline__ int wg_of(int64_t x, int64_t steps, int wgs) {
  return static_cast<int>(((x + 1) * wgs - 1) / steps);
}
__device__ __forceinline__ int sharing(int64_t steps, int wgs) {
  return static_cast<int>(min(static_cast<int64_t>(wgs), steps));
}

// Row blocks and steps of ragged sequences of any length: one workgroup.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void kv4_plan_kernel(Args g) {
  __shared__ int part[kPlanThreads / 64];
  const int tid = threadIdx.x;
  int items = 0, all;
  for (int b0 = 0; b0 < g.a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int c0, n = 0;
    if (b < g.a.B) seq_rows(g.a, b, c0, n);
    const int mine = (n * g.heads + g.rows - 1) / g.rows;
    const int upto = block_scan<kPlanThreads / 64>(mine, part, all, g.items);
    if (b < g.a.B) g.first[b] = min(items + max(upto - mine, 0), g.items);
    items = min(items + all, g.items);  // (more only if cu_q does not rise)
  }
  __threadfence_block();
  __syncthreads();
  int steps = 0;
  for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int mine = 0, b = 0;
    if (i < items) {
      b = place_of(g.first, g.a.B, i, 1);
      mine = make_block(g, b, i - g.first[b]).steps();
    }
    const int at = steps + block_scan<kPlanThreads / 64>(mine, part, all, kMostSteps) - mine;
    if (i < items) g.before[i] = at, g.seq[i] = b;
    steps += all;
  }
  if (tid == 0) g.before[items] = steps, *g.count = items;
}

// Eight codes as bf16, exactly: a byte c of 0 .. 15 is c 2^-9 in E4M3.
__device__ __forceinline__ uint4 wide_codes(uint32_t lo, uint32_t hi) {
  auto two = [](uint32_t v, auto upper) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, decltype(upper)::value));
  };
  return uint4{two(lo, std::false_type{}), two(lo, std::true_type{}), two(hi, std::false_type{}),
               two(hi, std::true_type{})};
}

template <int D, int G, int NQ>
struct Wave {
  static constexpr int C = D / 32, NG = D / G, CG = G / 32;

  struct alignas(D / 8 < 16 ? D / 8 : 16) Words {
    uint32_t w[C];
  };
  // a tile's codes and parameters as they lie in memory
  struct Raw {
    Words k[2], v[2];
    uint4 ks[2][NG], vs[2][NG];
  };

  uint4 q[NQ][C];
  float q_sum[NQ][NG];  // sum of a query's group, in its lanes
  int first[NQ], last[NQ];  // the keys [first, last) that the lane's query sees
  int all_lo, all_hi;       // the keys that every row sees
  int tiles_q;              // tiles that hold rows
  f32x4_t o[NQ][C][2], z[NQ][NG];
  float mid[NQ][NG], m[NQ], l[NQ];

  __device__ __forceinline__ void begin(const Args& g, const Block& k, int h) {
    const int lane = threadIdx.x & 63, col = lane & 15, seg = lane >> 4;
    tiles_q = max(1, (k.rows + 15) / 16);
    // every row sees what the first does, from where the last one's window begins
    all_hi = max(k.len - k.n + k.row0 / g.heads + 1, 0);
    all_lo = g.a.window > 0 ? max(k.len - k.n + (k.row0 + max(k.rows, 1) - 1) / g.heads + 1 - g.a.window, 0) : 0;
    const uint4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const int row = k.row0 + min(16 * t + col, max(k.rows, 1) - 1);  // rows past the end follow the last
      const int j = row / g.heads;
      last[t] = max(k.len - k.n + j + 1, 0);
      first[t] = g.a.window > 0 ? max(last[t] - g.a.window, 0) : 0;
      const uint16_t* from = g.a.q + (k.c0 + j) * g.a.q_stride + (h * g.heads + row - j * g.heads) * D + 8 * seg;
      const bool ok = 16 * t + col < k.rows;
#pragma unroll
      for (int c = 0; c < C; ++c) q[t][c] = ok ? *reinterpret_cast<const uint4*>(from + 32 * c) : uint4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = i * CG; c < (i + 1) * CG; ++c) s = mfma16(ones, q[t][c], s);
        q_sum[t][i] = s[0];
        z[t][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        mid[t][i] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) o[t][c][0] = o[t][c][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      m[t] = kLowest;
      l[t] = 0.f;
    }
  }

  static __device__ __forceinline__ void load(const Args& g, int page, int tile_in_page, int h, Raw& r) {
    const int lane = threadIdx.x & 63, col = lane & 15, seg = lane >> 4;
    const int64_t ph = static_cast<int64_t>(page) * g.c.n_kv + h;
    const int tok = tile_in_page * kTile;
    const int64_t codes = (ph * g.c.page_size + tok) * (D / 2);
    const uint8_t* kc = g.c.k_codes + codes + col * (D / 2) + seg * (D / 8);
    const uint8_t* vc = g.c.v_codes + codes + seg * (2 * D) + col * (D / 8);
    const int64_t par = (ph * NG * g.c.page_size + tok + 4 * seg) * 2;
    const uint16_t *ks = g.c.k_scales + par, *vs = g.c.v_scales + par;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      r.k[s] = *reinterpret_cast<const Words*>(kc + s * 16 * (D / 2));
      r.v[s] = *reinterpret_cast<const Words*>(vc + s * 8 * D);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        r.ks[s][i] = *reinterpret_cast<const uint4*>(ks + (i * g.c.page_size + 16 * s) * 2);
        r.vs[s][i] = *reinterpret_cast<const uint4*>(vs + (i * g.c.page_size + 16 * s) * 2);
      }
    }
  }

  static __device__ __forceinline__ float step(const uint4& p, int i) {
    const uint32_t w = i == 0 ? p.x : i == 1 ? p.y : i == 2 ? p.z : p.w;
    return __uint_as_float(w << 16);
  }
  static __device__ __forceinline__ float least(const uint4& p, int i) {
    const uint32_t w = i == 0 ? p.x : i == 1 ? p.y : i == 2 ? p.z : p.w;
    return __uint_as_float(w & 0xFFFF0000u);
  }

  // One tile: keys key0 .. key0 + 31. MASK: some row does not see some of them.
  template <bool MASK>
  __device__ __forceinline__ void tile(const Raw& r, int key0, float scale2) {
    const int seg = (threadIdx.x & 63) >> 4;
    float x[NQ][2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        f32x4_t acc[NQ];
#pragma unroll
        for (int t = 0; t < NQ; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = i * CG; c < (i + 1) * CG; ++c) {
          const uint32_t w = r.k[s].w[c];
          const uint4 wide = wide_codes(w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu);
#pragma unroll
          for (int t = 0; t < NQ; ++t)
            if (NQ == 1 || t < tiles_q) acc[t] = mfma16(wide, q[t][c], acc[t]);
        }
#pragma unroll
        for (int t = 0; t < NQ; ++t)
          if (NQ == 1 || t < tiles_q) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float b = least(r.ks[s][i], e) * q_sum[t][i];
              x[t][s][e] = __builtin_fmaf(step(r.ks[s][i], e), acc[t][e], i == 0 ? b : x[t][s][e] + b);
            }
          }
      }
    }
    uint4 p[NQ][NG];
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (NQ > 1 && t >= tiles_q) continue;
      if constexpr (MASK) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 16 * s + 4 * seg + e;
            if (key < first[t] || key >= last[t]) x[t][s][e] = -__builtin_inff();
          }
      }
      float top = x[t][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[t][e >> 2][e & 3]);
      top *= scale2;
      if (__any(top > m[t] + 8.f)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fmaxf(m[t], top), f = __builtin_amdgcn_exp2f(m[t] - now);
        m[t] = now;
        l[t] *= f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          mid[t][i] *= f;
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][i][e] *= f;
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][c][0][e] *= f, o[t][c][1][e] *= f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& v = x[t][e >> 2][e & 3];
        v = __builtin_amdgcn_exp2f(__builtin_fmaf(v, scale2, -m[t]));
        l[t] += v;
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = x[t][e >> 2][e & 3], s = step(r.vs[e >> 2][i], e & 3);
          const float centre = __builtin_fmaf(8.f, s, least(r.vs[e >> 2][i], e & 3));
          // (what a masked place holds may be no number)
          w[e] = MASK && v == 0.f ? 0.f : v * s;
          mid[t][i] = MASK && v == 0.f ? mid[t][i] : __builtin_fmaf(v, centre, mid[t][i]);
        }
        p[t][i] = uint4{pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]),
                        pack_bf16x2(w[6], w[7])};
      }
    }
    const uint4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int i = 0; i < NG; ++i) {
#pragma unroll
      for (int t = 0; t < NQ; ++t)
        if (NQ == 1 || t < tiles_q) z[t][i] = mfma16(ones, p[t][i], z[t][i]);
#pragma unroll
      for (int c = i * CG; c < (i + 1) * CG; ++c) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 a = wide_codes((r.v[0].w[c] >> (4 * half)) & 0x0F0F0F0Fu, (r.v[1].w[c] >> (4 * half)) & 0x0F0F0F0Fu);
          // the conversion's two words of a tile's four keys are operands 0 .. 3 and 4 .. 7
#pragma unroll
          for (int t = 0; t < NQ; ++t)
            if (NQ == 1 || t < tiles_q) o[t][c][half] = mfma16(a, p[t][i], o[t][c][half]);
        }
      }
    }
  }

  // The sums over the wave's lanes, centres applied: o holds sum p v of the tiles so far.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (NQ > 1 && t >= tiles_q) continue;
      l[t] += __shfl_xor(l[t], 16);
      l[t] += __shfl_xor(l[t], 32);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float c = mid[t][i];
        c += __shfl_xor(c, 16);
        c += __shfl_xor(c, 32);
        c = __builtin_fmaf(-8.f, z[t][i][0], c);
#pragma unroll
        for (int k = i * CG; k < (i + 1) * CG; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][k][0][e] += c, o[t][k][1][e] += c;
      }
    }
  }
};

template <int D>
struct Joined {
  static constexpr int kStride = D + 4;  // floats of a row in LDS: rows start 4 banks apart
  float o[kWaves][16][kStride];
  float m[kWaves][16], l[kWaves][16];
};

__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(a, b), pack_bf16x2(c, d)};
}

template <int D, int G, int NQ>
__global__ __launch_bounds__(kThreads) void kv4_attention_kernel(Args g) {
  constexpr int C = D / 32;
  __shared__ Joined<D> joined;
  __shared__ int listed[kListed + 1];
  __shared__ int part[kWaves];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n_kv = g.c.n_kv;

  // the steps before every row block
  int items;
  const int* before;
  if (g.per_sequence) {
    items = g.a.B;
    int steps = 0, all;
    for (int b0 = 0; b0 < items; b0 += kThreads) {
      const int b = b0 + tid;
      const int mine = b < items ? make_block(g, b, 0).steps() : 0;
      const int at = steps + block_scan<kWaves>(mine, part, all, kMostSteps);
      if (b < items) listed[b + 1] = at;
      steps += all;
    }
    if (tid == 0) listed[0] = 0;
    __syncthreads();
    before = listed;
  } else {
    items = *g.count;
    before = g.before;
  }
  const int64_t steps = static_cast<int64_t>(before[items]) * n_kv;
  const int wgs = sharing(steps, g.wgs), wg = blockIdx.x;
  if (wg >= wgs) {
    if (tid == 0) g.cut[wg].last = 0;
    return;
  }
  const int64_t end = step_of(wg + 1, steps, wgs), begin = step_of(wg, steps, wgs);

  Cut cut = {0, 0, 0, 0, 0};
  int64_t at = begin;
  int item = __builtin_amdgcn_readfirstlane(place_of(before, items, at, n_kv));
  while (at < end) {
    const int base = __builtin_amdgcn_readfirstlane(before[item]);
    const int own = __builtin_amdgcn_readfirstlane(before[item + 1]) - base;  // steps of the row block
    const int64_t in = at - static_cast<int64_t>(base) * n_kv;
    const int h = static_cast<int>(in / own);
    const int s0 = static_cast<int>(in - static_cast<int64_t>(h) * own);
    const int s1 = static_cast<int>(min(static_cast<int64_t>(own), s0 + end - at));
    const int b = g.per_sequence ? item : __builtin_amdgcn_readfirstlane(g.seq[item]);
    const Block k = make_block(g, b, g.per_sequence ? 0 : item - __builtin_amdgcn_readfirstlane(g.first[b]));

    Wave<D, G, NQ> w;
    w.begin(g, k, h);
    const int t_end = (k.hi + kTile - 1) / kTile;
    const int32_t* table = g.a.block_table + static_cast<int64_t>(b) * g.a.max_pages;
    for (int t = k.lo / kTile + kWaves * s0 + wave, s = s0; s < s1 && t < t_end; ++s, t += kWaves) {
      const int slot = g.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(t, g.page_inv));
      const int page = __builtin_amdgcn_readfirstlane(table[slot]);
      if (page < 0 || page >= g.c.n_pages) continue;
      typename Wave<D, G, NQ>::Raw raw;
      w.load(g, page, t - slot * g.tiles_per_page, h, raw);
      if (t * kTile >= w.all_lo && t * kTile + kTile <= w.all_hi)
        w.template tile<false>(raw, t * kTile, g.scale2);
      else
        w.template tile<true>(raw, t * kTile, g.scale2);
    }
    w.finish();

    // The waves' sums, 16 rows at a time. Whole: y. A part: slot 1 of the workgroup where the
    // row block begins in its share, 0 where it began before.
    const bool whole = s0 == 0 && s1 == own;
    const int64_t slot = 2 * static_cast<int64_t>(wg) + (s0 == 0 ? 1 : 0);
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (16 * t >= k.rows) break;
      __syncthreads();
      const int col = lane & 15, seg = lane >> 4;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<float4*>(&joined.o[wave][col][32 * c + 8 * seg + 2 * e]) =
              float4{w.o[t][c][0][e], w.o[t][c][1][e], w.o[t][c][0][e + 1], w.o[t][c][1][e + 1]};
      if (seg == 0) joined.m[wave][col] = w.m[t], joined.l[wave][col] = w.l[t];
      __syncthreads();
      for (int u = tid; u < 16 * (D / 4); u += kThreads) {
        const int r = u / (D / 4), d = u % (D / 4) * 4, row = 16 * t + r;
        if (row >= k.rows) break;
        float m = joined.m[0][r];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) m = fmaxf(m, joined.m[v][r]);
        float l = 0.f;
        float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          const float f = __builtin_amdgcn_exp2f(joined.m[v][r] - m);
          const float4 p = *reinterpret_cast<const float4*>(&joined.o[v][r][d]);
          l += f * joined.l[v][r];
          o.x += f * p.x, o.y += f * p.y, o.z += f * p.z, o.w += f * p.w;
        }
        if (whole) {
          const int j = (k.row0 + row) / g.heads;
          const int64_t out = static_cast<int64_t>(k.c0 + j) * g.a.n_q + h * g.heads + k.row0 + row - j * g.heads;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          store4(g.a.y + out * D + d, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
          if (g.a.lse != nullptr && d == 0)
            g.a.lse[out] = l > 0.f ? (m + __builtin_log2f(l)) * 0.69314718055994531f : -__builtin_inff();
        } else {
          *reinterpret_cast<float4*>(g.part_o + (slot * g.rows + row) * D + d) = o;
          if (d == 0) *reinterpret_cast<float2*>(g.part_ml + (slot * g.rows + row) * 2) = float2{m, l};
        }
      }
    }
    if (s0 == 0 && s1 < own) cut = {wg_of(at + own - 1, steps, wgs), h, k.c0, k.row0, k.rows};
    at += s1 - s0;
    if (s1 == own && h == n_kv - 1) ++item;
  }
  if (tid == 0) g.cut[wg] = cut;
}

// Joins the parts of the row blocks that were cut: one workgroup to a row of one, its threads
// in groups of D / 4 to every n-th part.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_join_kernel(Args g) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes;
  __shared__ float4 sum[kGroups][kLanes];
  __shared__ float top[kGroups], all[kGroups];
  const int w0 = blockIdx.x, row = blockIdx.y;
  const Cut k = g.cut[w0];
  const int w1 = k.last, h = k.head;
  if (w1 == 0 || row >= k.rows) return;

  const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  float m = kLowest, l = 0.f;
  float4 o = {0.f, 0.f, 0.f, 0.f};
  for (int w = w0 + grp; w <= w1; w += kGroups) {
    const int64_t at = (2 * static_cast<int64_t>(w) + (w == w0 ? 1 : 0)) * g.rows + row;
    const float2 ml = *reinterpret_cast<const float2*>(g.part_ml + at * 2);
    const float4 p = *reinterpret_cast<const float4*>(g.part_o + at * D + d);
    const float now = fmaxf(m, ml.x), f = __builtin_amdgcn_exp2f(m - now), e = __builtin_amdgcn_exp2f(ml.x - now);
    m = now;
    l = l * f + ml.y * e;
    o.x = o.x * f + p.x * e, o.y = o.y * f + p.y * e, o.z = o.z * f + p.z * e, o.w = o.w * f + p.w * e;
  }
  sum[grp][d / 4] = o;
  if (d == 0) top[grp] = m, all[grp] = l;
  __syncthreads();
  if (grp != 0) return;
  for (int v = 0; v < kGroups; ++v) m = fmaxf(m, top[v]);
  l = 0.f;
  o = float4{0.f, 0.f, 0.f, 0.f};
  for (int v = 0; v < kGroups; ++v) {
    const float e = __builtin_amdgcn_exp2f(top[v] - m);
    const float4 p = sum[v][d / 4];
    l += all[v] * e;
    o.x += p.x * e, o.y += p.y * e, o.z += p.z * e, o.w += p.w * e;
  }
  const int j = (k.row0 + row) / g.heads;
  const int64_t out = static_cast<int64_t>(k.c0 + j) * g.a.n_q + h * g.heads + k.row0 + row - j * g.heads;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  store4(g.a.y + out * D + d, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (g.a.lse != nullptr && d == 0)
    g.a.lse[out] = l > 0.f ? (m + __builtin_log2f(l)) * 0.69314718055994531f : -__builtin_inff();
}

// Rows of a row block: 16, 32 or 64, as many as a sequence's new tokens fill.
Plan plan_of(int64_t T, int64_t B, int n_q, int n_kv, int head_dim, int max_q) {
  const int64_t heads = n_q / n_kv;
  const int64_t most = max_q > 0 ? max_q * heads : (T * heads + B - 1) / B;
  Plan p;
  p.nq = most <= 16 ? 1 : most <= 32 ? 2 : 4;
  p.per_sequence = max_q > 0 && max_q * heads <= 16 * p.nq && B <= kListed;
  p.items = static_cast<int>(p.per_sequence ? B : T * heads / (16 * p.nq) + std::min(T, B));
  p.join_rows = static_cast<int>(max_q > 0 ? std::min<int64_t>(most, 16 * p.nq) : 16 * p.nq);
  p.wgs = p.nq == 4 || head_dim == 256 ? 512 : 1024;
  return p;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Space {
  size_t count, first, before, seq, part_o, part_ml, cut, all;
  Space(const Plan& p, int64_t B, int head_dim) {
    const size_t rows = static_cast<size_t>(p.wgs) * 2 * 16 * p.nq;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t here = at;
      at += up256(bytes);
      return here;
    };
    count = take(4);
    first = take(static_cast<size_t>(B) * 4);
    before = take((static_cast<size_t>(p.items) + 1) * 4);
    seq = take(static_cast<size_t>(p.items) * 4);
    part_o = take(rows * head_dim * 4);
    part_ml = take(rows * 8);
    cut = take(static_cast<size_t>(p.wgs) * sizeof(Cut));
    all = at;
  }
};

template <int D, int G>
void launch(const Args& g, const Plan& p, hipStream_t stream) {
  if (p.nq == 1)
    kv4_attention_kernel<D, G, 1><<<g.wgs, kThreads, 0, stream>>>(g);
  else if (p.nq == 2)
    kv4_attention_kernel<D, G, 2><<<g.wgs, kThreads, 0, stream>>>(g);
  else
    kv4_attention_kernel<D, G, 4><<<g.wgs, kThreads, 0, stream>>>(g);
  const dim3 grid(static_cast<unsigned>(p.wgs), static_cast<unsigned>(p.join_rows));
  kv4_join_kernel<D><<<grid, kThreads, 0, stream>>>(g);
}

template <int D>
void launch_group(const Args& g, const Plan& p, hipStream_t stream) {
  if (g.c.group == 32)
    launch<D, 32>(g, p, stream);
  else if (g.c.group == 64)
    launch<D, 64>(g, p, stream);
  else if constexpr (D >= 128)
    launch<D, 128>(g, p, stream);
}

}  // namespace

size_t kv4_attention_bytes(int64_t T, int64_t B, int n_q, int n_kv, int head_dim, int max_q) {
  return Space(plan_of(T, B, n_q, n_kv, head_dim, max_q), B, head_dim).all;
}

hipError_t launch_kv4_attention(const Kv4Attention& a, const ln_kv4_cache& c, void* workspace, hipStream_t stream) {
  const Plan p = plan_of(a.T, a.B, a.n_q, c.n_kv, c.head_dim, a.max_q);
  const Space sp(p, a.B, c.head_dim);
  auto* ws = static_cast<uint8_t*>(workspace);
  Args g;
  g.a = a;
  g.c = c;
  g.heads = a.n_q / c.n_kv;
  g.rows = 16 * p.nq;
  g.tiles_per_page = c.page_size / kTile;
  g.page_inv = static_cast<uint32_t>(((uint64_t(1) << 32) + g.tiles_per_page - 1) / g.tiles_per_page);
  g.scale2 = a.scale * 1.4426950408889634f;
  g.wgs = p.wgs;
  g.items = p.items;
  g.per_sequence = p.per_sequence;
  g.count = reinterpret_cast<int*>(ws + sp.count);
  g.first = reinterpret_cast<int*>(ws + sp.first);
  g.before = reinterpret_cast<int*>(ws + sp.before);
  g.seq = reinterpret_cast<int*>(ws + sp.seq);
  g.part_o = reinterpret_cast<float*>(ws + sp.part_o);
  g.part_ml = reinterpret_cast<float*>(ws + sp.part_ml);
  g.cut = reinterpret_cast<Cut*>(ws + sp.cut);
  if (!p.per_sequence) kv4_plan_kernel<<<1, kPlanThreads, 0, stream>>>(g);
  if (c.head_dim == 64)
    launch_group<64>(g, p, stream);
  else if (c.head_dim == 128)
    launch_group<128>(g, p, stream);
  else
    launch_group<256>(g, p, stream);
  return hipGetLastError();
}

}  // namespace lnf4
