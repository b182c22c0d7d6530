// Attention over the paged 4-bit cache (gfx950). Layout and definitions: kv4.h.
//
//     y = sum_t p_t v_t / sum_t p_t,   p_t = 2^(c q.k_t - m),   c = scale log2 e
// in one pass over the keys with a running m. The matrix instruction multiplies codes, which widen
// to bf16 exactly; steps and least values are applied to its 16 x 16 results:
//     q.k_t  = sum_g s_tg (q_g . c_tg) + lo_tg sum(q_g)
//     y_g    = sum_t (p_t s_tg) (c_tg - 8) + sum_t p_t (lo_tg + 8 s_tg)
// (around 8 the rounding of p s to bf16 multiplies the deviation from the middle of the range,
// not the value; sum_t p_t s_tg over the rounded products is one more instruction against ones).
//
// A wave works on tiles of 32 keys, alone: keys are the rows of the first product and queries
// its columns (16 a tile: the tokens of a sequence times the query heads of a key head), so that
// a lane's results are eight keys of one query. That is the operand of the second product as it
// is, whose rows are elements of the head: nothing moves between lanes in a tile, and codes
// reach the lanes that multiply them straight from global memory. m is raised only when a score
// passes it by 8 (a vote); p then stays below 2^8, which costs no accuracy, and the cross-lane
// maximum and the rescaling drop out of most tiles.
//
// Row blocks, up to 16 NQ rows of one sequence and key head, are laid end to end in units of the
// time they take, and each worker has an equal share of that line, whatever the sequences'
// lengths. A worker is a workgroup, whose four waves take every fourth tile and join in LDS, or,
// where row blocks are many and short, a wave. A row block that is cut is written as float32
// parts, which a second launch joins in order.
//
// What bounds it: with few rows the loads of this pattern and the vector units, by turns (64
// sequences of up to 16384 keys, 554 MB: 114 us; when the kernel took 150, its loads alone took 113
// and its arithmetic alone 110; the vector units issue in 55 % of the CUs' cycles, the matrix units work
// in 15 %). Many rows are bound by the vector units, which overlap little with the matrix units at two
// waves a SIMD (512 tokens against up to 16384 keys: 252 us, 546 TFLOP/s, 70 % and 29 %; prompts of 2500
// tokens 78 % and 26 %).
// Measured and not kept, each against the build of its time: codes as 16 + c by shifts and masks, in
// place of the conversion (64 sequences 128 -> 159 us); row blocks of 16 rows only (the chunk of
// 512 tokens 1496 us, 261 with larger ones); twice the workers (1 x 131071 keys 46 -> 59 us).
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
constexpr float kBar = 8.f;           // p stays below 2^8
constexpr uint32_t kNoNumber = 0x7FC07FC0u;  // a step and a least value
constexpr int kListed = 512;          // row blocks whose units are summed in LDS

// 16-row tiles of a row block at most, and the waves a SIMD that the registers are cut for
// (workgroups a CU, then): as many as need no scratch memory, but for four registers of <64, 64, 4>
// with workgroups as workers. 48 rows of heads of 128 spill 24 to 156.
constexpr int most_nq(int D, int G) { return D == 64 ? (G == 64 ? 4 : 2) : D == 128 ? 2 : 1; }
constexpr int waves_of(int D, int G, int NQ, bool SOLO) {
  if (D == 64) return NQ == 1 ? 4 : NQ == 2 && (SOLO || G == 64) ? 3 : 2;
  if (D == 128 && NQ == 1) return 3;
  return 2;
}

// A value that all lanes share, as one scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
  return (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32))) << 32) | lo;
}

// Memory that the kernel reading it does not write: a read at a shared place is a scalar one, and is not
// counted with the loads of codes. (The lists of row blocks are written by the launch before; the scalar
// cache is only sure to see that from the next launch on.)
typedef const __attribute__((address_space(4))) int32_t* Const;

struct Plan {
  bool solo;         // workers are waves, not workgroups
  int workers;
  int items;         // row blocks at most
  int in_seq;        // row blocks of a sequence, where workgroups sum the units themselves; else 0
  int nq;            // 16-row tiles of a row block
  int join_rows;     // rows of one at most
  bool whole;        // a worker to each row block and head
  bool by_head;      // cuts are listed by row block and head, not by worker
  int cuts;
};

// Units of time: of a step, of one where 16 rows do (measured 5 : 2 of 64 rows, 3 : 2 of 32; one set
// for all head widths and groups), of a row block itself. tiles: a step's.
struct Cost {
  int tiles, step, step16, block;
};

// A row block of a head that begins in worker `begun`'s share and goes on in others', the last of
// them `last` (0: there is none).
struct alignas(32) Cut {
  int begun, last, head, c0, row0, rows;
};

struct Args {
  Kv4Attention a;
  ln_kv4_cache c;
  int heads;          // query heads of a key head
  int rows;           // of a row block, 16 NQ
  int tiles_per_page;
  uint32_t page_inv;  // 2^32 / tiles_per_page, rounded up
  float scale2;       // scale log2 e
  int workers, items;
  int whole;          // a worker to each row block and head, which nothing cuts
  int in_seq;         // row blocks of every sequence, which workgroups then list themselves; 0: seq lists them
  Cost cost;
  // workspace: first[b] = row blocks before sequence b, before[i] = steps before row block i of
  // one key head, before[n] all of them, seq[i] its sequence; the parts; a workgroup's cut
  int *count, *first, *seq;
  int64_t* before;
  float *part_o, *part_ml;
  Cut* cut;      // of every worker, of which one at most begins what it does not end; or (by_head) of every
  int by_head;   // row block and head, where those are fewer
};

// A row block: rows [row0, row0 + rows) of a sequence's n_b heads rows, keys [lo, hi) that any
// of them sees.
struct Block {
  int b, c0, n, len, row0, rows, lo, hi;
  // The time of a row block in units: of each step of g.step key tiles, and of what it takes besides
  // (its place, its queries, its output: 2 to 4 us, which is two or three steps. Without it the workers
  // with the shortest sequences ended last, 96 x 40 heads 168 us, not 106).
  __device__ __forceinline__ int per_step(const Cost& c) const { return rows <= 16 ? c.step16 : c.step; }
  __device__ __forceinline__ int64_t units(const Cost& c) const {
    const int steps = ((hi + kTile - 1) / kTile - lo / kTile + c.tiles - 1) / c.tiles;
    return c.block + static_cast<int64_t>(steps) * per_step(c);
  }
  // The first step that begins at unit x or behind it.
  __device__ __forceinline__ int step_at(int64_t x, const Cost& c) const {
    const int u = per_step(c);
    return x <= c.block ? 0 : static_cast<int>((x - c.block + u - 1) / u);
  }
};

__device__ __forceinline__ void seq_rows(const Kv4Attention& a, int b, int& c0, int& n) {
  if (a.cu_q == nullptr) {
    c0 = b, n = 1;
  } else {
    const Const cu = (Const)a.cu_q;
    c0 = min(max(cu[b], 0), a.T);
    n = min(max(cu[b + 1], c0), a.T) - c0;
  }
}

__device__ __forceinline__ Block make_block(const Args& g, int b, int rb) {
  Block k;
  k.b = b;
  seq_rows(g.a, b, k.c0, k.n);
  k.len = min(max(((Const)g.a.lens)[b], 0), g.a.max_pages * g.c.page_size);
  k.row0 = rb * g.rows;
  k.rows = min(g.rows, k.n * g.heads - k.row0);
  const int j0 = k.row0 / g.heads, j1 = (k.row0 + max(k.rows, 1) - 1) / g.heads;
  k.hi = max(k.len - k.n + j1 + 1, 0);
  k.lo = g.a.window > 0 ? max(k.len - k.n + j0 + 1 - g.a.window, 0) : 0;
  if (k.rows <= 0 || k.lo >= k.hi) k.lo = k.hi = 0;
  return k;
}

template <typename V>
__device__ __forceinline__ V wave_scan(V v, V most) {
  const int lane = threadIdx.x & 63;
  v = min(v, most);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const V o = __shfl_up(v, d);
    if (lane >= d) v = min(v + o, most);
  }
  return v;
}

// Inclusive sum of v over the workgroup's threads, all the sum, both held at `most` (below 2^30 where
// V is int). part: one place a wave.
template <int WAVES, typename V>
__device__ __forceinline__ V block_scan(V v, V* part, V& all, V most) {
  const int wave = threadIdx.x >> 6;
  v = wave_scan(v, most);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) part[wave] = v;
  __syncthreads();
  V before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before = min(before + (w < wave ? part[w] : V(0)), most);
    all = min(all + part[w], most);
  }
  return min(v + before, most);
}

// The number of entries of the rising list at[0 .. n) that are <= x, less one.
template <typename V>
__device__ __forceinline__ int place_of(const V* at, int n, int64_t x, int64_t times) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] * times <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Worker w's share begins at unit share_of(w) of all units; the worker that has unit x. (Units are
// fewer than 2^36 5 LN_KV4_MAX_HEADS and workers than 2^13: products stay below 2^62.)
__device__ __forceinline__ int64_t share_of(int w, int64_t units, int workers) { return w * units / workers; }
__device__ __forceinline__ int worker_of(int64_t x, int64_t units, int workers) {
  return static_cast<int>(((x + 1) * workers - 1) / units);
}
__device__ __forceinline__ int sharing(int64_t units, int workers) {
  return static_cast<int>(min(static_cast<int64_t>(workers), units));
}

constexpr int64_t kMostUnits = int64_t(1) << 60;

// Row blocks and their units, of ragged sequences of any length: one workgroup.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void kv4_plan_kernel(Args g) {
  __shared__ int64_t part[kPlanThreads / 64];
  int* counts = reinterpret_cast<int*>(part);
  const int tid = threadIdx.x;
  int items = 0, all;
  for (int b0 = 0; b0 < g.a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int c0, n = 0;
    if (b < g.a.B) seq_rows(g.a, b, c0, n);
    const int mine = (n * g.heads + g.rows - 1) / g.rows;
    const int upto = block_scan<kPlanThreads / 64>(mine, counts, all, g.items);
    if (b < g.a.B) g.first[b] = min(items + max(upto - mine, 0), g.items);
    items = min(items + all, g.items);  // (more only if cu_q does not rise)
  }
  __threadfence_block();
  __syncthreads();
  int64_t units = 0, sum;
  for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int64_t mine = 0;
    int b = 0;
    if (i < items) {
      b = place_of(g.first, g.a.B, i, 1);
      mine = make_block(g, b, i - g.first[b]).units(g.cost);
    }
    const int64_t upto = units + block_scan<kPlanThreads / 64>(mine, part, sum, kMostUnits);
    if (i < items) g.before[i + 1] = upto, g.seq[i] = b;
    units += sum;
  }
  if (tid == 0) g.before[0] = 0, *g.count = items;
}

// Eight codes as bf16, exactly: a byte c of 0 .. 15 is c 2^-9 in E4M3.
__device__ __forceinline__ uint4 wide_codes(uint32_t lo, uint32_t hi) {
  auto two = [](uint32_t v, auto upper) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, decltype(upper)::value));
  };
  return uint4{two(lo, std::false_type{}), two(lo, std::true_type{}), two(hi, std::false_type{}),
               two(hi, std::true_type{})};
}

// The steps of a wave's tile, and its least values or (of values) those of code 8, in LDS: they
// come as one word a lane, widen there once, and are read as four keys' at a time, so that
// registers hold them only while they are used. Keys' are in units of 2^x's argument.
template <int NG>
struct Scales {
  float step[2][NG][kTile], base[2][NG][kTile];  // [keys, values]
};

// What the lanes of a wave wrote to LDS above is there for all of them below, and what they read above
// is not written before. (The LDS serves a wave's accesses in their order, so this is the compiler's
// order alone, and no instruction.)
__device__ __forceinline__ void wave_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

template <int D, int G, int NQ>
struct Wave {
  static constexpr int C = D / 32, NG = D / G, CG = G / 32;
  static constexpr int NP = NG < 2 ? 1 : NG / 2;  // words of scales a lane loads
  static constexpr int NZ = (NG + 3) / 4;

  struct alignas(D / 8 < 16 ? D / 8 : 16) Words {
    uint32_t w[C];
  };
  // A tile's codes and scales, of keys or of values. With one group a row the word of scales that
  // comes with the keys is a key's in the lower lanes and a value's in the upper ones.
  struct Raw {
    Words w[2];
    uint32_t p[NP];
  };

  uint4 q[NQ][C];
  Scales<NG>* scales;
  float q_sum[NQ][NG];      // sum of a query's group, in its lanes
  int first[NQ], last[NQ];  // the keys [first, last) that the lane's query sees
  int all_lo, all_hi;       // the keys that every row sees
  f32x4_t o[NQ][C][2];
  f32x4_t z[NQ][NZ];        // sum of the rounded p s, four groups in turn in a result's rows
  float mid[NQ][NG], l[NQ];
  float m[NQ];              // what is subtracted of scores
  float bar[NQ];            // the score that raises it
  float x[NQ][2][4];        // a tile's scores, m subtracted

  __device__ __forceinline__ void begin(const Args& g, const Block& k, int h) {
    const int lane = threadIdx.x & 63, col = lane & 15, seg = lane >> 4;
    // every row sees what the first does, from where the last one's window begins
    all_hi = max(k.len - k.n + k.row0 / g.heads + 1, 0);
    all_lo = g.a.window > 0 ? max(k.len - k.n + (k.row0 + max(k.rows, 1) - 1) / g.heads + 1 - g.a.window, 0) : 0;
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
    }
    const uint4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = i * CG; c < (i + 1) * CG; ++c) s = mfma16(ones, q[t][c], s);
        q_sum[t][i] = s[0];
        mid[t][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < NZ; ++i) z[t][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) o[t][c][0] = o[t][c][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      m[t] = l[t] = 0.f;
      bar[t] = kLowest;
    }
  }

  // row: the tile's first token in its page and head, counted over all pages and heads; par: the
  // same of its scales.
  static __device__ __forceinline__ void load_keys(const Args& g, int64_t row, int64_t par, Raw& r) {
    const int lane = threadIdx.x & 63, col = lane & 15, seg = lane >> 4;
    load_codes(g.c.k_codes + row * (D / 2), col * (D / 2) + seg * (D / 8), 16 * (D / 2), r);
    load_scales(NG == 1 && lane >= kTile ? g.c.v_scales : g.c.k_scales, par, g.c.page_size, r);
  }
  static __device__ __forceinline__ void load_values(const Args& g, int64_t row, int64_t par, Raw& r) {
    const int lane = threadIdx.x & 63, col = lane & 15, seg = lane >> 4;
    load_codes(g.c.v_codes + row * (D / 2), seg * (2 * D) + col * (D / 8), 8 * D, r);
    if constexpr (NG > 1) load_scales(g.c.v_scales, par, g.c.page_size, r);
  }
  static __device__ __forceinline__ void load_codes(const uint8_t* codes, int at, int half, Raw& r) {
#pragma unroll
    for (int s = 0; s < 2; ++s) r.w[s] = *reinterpret_cast<const Words*>(codes + s * half + at);
  }
  static __device__ __forceinline__ void load_scales(const uint16_t* scales, int64_t par, int page_size, Raw& r) {
    const int lane = threadIdx.x & 63;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(scales) + par + lane % kTile;
    if constexpr (NG == 1) {
      r.p[0] = *from;
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) r.p[i] = from[(2 * i + lane / kTile) * page_size];
    }
  }
  // The keys of a tile, a bit each, whose values have a step or least value that is infinite or no
  // number. Where some row does not see them they must not reach its sums, in which their weight is 0:
  // their scales become 0, and the least values of their keys no numbers, so that the rows that see
  // them have no numbers (the others' scores are replaced).
  static __device__ __forceinline__ uint32_t improper(const Raw& keys, const Raw& values) {
    uint64_t bad = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t w = NG == 1 ? keys.p[i] : values.p[i];
      bad |= __ballot((w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u);
    }
    return static_cast<uint32_t>(bad >> 32) | (NG == 1 ? 0u : static_cast<uint32_t>(bad));
  }
  // Keys outside [lo, hi), which no row sees, may have any scales too: those of their values become 0.
  __device__ __forceinline__ void put_key_scales(const Raw& r, int key0, int lo, int hi, float scale2, uint32_t bad) {
    const int lane = threadIdx.x & 63, key = key0 + lane % kTile;
    const bool is_bad = (bad >> (lane % kTile)) & 1;
    if constexpr (NG == 1) {
      const bool value = lane >= kTile;
      put(lane, value && (key < lo || key >= hi || is_bad) ? 0u : is_bad ? kNoNumber : r.p[0], value ? 1.f : scale2,
          value ? 8.f : 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) put(64 * i + lane, is_bad ? kNoNumber : r.p[i], scale2, 0.f);
    }
  }
  __device__ __forceinline__ void put_value_scales(const Raw& r, int key0, int lo, int hi, uint32_t bad) {
    if constexpr (NG > 1) {
      const int lane = threadIdx.x & 63, key = key0 + lane % kTile;
      const bool zero = key < lo || key >= hi || ((bad >> (lane % kTile)) & 1);
#pragma unroll
      for (int i = 0; i < NP; ++i) put(NG * kTile + 64 * i + lane, zero ? 0u : r.p[i], 1.f, 8.f);
    }
  }
  __device__ __forceinline__ void put(int at, uint32_t word, float times, float code) {
    const float step = __uint_as_float(word << 16), least = __uint_as_float(word & 0xFFFF0000u);
    (&scales->step[0][0][0])[at] = step * times;
    (&scales->base[0][0][0])[at] = __builtin_fmaf(code, step, least) * times;
  }

  // Four keys' floats.
  static __device__ __forceinline__ void four(const float* from, float (&v)[4]) {
    const float4 p = *reinterpret_cast<const float4*>(from);
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
  }

  // The scores of a tile's keys, of NT tiles of queries.
  template <int NT>
  __device__ __forceinline__ void score(const Raw& r) {
    const int seg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        f32x4_t acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = i * CG; c < (i + 1) * CG; ++c) {
          const uint32_t w = r.w[s].w[c];
          const uint4 wide = wide_codes(w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t] = mfma16(wide, q[t][c], acc[t]);
        }
        float step[4], least[4];
        four(&scales->step[0][i][16 * s + 4 * seg], step);
        four(&scales->base[0][i][16 * s + 4 * seg], least);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float b = __builtin_fmaf(least[e], q_sum[t][i], i == 0 ? -m[t] : x[t][s][e]);
            x[t][s][e] = __builtin_fmaf(step[e], acc[t][e], b);
          }
      }
    }
    // Nothing that reads the keys comes after this and no load before (else the next keys are
    // loaded into other registers, and moves at the tile's end wait for them).
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        asm volatile("" : "+v"(x[t][s][0]), "+v"(x[t][s][1]), "+v"(x[t][s][2]), "+v"(x[t][s][3]) : : "memory");
  }

  // Some row does not see some of the keys key0 .. key0 + 31, and no row those below lo.
  template <int NT>
  __device__ __forceinline__ void hide(int key0, int lo) {
    const int seg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int key = key0 + 16 * (e >> 2) + 4 * seg + (e & 3);
        if (key < max(first[t], lo) || key >= last[t]) x[t][e >> 2][e & 3] = -__builtin_inff();
      }
  }
  // The tile's part of the sums.
  template <int NT>
  __device__ __forceinline__ void sum(const Raw& r) {
    const int seg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top = x[t][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[t][e >> 2][e & 3]);
      if (__any(top > bar[t])) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // what is subtracted rises by the tile's largest score where that passes the bar (a query's
        // sums do not depend on its neighbours); of a query's first keys (its sums are 0) it goes
        // to their largest, which may lie far below 0
        const bool new_query = bar[t] != kBar;
        const float was = m[t];
        m[t] += new_query ? (top < kLowest ? 0.f : top) : top > kBar ? top : 0.f;
        bar[t] = new_query && top < kLowest ? kLowest : kBar;
        const float rise = m[t] - was, f = new_query ? 1.f : __builtin_amdgcn_exp2f(-rise);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[t][e >> 2][e & 3] -= rise;
        l[t] *= f;
#pragma unroll
        for (int i = 0; i < NG; ++i) mid[t][i] *= f;
#pragma unroll
        for (int i = 0; i < NZ; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][i][e] *= f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][c][0][e] *= f, o[t][c][1][e] *= f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& v = x[t][e >> 2][e & 3];
        v = __builtin_amdgcn_exp2f(v);
        l[t] += v;
      }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      // group i's sum goes to the rows that are i modulo four
      const uint32_t one = NG == 1 || (threadIdx.x & 3) == i % 4 ? 0x3F803F80u : 0u;
      const uint4 ones = {one, one, one, one};
      float step[2][4], centre[2][4];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        four(&scales->step[1][i][16 * s + 4 * seg], step[s]);
        four(&scales->base[1][i][16 * s + 4 * seg], centre[s]);
      }
      uint4 p[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = x[t][e >> 2][e & 3];
          w[e] = v * step[e >> 2][e & 3];
          mid[t][i] = __builtin_fmaf(v, centre[e >> 2][e & 3], mid[t][i]);
        }
        p[t] = uint4{pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7])};
        z[t][i / 4] = mfma16(ones, p[t], z[t][i / 4]);
      }
#pragma unroll
      for (int c = i * CG; c < (i + 1) * CG; ++c) {
        // Products come in this order (an empty statement, no instruction: else every code is
        // widened ahead of all of them, into registers that more waves need)
        uint32_t w0 = r.w[0].w[c], w1 = r.w[1].w[c];
        if (c == 0) {
          asm volatile("" : "+v"(w0), "+v"(w1));
        } else if constexpr (NT == 1) {
          asm volatile("" : "+v"(w0), "+v"(w1), "+v"(o[0][c - 1][0]), "+v"(o[0][c - 1][1]));
        } else {
#pragma unroll
          for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(w0), "+v"(w1), "+v"(o[t][c - 1][0]), "+v"(o[t][c - 1][1]));
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 a = wide_codes((w0 >> (4 * half)) & 0x0F0F0F0Fu, (w1 >> (4 * half)) & 0x0F0F0F0Fu);
#pragma unroll
          for (int t = 0; t < NT; ++t) o[t][c][half] = mfma16(a, p[t], o[t][c][half]);
        }
      }
    }
  }

  // The wave's tiles t, t + STEP, .. below t_end of a key head. A tile's keys are loaded while the
  // values of the one before are multiplied, its values while its keys are, each into the registers
  // that were just read.
  template <int NT, int STEP>
  __device__ __forceinline__ void tiles(const Args& g, const Block& k, int h, int t, int t_end) {
    const Const table = (Const)(g.a.block_table + static_cast<int64_t>(k.b) * g.a.max_pages);
    auto slot_of = [&](int t) { return g.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(t, g.page_inv)); };
    // a tile's place in the cache; of a page that does not exist page 0, with its keys hidden
    int64_t row, par;
    bool gone;
    auto place = [&](int t, int slot, int page) {
      gone = page < 0 || page >= g.c.n_pages;
      const int64_t ph = static_cast<int64_t>(gone ? 0 : page) * g.c.n_kv + h;
      const int tok = (t - slot * g.tiles_per_page) * kTile;
      row = ph * g.c.page_size + tok;
      par = ph * NG * g.c.page_size + tok;
    };
    Raw keys, values;
    const int slot = slot_of(t);
    place(t, slot, table[slot]);
    load_keys(g, row, par, keys);
    load_values(g, row, par, values);
    int next_slot = slot_of(min(t + STEP, t_end - 1)), page = table[next_slot];
    bool more;
    do {
      const int key0 = t * kTile, lo = gone ? key0 + kTile : k.lo;
      const bool border = gone || key0 < all_lo || key0 + kTile > all_hi;
      t += STEP;
      more = t < t_end;
      // A tile's second half goes first where waves meet: the first one (the older wave's, at equal
      // priority) leaves the younger wave behind, to end alone (a chunk of 512 tokens 263 -> 251 us)
      __builtin_amdgcn_s_setprio(0);
      const uint32_t bad = border ? improper(keys, values) : 0;
      wave_in_order();
      put_key_scales(keys, key0, lo, k.hi, g.scale2, bad);
      wave_in_order();
      score<NT>(keys);
      if (more) place(t, next_slot, page);  // (the last tile is loaded again: counted waits need no two ways)
      load_keys(g, row, par, keys);
      next_slot = slot_of(min(t + STEP, t_end - 1));
      page = table[next_slot];
      __builtin_amdgcn_s_setprio(1);
      put_value_scales(values, key0, lo, k.hi, bad);
      wave_in_order();
      if (border) hide<NT>(key0, lo);
      sum<NT>(values);
      load_values(g, row, par, values);
    } while (more);
    __builtin_amdgcn_s_setprio(0);
  }

  // The sums over the wave's lanes, centres applied: o holds sum p v of the tiles so far.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (bar[t] != kBar) m[t] = kLowest;
      l[t] += __shfl_xor(l[t], 16);
      l[t] += __shfl_xor(l[t], 32);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float c = mid[t][i];
        c += __shfl_xor(c, 16);
        c += __shfl_xor(c, 32);
        c = __builtin_fmaf(-8.f, z[t][i / 4][i % 4], c);
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

template <>
struct Joined<0> {};

// Where a row of a row block and head goes: y and lse, or a part.
struct Out {
  const Args& g;
  const Block& k;
  int h;
  bool whole;
  int64_t slot;

  // Four sums from element d on, of weights 2^(score - m) that add up to l.
  template <int D>
  __device__ __forceinline__ void put(int row, int d, float m, float l, const float4& o) const {
    if (whole) {
      const int j = (k.row0 + row) / g.heads;
      const int64_t out = static_cast<int64_t>(k.c0 + j) * g.a.n_q + h * g.heads + k.row0 + row - j * g.heads;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(g.a.y + out * D + d) =
          uint2{pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv)};
      if (g.a.lse != nullptr && d == 0)
        g.a.lse[out] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994531f;
    } else {
      *reinterpret_cast<float4*>(g.part_o + (slot * g.rows + row) * D + d) = o;
      if (d == 0) *reinterpret_cast<float2*>(g.part_ml + (slot * g.rows + row) * 2) = float2{m, l};
    }
  }
};

// SOLO: the waves are workers on their own, each with its share of tiles, and join nothing.
// Otherwise a workgroup is one, and its waves take every fourth tile of its share.
template <int D, int G, int NQ, bool SOLO>
__global__ __launch_bounds__(kThreads, waves_of(D, G, NQ, SOLO)) void kv4_attention_kernel(Args g) {
  typedef Wave<D, G, NQ> W;
  constexpr int C = D / 32, kStep = SOLO ? 1 : kWaves;
  __shared__ union {
    Scales<W::NG> scales[kWaves];   // in the loop over tiles
    Joined<SOLO ? 0 : D> joined;    // after it
  } space;
  auto& scales = space.scales;
  auto& joined = space.joined;
  __shared__ int64_t listed[kListed + 1];
  __shared__ int64_t part[kWaves];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63;
  const int col = lane & 15, seg = lane >> 4, n_kv = g.c.n_kv;

  // the units before every row block
  int items;
  const int64_t* before = nullptr;
  if (g.whole) {
    items = g.items;
  } else if (g.in_seq != 0) {
    items = g.a.B * g.in_seq;
    int64_t units = 0, all;
    for (int b0 = 0; b0 < items; b0 += kThreads) {
      const int i = b0 + tid;
      int64_t mine = 0;
      if (i < items) {
        const Block k = make_block(g, i / g.in_seq, i % g.in_seq);
        mine = k.row0 == 0 || k.rows > 0 ? k.units(g.cost) : 0;  // (sequences differ in rows)
      }
      const int64_t upto = units + block_scan<kWaves>(mine, part, all, kMostUnits);
      if (i < items) listed[i + 1] = upto;
      units += all;
    }
    if (tid == 0) listed[0] = 0;
    __syncthreads();
    before = listed;
  } else {
    items = *(Const)g.count;
    before = g.before;
  }
  const int64_t units = g.whole ? g.workers : uniform(before[items]) * n_kv;
  const int workers = sharing(units, g.workers), me = SOLO ? kWaves * blockIdx.x + wave : blockIdx.x;
  const bool writer = SOLO ? lane == 0 : tid == 0;
  if (me >= workers) {
    if (writer && !g.by_head) g.cut[me].last = 0;
    return;
  }
  const int64_t end = share_of(me + 1, units, workers);

  Cut cut = {0, 0, 0, 0, 0, 0};
  int64_t at = share_of(me, units, workers);
  int item = g.whole ? me / n_kv : uniform(place_of(before, items, at, n_kv));
  while (at < end) {
    const int64_t base = g.whole ? item : uniform(before[item]);
    const int64_t own = g.whole ? 1 : uniform(before[item + 1]) - base;  // units of the row block
    if (own == 0) {
      ++item;
      continue;
    }
    const int64_t in = at - base * n_kv;
    const int h = uniform((in | own) >> 32 ? static_cast<int>(in / own)
                                           : static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(own)));
    const int64_t u0 = in - h * own, u1 = min(own, u0 + end - at);
    const int b = g.in_seq != 0 ? item / g.in_seq : ((Const)g.seq)[item];
    Block k = make_block(g, b, item - (g.in_seq != 0 ? b * g.in_seq : ((Const)g.first)[b]));
    k.c0 = uniform(k.c0), k.n = uniform(k.n), k.len = uniform(k.len), k.row0 = uniform(k.row0);
    k.rows = uniform(k.rows), k.lo = uniform(k.lo), k.hi = uniform(k.hi);
    const int s0 = uniform(k.step_at(u0, g.cost)), s1 = g.whole ? 1 << 20 : uniform(k.step_at(u1, g.cost));

    W w;
    w.scales = &scales[wave];
    w.begin(g, k, h);
    const int t_first = k.lo / kTile + kStep * s0 + (SOLO ? 0 : wave);
    const int t_end = min((k.hi + kTile - 1) / kTile, k.lo / kTile + kStep * s1);
    if (t_first < t_end) {
      if (NQ > 1 && k.rows <= 16)
        w.template tiles<1, kStep>(g, k, h, t_first, t_end);
      else
        w.template tiles<NQ, kStep>(g, k, h, t_first, t_end);
    }
    w.finish();

    // Whole: y. A part: slot 1 of the worker where the row block begins in its share, 0 where
    // it began before.
    const bool whole = u0 == 0 && u1 == own;
    const int64_t slot = 2 * static_cast<int64_t>(me) + (u0 == 0 ? 1 : 0);
    const Out to = {g, k, h, whole, slot};
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (16 * t >= k.rows) break;
      if constexpr (SOLO) {
        const int row = 16 * t + col;
        if (row < k.rows) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              to.template put<D>(row, 32 * c + 8 * seg + 2 * e, w.m[t], w.l[t],
                                 float4{w.o[t][c][0][e], w.o[t][c][1][e], w.o[t][c][0][e + 1], w.o[t][c][1][e + 1]});
        }
      } else {
        __syncthreads();
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
          to.template put<D>(row, d, m, l, o);
        }
      }
    }
    if constexpr (!SOLO) __syncthreads();
    if (u0 == 0) {
      const bool goes_on = u1 < own;
      if (goes_on) cut = {me, worker_of(at + own - 1, units, workers), h, k.c0, k.row0, k.rows};
      if (g.by_head && writer) g.cut[static_cast<int64_t>(item) * n_kv + h] = goes_on ? cut : Cut{0, 0, 0, 0, 0, 0};
    }
    at += u1 - u0;
    if (u1 == own && h == n_kv - 1) ++item;
  }
  if (writer && !g.by_head && !g.whole) g.cut[me] = cut;
}

// Joins the parts of the row blocks that were cut, a few workgroups to a cut. Threads in
// groups of D / 4 have a row each where the parts are few (some workers' shares), or every n-th part
// of one row, four parts' loads in flight.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_join_kernel(Args g) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes;
  __shared__ float4 sum[kGroups][kLanes];
  __shared__ float top[kGroups], all[kGroups];
  const Cut k = g.cut[blockIdx.x];
  const int w0 = k.begun, w1 = k.last, h = k.head;
  if (w1 == 0) return;

  const int rows_at = w1 - w0 < 4 ? kGroups : 1;
  const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  const int own = grp % rows_at, turn = grp / rows_at, turns = kGroups / rows_at;
  for (int row0 = blockIdx.y * rows_at; row0 < k.rows; row0 += gridDim.y * rows_at) {
    const int row = row0 + own, from = min(row, k.rows - 1);
    float m = kLowest, l = 0.f;
    float4 o = {0.f, 0.f, 0.f, 0.f};
    for (int w = w0 + turn; w <= w1; w += 4 * turns) {
      float2 ml[4];
      float4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = min(w + i * turns, w1);
        const int64_t at = (2 * static_cast<int64_t>(v) + (v == w0 ? 1 : 0)) * g.rows + from;
        ml[i] = *reinterpret_cast<const float2*>(g.part_ml + at * 2);
        p[i] = *reinterpret_cast<const float4*>(g.part_o + at * D + d);
      }
      float now = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (w + i * turns > w1) ml[i] = float2{kLowest, 0.f}, p[i] = float4{0.f, 0.f, 0.f, 0.f};
        now = fmaxf(now, ml[i].x);
      }
      const float f = __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
      o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(ml[i].x - now);
        l += ml[i].y * e;
        o.x += p[i].x * e, o.y += p[i].y * e, o.z += p[i].z * e, o.w += p[i].w * e;
      }
    }
    if (turns > 1) {
      sum[grp][d / 4] = o;
      if (d == 0) top[grp] = m, all[grp] = l;
      __syncthreads();
      if (turn == 0) {
        for (int v = 0; v < kGroups; ++v) m = fmaxf(m, top[v]);
        l = 0.f;
        o = float4{0.f, 0.f, 0.f, 0.f};
        for (int v = 0; v < kGroups; ++v) {
          const float e = __builtin_amdgcn_exp2f(top[v] - m);
          const float4 p = sum[v][d / 4];
          l += all[v] * e;
          o.x += p.x * e, o.y += p.y * e, o.z += p.z * e, o.w += p.w * e;
        }
      }
      __syncthreads();
    }
    if (turn == 0 && row < k.rows) {
      Block b;
      b.c0 = k.c0, b.row0 = k.row0;
      const Out to = {g, b, h, true, 0};
      to.template put<D>(row, d, m, l, o);
    }
  }
}

// Workers are waves where there are row blocks enough that each has few parts. Workgroups -> waves:
// prompts of 2500 tokens 188 -> 135 us, 96 x 40 heads 122 -> 110; below the limit 1 x 131071 keys 41 ->
// 92, 64 sequences of 8 heads 114 -> 121. Several tokens below it go either way (8 of 16 sequences of 32
// query heads 45 -> 39, 4 of 64 sequences 39 -> 47).
bool solo_of(int64_t items, int n_kv) { return items * n_kv >= 1024; }

// Rows of a row block: 16, 32 or 64, as many as a sequence's new tokens fill; without a bound the
// average's.
Plan plan_of(int64_t T, int64_t B, int n_q, int n_kv, int head_dim, int max_q, int64_t max_len, int group) {
  const int64_t heads = n_q / n_kv;
  const int64_t most = max_q > 0 ? max_q * heads : (T * heads + B - 1) / B;
  Plan p;
  p.nq = std::min(most <= 16 ? 1 : most <= 32 ? 2 : 4, most_nq(head_dim, group));
  const int64_t blocks = (most + 16 * p.nq - 1) / (16 * p.nq);
  p.in_seq = max_q > 0 && B * blocks <= kListed ? static_cast<int>(blocks) : 0;
  p.items = static_cast<int>(p.in_seq != 0 ? B * blocks : T * heads / (16 * p.nq) + std::min(T, B));
  p.join_rows = static_cast<int>(max_q > 0 ? std::min<int64_t>(most, 16 * p.nq) : 16 * p.nq);
  p.solo = solo_of(p.items, n_kv);
  p.by_head = p.in_seq == 1;  // (the row blocks of others are known to the GPU only)
  p.workers = 256 * waves_of(head_dim, group, p.nq, p.solo) * (p.solo ? kWaves : 1);
  if (p.by_head && static_cast<int64_t>(p.items) * n_kv >= p.workers) p.by_head = false;
  p.cuts = p.by_head ? p.items * n_kv : p.workers;
  // Up to 512 keys are four tiles a wave, which take no longer than a second launch does (a token
  // after 500 keys, back-to-back calls: 12.0 us, 15.2 in two launches).
  p.whole = p.in_seq != 0 && !p.solo && max_len <= 512 && static_cast<int64_t>(p.items) * n_kv <= p.workers;
  if (p.whole) p.workers = p.items * n_kv, p.by_head = false, p.cuts = 0;
  return p;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Space {
  size_t count, first, before, seq, part_o, part_ml, cut, all;
  Space(const Plan& p, int64_t B, int head_dim) {
    const size_t rows = p.whole ? 0 : static_cast<size_t>(p.workers) * 2 * 16 * p.nq;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t here = at;
      at += up256(bytes);
      return here;
    };
    count = take(4);
    first = take(static_cast<size_t>(B) * 4);
    before = take((static_cast<size_t>(p.items) + 1) * 8);
    seq = take(static_cast<size_t>(p.items) * 4);
    part_o = take(rows * head_dim * 4);
    part_ml = take(rows * 8);
    cut = take(static_cast<size_t>(p.cuts) * sizeof(Cut));
    all = at;
  }
};

template <int D, int G>
void launch(const Args& g, const Plan& p, hipStream_t stream) {
  auto run = [&](auto nq) {
    constexpr int NQ = decltype(nq)::value;
    if constexpr (NQ <= most_nq(D, G)) {
      if (p.solo)
        kv4_attention_kernel<D, G, NQ, true><<<p.workers / kWaves, kThreads, 0, stream>>>(g);
      else
        kv4_attention_kernel<D, G, NQ, false><<<p.workers, kThreads, 0, stream>>>(g);
    }
  };
  if (p.nq == 1)
    run(std::integral_constant<int, 1>{});
  else if (p.nq == 2)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 4>{});
  if (p.whole) return;
  const int at_once = p.solo ? kThreads / (D / 4) : 1;  // rows of a workgroup
  const dim3 grid(static_cast<unsigned>(p.cuts), static_cast<unsigned>(std::min((p.join_rows + at_once - 1) / at_once, 8)));
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

size_t kv4_attention_bytes(int64_t T, int64_t B, int n_q, int n_kv, int head_dim, int max_q, int64_t max_len) {
  size_t most = 0;
  for (int group = 32; group <= 128; group *= 2)
    most = std::max(most, Space(plan_of(T, B, n_q, n_kv, head_dim, max_q, max_len, group), B, head_dim).all);
  return most;
}

hipError_t launch_kv4_attention(const Kv4Attention& a, const ln_kv4_cache& c, void* workspace, hipStream_t stream) {
  const Plan p = plan_of(a.T, a.B, a.n_q, c.n_kv, c.head_dim, a.max_q, static_cast<int64_t>(a.max_pages) * c.page_size, c.group);
  const Space sp(p, a.B, c.head_dim);
  auto* ws = static_cast<uint8_t*>(workspace);
  Args g;
  g.a = a;
  if (g.a.window >= 1 << 30) g.a.window = 0;  // (no sequence is longer)
  g.c = c;
  g.heads = a.n_q / c.n_kv;
  g.rows = 16 * p.nq;
  g.tiles_per_page = c.page_size / kTile;
  g.page_inv = static_cast<uint32_t>(((uint64_t(1) << 32) + g.tiles_per_page - 1) / g.tiles_per_page);
  g.scale2 = a.scale * kLog2E;
  g.workers = p.workers;
  g.by_head = p.by_head;
  g.whole = p.whole;
  g.items = p.items;
  g.in_seq = p.in_seq;
  const int tiles = p.solo ? 1 : kWaves;
  g.cost = p.nq == 1 ? Cost{tiles, 1, 1, 2} : p.nq == 2 ? Cost{tiles, 3, 2, 6} : Cost{tiles, 5, 2, 15};
  g.count = reinterpret_cast<int*>(ws + sp.count);
  g.first = reinterpret_cast<int*>(ws + sp.first);
  g.before = reinterpret_cast<int64_t*>(ws + sp.before);
  g.seq = reinterpret_cast<int*>(ws + sp.seq);
  g.part_o = reinterpret_cast<float*>(ws + sp.part_o);
  g.part_ml = reinterpret_cast<float*>(ws + sp.part_ml);
  g.cut = reinterpret_cast<Cut*>(ws + sp.cut);
  if (p.in_seq == 0) kv4_plan_kernel<<<1, kPlanThreads, 0, stream>>>(g);
  if (c.head_dim == 64)
    launch_group<64>(g, p, stream);
  else if (c.head_dim == 128)
    launch_group<128>(g, p, stream);
  else
    launch_group<256>(g, p, stream);
  return hipGetLastError();
}

}  // namespace lnf4
