// C ABI of the paged 4-bit cache of keys and values (declared in include/kv4.h).
//
// Every entry point validates its arguments on the host before touching HIP, so
// argument errors are reported without a GPU and nothing is enqueued on error.
#include <cmath>
#include <cstdint>

#include "api_check.h"
#include "kv4.h"
#include "kv4_launch.h"

namespace {

using namespace lnf4;

constexpr int64_t kMaxTokens = int64_t(1) << 24;  // below it: launches of fewer than 2^32 threads along x

int check_dims(int64_t page_size, int64_t n_kv, int32_t head_dim) {
  if (page_size < 1 || n_kv < 1 || head_dim < 1) return LN_EINVAL;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return LN_ESHAPE;
  if (page_size % 32 != 0 || page_size > LN_KV4_MAX_PAGE || n_kv > LN_KV4_MAX_HEADS) return LN_ESHAPE;
  return LN_OK;
}

int check_cache(const ln_kv4_cache* c) {
  if (c == nullptr || c->k_codes == nullptr || c->k_scales == nullptr || c->v_codes == nullptr || c->v_scales == nullptr)
    return LN_EINVAL;
  if (c->n_pages < 1) return LN_EINVAL;
  const int st = check_dims(c->page_size, c->n_kv, c->head_dim);
  if (st != LN_OK) return st;
  if ((c->group != 32 && c->group != 64 && c->group != 128) || c->head_dim % c->group != 0) return LN_ESHAPE;
  if (c->n_pages > kMaxDim || c->n_pages * c->page_size >= int64_t(1) << 40) return LN_ESHAPE;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
    return LN_EALIGN;
  return LN_OK;
}

// The four tensors of a cache.
void cache_spans(const ln_kv4_cache& c, Span (&s)[4]) {
  const size_t rows = static_cast<size_t>(c.n_pages) * c.page_size * c.n_kv;
  const size_t codes = rows * (c.head_dim / 2), scales = rows * (c.head_dim / c.group) * 4;
  s[0] = {c.k_codes, codes}, s[1] = {c.k_scales, scales}, s[2] = {c.v_codes, codes}, s[3] = {c.v_scales, scales};
}

// Bytes from the first to the last of T rows.
size_t strided(int64_t T, int64_t stride, int64_t row, size_t e) { return static_cast<size_t>((T - 1) * stride + row) * e; }

int check_attention(int64_t T, int64_t B, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t max_q, int64_t max_pages,
                    int64_t page_size) {
  if (T < 0 || B < 1 || n_q < 1 || max_q < 0 || max_pages < 1) return LN_EINVAL;
  const int st = check_dims(page_size, n_kv, head_dim);
  if (st != LN_OK) return st;
  if (n_q > LN_KV4_MAX_HEADS || n_q % n_kv != 0) return LN_ESHAPE;
  if (T >= kMaxTokens || T * n_q > int64_t(1) << 30 || B >= int64_t(1) << 20) return LN_ESHAPE;
  if (max_pages > (int64_t(1) << 30) / page_size) return LN_ESHAPE;
  if ((T * (n_q / n_kv) / 16 + B) * (max_pages * page_size / 32 + 2) >= int64_t(1) << 36) return LN_ESHAPE;
  return LN_OK;
}

}  // namespace

extern "C" {

int kv4_append(int64_t T, int32_t n_q, int dtype, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
               const void* v, int64_t v_stride, const float* cos, const float* sin, int64_t n_pos, int32_t rot_dim,
               int32_t interleaved, const int64_t* positions, const int64_t* slots, uint16_t* q_out,
               const ln_kv4_cache* cache, void* stream) {
  if (T < 0 || (dtype != LN_F32 && dtype != LN_BF16) || rot_dim < 0 || (interleaved != 0 && interleaved != 1))
    return LN_EINVAL;
  const int st = check_cache(cache);
  if (st != LN_OK) return st;
  const bool turned = rot_dim != 0;
  if ((cos != nullptr) != turned || (sin != nullptr) != turned || (turned && n_pos < 1)) return LN_EINVAL;
  if (rot_dim % 16 != 0 || rot_dim > cache->head_dim) return LN_ESHAPE;
  if (T >= kMaxTokens || (turned && n_pos > kMaxDim)) return LN_ESHAPE;
  if ((q == nullptr) != (q_out == nullptr) && T != 0) return LN_EINVAL;
  const bool with_q = q != nullptr;
  if (with_q && n_q < 1) return LN_EINVAL;
  if (with_q && n_q > LN_KV4_MAX_HEADS) return LN_ESHAPE;
  if (T == 0) return LN_OK;
  if (k == nullptr || v == nullptr || slots == nullptr || (turned && positions == nullptr)) return LN_EINVAL;
  const int64_t d = cache->head_dim, kv_row = cache->n_kv * d, q_row = with_q ? n_q * d : 0;
  const size_t e = dtype == LN_F32 ? 4 : 2;
  const int64_t unit = static_cast<int64_t>(16 / e), strides[3] = {with_q ? q_stride : 0, k_stride, v_stride};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < (i == 0 ? q_row : kv_row) || strides[i] > kMaxDim) return LN_ESHAPE;
    if (strides[i] % unit != 0) return LN_EALIGN;
  }
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cos) || !aligned16(sin) || !aligned16(q_out) ||
      !aligned16(positions) || !aligned16(slots))
    return LN_EALIGN;
  const size_t t = static_cast<size_t>(T), table = turned ? static_cast<size_t>(n_pos) * (rot_dim / 2) * 4 : 0;
  Span parts[4];
  cache_spans(*cache, parts);
  const Span outs[5] = {parts[0], parts[1], parts[2], parts[3], {q_out, t * q_row * 2}};
  const Span ins[7] = {{q, with_q ? strided(T, q_stride, q_row, e) : 0}, {k, strided(T, k_stride, kv_row, e)},
                       {v, strided(T, v_stride, kv_row, e)}, {cos, table}, {sin, table},
                       {turned ? positions : nullptr, t * 8}, {slots, t * 8}};
  if (any_alias(outs, 5, ins, 7)) return LN_EALIAS;
  const Kv4Append a = {T,   n_q,     q,           k,         v,     q_stride, k_stride, v_stride, cos,
                       sin, n_pos, rot_dim, interleaved != 0, positions, slots, q_out};
  return hip_status(launch_kv4_append(a, dtype == LN_BF16, *cache, static_cast<hipStream_t>(stream)));
}

int kv4_read(int64_t T, const int64_t* slots, const ln_kv4_cache* cache, int out_dtype, void* k, void* v,
             void* stream) {
  if (T < 0 || (out_dtype != LN_F32 && out_dtype != LN_BF16)) return LN_EINVAL;
  const int st = check_cache(cache);
  if (st != LN_OK) return st;
  if (T >= kMaxTokens) return LN_ESHAPE;
  if (T == 0) return LN_OK;
  if (slots == nullptr || (k == nullptr && v == nullptr)) return LN_EINVAL;
  if (!aligned16(slots) || !aligned16(k) || !aligned16(v)) return LN_EALIGN;
  const size_t t = static_cast<size_t>(T), bytes = t * cache->n_kv * cache->head_dim * (out_dtype == LN_F32 ? 4 : 2);
  Span parts[4];
  cache_spans(*cache, parts);
  const Span outs[2] = {{k, bytes}, {v, bytes}};
  const Span ins[5] = {parts[0], parts[1], parts[2], parts[3], {slots, t * 8}};
  if (any_alias(outs, 2, ins, 5)) return LN_EALIAS;
  return hip_status(launch_kv4_read(T, slots, *cache, out_dtype == LN_BF16, k, v, static_cast<hipStream_t>(stream)));
}

size_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t max_q,
                                     int64_t max_pages, int32_t page_size) {
  if (T == 0 || check_attention(T, B, n_q, n_kv, head_dim, max_q, max_pages, page_size) != LN_OK) return 0;
  return kv4_attention_bytes(T, B, n_q, n_kv, head_dim, max_q, max_pages * page_size);
}

int kv4_attention(int64_t T, int64_t B, int32_t n_q, const uint16_t* q, int64_t q_stride, const int32_t* cu_q,
                  int32_t max_q, const int32_t* lens, const int32_t* block_table, int64_t max_pages, int32_t window,
                  float scale, const ln_kv4_cache* cache, uint16_t* y, float* lse, void* workspace,
                  size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != LN_OK) return st;
  if (window < 0 || !std::isfinite(scale * kLog2E) || !(scale > 0.f)) return LN_EINVAL;
  st = check_attention(T, B, n_q, cache->n_kv, cache->head_dim, max_q, max_pages, cache->page_size);
  if (st != LN_OK) return st;
  if (cu_q == nullptr && T != B) return LN_ESHAPE;
  if (T == 0) return LN_OK;
  if (q == nullptr || lens == nullptr || block_table == nullptr || y == nullptr) return LN_EINVAL;
  const int64_t row = static_cast<int64_t>(n_q) * cache->head_dim;
  if (q_stride < row || q_stride > kMaxDim) return LN_ESHAPE;
  if (q_stride % 8 != 0 || !aligned16(q) || !aligned16(cu_q) || !aligned16(lens) || !aligned16(block_table) ||
      !aligned16(y) || !aligned16(lse))
    return LN_EALIGN;
  const int32_t bound = cu_q == nullptr ? 1 : max_q;
  const size_t need = kv4_attention_bytes(T, B, n_q, cache->n_kv, cache->head_dim, bound, max_pages * cache->page_size);
  if (workspace == nullptr || workspace_bytes < need) return LN_EWORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LN_EALIGN;
  const size_t t = static_cast<size_t>(T), b = static_cast<size_t>(B);
  Span parts[4];
  cache_spans(*cache, parts);
  const Span outs[3] = {{y, t * row * 2}, {lse, t * n_q * 4}, {workspace, need}};
  const Span ins[8] = {parts[0], parts[1], parts[2], parts[3], {q, strided(T, q_stride, row, 2)},
                       {cu_q, (b + 1) * 4}, {lens, b * 4}, {block_table, b * static_cast<size_t>(max_pages) * 4}};
  if (any_alias(outs, 3, ins, 8)) return LN_EALIAS;
  const Kv4Attention a = {static_cast<int>(T), static_cast<int>(B), n_q, q, q_stride, cu_q, bound, lens, block_table,
                          static_cast<int>(max_pages), window, scale, y, lse};
  return hip_status(launch_kv4_attention(a, *cache, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
