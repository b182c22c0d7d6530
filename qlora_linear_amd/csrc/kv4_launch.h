// Internal launchers of the paged 4-bit cache. Arguments are validated by kv4_api.hip;
// each launcher only enqueues work on `stream` and returns the hipGetLastError() of its
// launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv4.h"

namespace lnf4 {

struct Kv4Append {
  int64_t T;
  int n_q;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements
  const float *cos, *sin;
  int64_t n_pos;
  int rot_dim;
  bool interleaved;
  const int64_t *positions, *slots;
  uint16_t* q_out;
};
hipError_t launch_kv4_append(const Kv4Append& a, bool bf16, const ln_kv4_cache& c, hipStream_t stream);
hipError_t launch_kv4_read(int64_t T, const int64_t* slots, const ln_kv4_cache& c, bool bf16, void* k, void* v,
                           hipStream_t stream);

constexpr float kLog2E = 1.4426950408889634f;

struct Kv4Attention {
  int T, B, n_q;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* cu_q;
  int max_q;
  const int32_t *lens, *block_table;
  int max_pages, window;
  float scale;
  uint16_t* y;
  float* lse;
};
size_t kv4_attention_bytes(int64_t T, int64_t B, int n_q, int n_kv, int head_dim, int max_q, int64_t max_len);
hipError_t launch_kv4_attention(const Kv4Attention& a, const ln_kv4_cache& c, void* workspace, hipStream_t stream);

}  // namespace lnf4
