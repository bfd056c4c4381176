// Internal interface between the C entry points of the cache calls (rf_cache.cpp) and their
// kernels (rf_rope.hip, rf_attend.hip, rf_weight.hip, rf_evict.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rf_internal.h"

namespace rf {

// Host-side copy of rf_paged_batch.
struct Batch {
  const int32_t* tables;
  const int32_t* lengths;
  int64_t table_stride;
  int batch, max_len, page_size, num_pages, n_kv, hd;
};

// Rotation: angle of pair j in turns (revolutions) per position, the factor of cos and sin.
constexpr int kMaxPairs = 128;
struct RopeFreq {
  double turns[kMaxPairs];
  float m;
  int rot;                      // rotary_dim
  int layout;                   // RF_ROPE_HALF or RF_ROPE_INTERLEAVED
};

struct RopeCall {
  const void* x;
  void* out;
  const int32_t* pos;
  int64_t n, x_stride, out_stride;
  int heads, hd, transpose;
};
hipError_t launch_rope(const RopeFreq& f, const RopeCall& c, bool f32, hipStream_t stream);

struct AppendCall {
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* kp;
  uint16_t* vp;
  const int32_t* seq;
  const int32_t* rows;
  const int32_t* pos;
  unsigned* status;
  int64_t n, q_stride, qo_stride, k_stride, v_stride;
  int n_q;
};
hipError_t launch_append(const RopeFreq& f, const Batch& b, const AppendCall& c,
                         hipStream_t stream);

// Queries of a batch, as the attention and the weight accumulation take them.
struct Queries {
  const uint16_t* q;
  const int32_t* start;
  const uint64_t* mask;
  int64_t q_stride, n_q;
  int n_heads, max_q;
  float scale;
};
size_t attend_workspace(const Batch& b, int n_heads, int max_q);
hipError_t launch_attend(const Batch& b, const uint16_t* kp, const uint16_t* vp, const Queries& q,
                         uint16_t* out, int64_t out_stride, float* lse, void* ws,
                         hipStream_t stream);
size_t weight_workspace(const Batch& b, int n_heads, int max_q);
hipError_t launch_weight(const Batch& b, const uint16_t* kp, const Queries& q, const float* lse,
                         float decay, const float* acc, float* acc_out, int64_t acc_stride,
                         void* ws, hipStream_t stream);

constexpr int kEvictPools = 128;   // page pools moved by one launch
struct EvictPools {
  uint16_t* p[kEvictPools];
};
struct EvictCall {
  const float* acc;
  const int32_t* pos;
  float* acc_out;
  int32_t* pos_out;
  int32_t* len_out;
  int64_t stride;
  int n_keep, n_sink, n_recent;
};
size_t evict_workspace(const Batch& b, int n_keep);
hipError_t launch_evict(const Batch& b, const EvictCall& c, uint16_t* const* pools, int n_pools,
                        void* ws, hipStream_t stream);

}  // namespace rf
