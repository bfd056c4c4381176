// The attention weight that the rows of the paged cache receive, on gfx950 (section "Which
// rows to compute exactly" of the English RidgeFill review).
//
// The plain kernel: one wave per row adds up the weights of all queries and heads.
#include "rf_cache.h"
#include "rf_common.h"

namespace rf {

namespace {

__device__ __forceinline__ int pool_slot(const Batch& b, int seq, int row) {
  const int page = b.tables[(int64_t)seq * b.table_stride + row / b.page_size];
  if (page < 0 || page >= b.num_pages) return -1;
  return page * b.page_size + row % b.page_size;
}

// Sequence `seq`: its length, its queries; false if it is to be skipped (with *bad set where
// that is an error).
__device__ __forceinline__ bool sequence_of(const Batch& b, const Queries& q, int seq, int* len,
                                            int* first, int* n, bool* bad) {
  *len = b.lengths[seq];
  *first = q.start[seq];
  *n = q.start[seq + 1] - *first;
  *bad = *len < 0 || *len > b.max_len || *first < 0 || *n < 0 || *n > q.max_q || *n > *len ||
         (int64_t)*first + *n > q.n_q;
  return !*bad && *n > 0;
}

__device__ __forceinline__ bool sees(const Queries& q, int query, int i, int draft) {
  if (draft < 0) return true;
  return q.mask ? (q.mask[query] >> draft) & 1 : draft <= i;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__global__ void weight_plain_kernel(Batch b, const uint16_t* kp, Queries q, const float* lse,
                                    float decay, const float* acc, float* acc_out,
                                    int64_t acc_stride, unsigned* status) {
  const int seq = blockIdx.y, t = blockIdx.x, lane = threadIdx.x;
  int len, first, n;
  bool bad;
  const bool go = sequence_of(b, q, seq, &len, &first, &n, &bad);
  if (bad) atomicOr(status, kStatusRowsBit);
  if (!go || t >= len) return;
  const int per = b.hd / 64, group = q.n_heads / b.n_kv, ctx = len - n;
  const int slot = pool_slot(b, seq, t);
  float w = 0.f;
  if (slot < 0) {
    atomicOr(status, kStatusRowsBit);
  } else {
    for (int kh = 0; kh < b.n_kv; ++kh) {
      const int64_t at = ((int64_t)slot * b.n_kv + kh) * b.hd + lane * per;
      for (int i = 0; i < n; ++i) {
        if (!sees(q, first + i, i, t - ctx)) continue;
        for (int h = kh * group; h < (kh + 1) * group; ++h) {
          const uint16_t* qp = q.q + (first + i) * q.q_stride + h * b.hd + lane * per;
          const float l = lse[(int64_t)(first + i) * q.n_heads + h];
          float s = 0.f;
          for (int e = 0; e < per; ++e) s += bf16_to_f32(qp[e]) * bf16_to_f32(kp[at + e]);
          s = wave_sum(s) * q.scale;
          if (l != -INFINITY) w += expf(s - l);
        }
      }
    }
  }
  if (lane == 0) {
    const int64_t a = seq * acc_stride + t;
    acc_out[a] = acc ? decay * acc[a] + w : w;
  }
}

}  // namespace

size_t weight_workspace(const Batch&, int, int) { return kStatusBytes; }

hipError_t launch_weight(const Batch& b, const uint16_t* kp, const Queries& q, const float* lse,
                         float decay, const float* acc, float* acc_out, int64_t acc_stride,
                         void* ws, hipStream_t stream) {
  unsigned* status = static_cast<unsigned*>(ws);
  const hipError_t e = launch_clear_status(status, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(weight_plain_kernel, dim3(b.max_len, b.batch), dim3(64), 0, stream, b, kp, q,
                     lse, decay, acc, acc_out, acc_stride, status);
  return hipGetLastError();
}

}  // namespace rf
