// Differential attention: what its kernels share.
//
//   O_h = (softmax(s q1 K1^T) - lambda softmax(s q2 K2^T)) V,  q1, q2 the head's two query rows,
//   K1, K2 its KV group's two key rows, V the group's value row of 2 d elements (halves V1, V2)
//   out_h = O_h, or O_h / sqrt(mean(O_h^2) + eps) * w
//
// Each map is an online softmax of its own (maximum m in log2 units, sum l, weighted sum a of V);
// with a1, l1 and a2, l2 joined over a row's partitions, O = a1 / l1 - lambda a2 / l2.  All of it
// is fp32; the result is rounded once, behind the norm.
#pragma once

#include "pa_common.cuh"

namespace pa {

__device__ __forceinline__ float diff_lambda(const DiffParams& p, long long row, int head) {
  return p.lambda[row * p.lambda_row_stride + head * p.lambda_head_stride];
}

// A row whose keys and partial states have their places: row_info's checks, and no more tokens in its
// request than the call was told of (the plan has flagged such a request and keeps no room for it).
__device__ __forceinline__ bool diff_row_ok(const AttnParams& a, const RowInfo& ri) {
  return ri.ok && ri.q_len <= a.max_query_len;
}

// A map's weight in the difference, with its sum divided out; 0 where the map attends nothing.
__device__ __forceinline__ float diff_weight(float l) { return l > 0.f ? 1.f / l : 0.f; }

// A warp's head: lane i holds elements 64 k + 2 i, 64 k + 2 i + 1 of the difference's `width` in
// o[k].  Norm, rounding and store.
template <int QDT, int N>
__device__ __forceinline__ void diff_finish(const DiffParams& p, long long row, int head, int width, float2 (&o)[N]) {
  using QE = Elem<QDT>;
  const int lane = threadIdx.x & 31;
  if (p.norm_weight) {
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (64 * k + 2 * lane < width) sq += o[k].x * o[k].x + o[k].y * o[k].y;
    sq = warp_sum_xor(sq, 1, 16);
    const float r = rsqrtf(sq / width + p.norm_eps);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = 64 * k + 2 * lane;
      if (c < width) {
        o[k].x *= r * p.norm_weight[c];
        o[k].y *= r * p.norm_weight[c + 1];
      }
    }
  }
  typename QE::T* out = static_cast<typename QE::T*>(p.a.out) + (row * (p.a.num_q_heads / 2) + head) * width;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = 64 * k + 2 * lane;
    if (c < width) {
      out[c] = QE::from_float(o[k].x);
      out[c + 1] = QE::from_float(o[k].y);
    }
  }
}

}  // namespace pa
