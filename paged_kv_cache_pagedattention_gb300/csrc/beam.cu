// Beam selection: the best continuations of every sequence's beams.
//
//   score(w, v) = beam_score[w] + (x[w][v] - m_w) - log sum_u exp(x[w][u] - m_w),   m_w = max_u x[w][u]
//
// (the maximum comes off first: log sum exp itself would be lost in a maximum of 1e30)
// keeps the num_candidates largest of a sequence's num_beams x vocab_size scores.  Within a
// row the order is the logits' own, so the rows are cut into segments; each gives its
// running maximum and sum of the softmax and its best logits, and a second kernel joins the
// segments of a sequence's rows.
#include "pa_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -INFINITY;

// A logit as fp32: NaN counts as -inf, +inf as the type's largest finite value, and -0 as 0.
template <int DT>
__device__ __forceinline__ float clean_logit(typename Elem<DT>::T raw) {
  constexpr float top = DT == PA_F16 ? 65504.f : DT == PA_BF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f;
  const float x = Elem<DT>::load(&raw);
  return x != x ? kNegInf : fminf(x, top) + 0.f;
}

// Keys order logits by value, then by the lower index; 0 is below every key.
__device__ __forceinline__ unsigned long long make_key(float x, unsigned index) {
  const unsigned b = __float_as_uint(x);
  const unsigned ordered = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(ordered) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const unsigned o = static_cast<unsigned>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned key_index(unsigned long long key) {
  return 0xffffffffu - static_cast<unsigned>(key);
}

// m, s <- the softmax state of both: s is sum exp(x - m); (-inf, 0) is empty.
__device__ __forceinline__ void join_state(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  if (top == kNegInf) return;
  s = s * expf(m - top) + s2 * expf(m2 - top);
  m = top;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) beam_segment_kernel(const BeamParams p) {
  using T = typename Elem<DT>::T;
  __shared__ float sm[kThreads / 32], ss[kThreads / 32];
  __shared__ unsigned long long sk[kThreads / 32];
  const int seg = blockIdx.x;
  const long long row = blockIdx.y;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  const int lo = seg * p.segment, hi = min(p.vocab_size, lo + p.segment);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float m = kNegInf, s = 0.f;
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) join_state(m, s, clean_logit<DT>(x[i]), 1.f);
  for (int o = 16; o; o >>= 1) join_state(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
  if (lane == 0) {
    sm[warp] = m;
    ss[warp] = s;
  }
  __syncthreads();
  const long long part = row * p.num_segments + seg;
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) join_state(m, s, sm[w], ss[w]);
    p.state[part] = make_float2(m, s);
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < p.num_candidates; ++k) {
    unsigned long long best = 0;
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
      const float v = clean_logit<DT>(x[i]);
      if (v == kNegInf) continue;
      const unsigned long long key = make_key(v, i);
      if (key < last && key > best) best = key;
    }
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(~0u, best, o));
    if (lane == 0) sk[warp] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < kThreads / 32; ++w) best = max(best, sk[w]);
    __syncthreads();
    if (threadIdx.x == 0) p.keys[part * p.num_candidates + k] = best;
    last = best;  // 0 once the segment is used up: nothing is below it
  }
}

// A candidate of a sequence, and the order of candidates: by score, then the lower beam,
// then the key (larger logit, lower token).  Key 0 is none and comes last.
struct Candidate {
  double score;
  unsigned long long key;
  int beam;
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  if (a.key == 0 || b.key == 0) return a.key != 0;
  if (a.score != b.score) return a.score > b.score;
  if (a.beam != b.beam) return a.beam < b.beam;
  return a.key > b.key;
}

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamParams p) {
  extern __shared__ double2 norm[];  // [num_beams] (maximum, log of the sum against it)
  __shared__ Candidate found[kThreads / 32];
  const long long seq = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int w = threadIdx.x; w < p.num_beams; w += kThreads) {
    const float2* st = p.state + (seq * p.num_beams + w) * p.num_segments;
    float m = kNegInf;
    for (int i = 0; i < p.num_segments; ++i) m = fmaxf(m, st[i].x);
    double sum = 0.0;
    if (m != kNegInf)
      for (int i = 0; i < p.num_segments; ++i) sum += static_cast<double>(st[i].y * expf(st[i].x - m));
    norm[w] = make_double2(m, log(sum));
  }
  __syncthreads();
  const int per_beam = p.num_segments * p.num_candidates, n = p.num_beams * per_beam;
  const unsigned long long* keys = p.keys + seq * n;
  Candidate last = {INFINITY, ~0ull, -1};
  for (int k = 0; k < p.num_candidates; ++k) {
    Candidate best = {0.0, 0, 0};
    for (int c = threadIdx.x; c < n; c += kThreads) {
      Candidate cand = {0.0, keys[c], c / per_beam};
      if (cand.key == 0) continue;
      float cum = p.beam_scores[seq * p.num_beams + cand.beam];
      if (cum != cum || cum == kNegInf) continue;
      cum = fminf(cum, 3.4028234663852886e38f);
      cand.score = cum + ((key_value(cand.key) - norm[cand.beam].x) - norm[cand.beam].y);
      if (before(last, cand) && before(cand, best)) best = cand;
    }
    for (int o = 16; o; o >>= 1) {
      const Candidate other = {__shfl_xor_sync(~0u, best.score, o), __shfl_xor_sync(~0u, best.key, o),
                               __shfl_xor_sync(~0u, best.beam, o)};
      if (before(other, best)) best = other;
    }
    if (lane == 0) found[warp] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w)
      if (before(found[w], best)) best = found[w];
    __syncthreads();
    if (threadIdx.x == 0) {
      const long long at = seq * p.num_candidates + k;
      const bool none = best.key == 0;
      p.out_scores[at] = none ? kNegInf : static_cast<float>(best.score);
      p.out_tokens[at] = none ? -1 : static_cast<int>(key_index(best.key));
      p.out_parents[at] = none ? -1 : static_cast<int>(seq * p.num_beams + best.beam);
    }
    last = best;
  }
}

}  // namespace

// Elements of a row that one block takes: rows are cut until the grid has some four blocks
// an SM, but no finer than 2048 elements.
int beam_segment(long long rows, int vocab_size) {
  const long long want = 152 * 4;
  long long parts = (want + rows - 1) / rows;
  const long long most = (vocab_size + 2047) / 2048;
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  const long long seg = (vocab_size + parts - 1) / parts;
  return static_cast<int>((seg + 7) / 8 * 8);
}

cudaError_t launch_beam_select(const BeamParams& p, int dtype, cudaStream_t stream) {
  const dim3 grid(p.num_segments, p.num_seqs * p.num_beams);
  if (dtype == PA_F32) beam_segment_kernel<PA_F32><<<grid, kThreads, 0, stream>>>(p);
  else if (dtype == PA_F16) beam_segment_kernel<PA_F16><<<grid, kThreads, 0, stream>>>(p);
  else beam_segment_kernel<PA_BF16><<<grid, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  beam_join_kernel<<<p.num_seqs, kThreads, p.num_beams * sizeof(double2), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
