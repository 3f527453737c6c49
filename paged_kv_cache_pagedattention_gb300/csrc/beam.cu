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
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 16;                   // elements of a tile that one thread holds
constexpr int kTile = kThreads * kPerThread;
constexpr int kSpare = 64;                       // kept candidates that do not force a merge
constexpr int kMaxKeep = PA_MAX_BEAM_CANDIDATES;
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kMaxKeep <= 32 && kSpare == 64, "the threshold is one of 32 group maxima");

template <int DT>
constexpr float largest() {
  return DT == PA_F16 ? 65504.f : DT == PA_BF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f;
}

// Keys order logits by value (-0 as 0), then by the lower index; 0 is below every key.
using Key = unsigned long long;
__device__ __forceinline__ Key make_key(float x, unsigned index) {
  const unsigned b = __float_as_uint(x + 0.f);
  const unsigned ordered = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<Key>(ordered) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(Key key) {
  const unsigned o = static_cast<unsigned>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned key_index(Key key) { return 0xffffffffu - static_cast<unsigned>(key); }

// m, s <- the softmax state of both: s is sum exp(x - m); (-inf, 0) is empty.
__device__ __forceinline__ void join_state(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  if (top == kNegInf) return;
  s = s * ex2_approx((m - top) * kLog2e) + s2 * ex2_approx((m2 - top) * kLog2e);
  m = top;
}

// The k-th largest of the block's 32 groups of neighbouring threads, by each group's largest
// v.  The values of k groups are at or above it, so the k largest of all are too.
template <class V>
__device__ __forceinline__ V group_threshold(V v, int k, V* groups, V* result) {
  constexpr int kGroup = kThreads / 32;
#pragma unroll
  for (int o = 1; o < kGroup; o <<= 1) v = max(v, __shfl_xor_sync(~0u, v, o));
  if (threadIdx.x % kGroup == 0) groups[threadIdx.x / kGroup] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    const V mine = groups[threadIdx.x];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const V other = groups[i];
      rank += other > mine || (other == mine && i < static_cast<int>(threadIdx.x));
    }
    if (rank == k - 1) *result = mine;
  }
  __syncthreads();
  return *result;
}

// The same of the block's threads, each a group of its own: a sharper bound for more work.
__device__ __forceinline__ float thread_threshold(float v, int k, float* values, float* result) {
  values[threadIdx.x] = v;
  __syncthreads();
  int rank = 0;
  for (int i = 0; i < kThreads; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(values + i);
    const int behind = static_cast<int>(threadIdx.x) - i;  // of equal values the lower thread's is first
    rank += (w.x > v || (w.x == v && behind > 0)) + (w.y > v || (w.y == v && behind > 1)) +
            (w.z > v || (w.z == v && behind > 2)) + (w.w > v || (w.w == v && behind > 3));
  }
  if (rank == k - 1) *result = v;
  __syncthreads();
  return *result;
}

// The key of a candidate as it is pushed: its value's bits above its index.
__device__ __forceinline__ Key key_of(Key pushed) {
  return make_key(__uint_as_float(static_cast<unsigned>(pushed >> 32)), static_cast<unsigned>(pushed));
}

struct SegmentShared {
  Key buffer[kTile + kSpare];  // candidates: the k best so far as keys, then (value, index) as they come
  unsigned short picked[kTile + kSpare];  // merge: places of the ones above the threshold
  Key groups[32];
  float float_groups[32];
  Key best[kMaxKeep];
  Key threshold;
  float float_threshold;
  float m[kWarps], s[kWarps];
  int count, picked_count;
};

// Reduce the block's candidates to the k best, in order, at the buffer's start and, with 0
// behind them, in `best`; the first `keys` entries are keys already.  Returns the k-th best
// key, or 0 where there are fewer.
__device__ Key merge_candidates(SegmentShared& sh, int k, int keys) {
  const int n = sh.count;
  if (n <= kSpare) {  // the usual case: one warp ranks them, two a lane
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      Key mine[2];
      sh.best[lane] = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = lane + 32 * i;
        mine[i] = at < n ? sh.buffer[at] : 0;
        if (at < n && at >= keys) sh.buffer[at] = mine[i] = key_of(mine[i]);
      }
      __syncwarp();
      int rank[2] = {0, 0};
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const Key other = sh.buffer[j];
        rank[0] += other > mine[0];
        rank[1] += other > mine[1];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < n && rank[i] < k) sh.buffer[rank[i]] = sh.best[rank[i]] = mine[i];
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.count = min(n, k);
    const Key last = sh.best[k - 1];
    __syncthreads();
    return last;
  }
  Key top = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    Key key = sh.buffer[i];
    if (i >= keys) sh.buffer[i] = key = key_of(key);
    top = max(top, key);
  }
  if (threadIdx.x < kMaxKeep) sh.best[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.picked_count = 0;
  const Key threshold = group_threshold(top, k, sh.groups, &sh.threshold);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if (sh.buffer[i] >= threshold) sh.picked[atomicAdd(&sh.picked_count, 1)] = i;
  }
  __syncthreads();
  const int m = sh.picked_count;
  for (int i = threadIdx.x; i < m; i += kThreads) {
    const Key key = sh.buffer[sh.picked[i]];
    int rank = 0;
    for (int j = 0; j < m; ++j) rank += sh.buffer[sh.picked[j]] > key;  // keys are distinct
    if (rank < k) sh.best[rank] = key;
  }
  __syncthreads();
  if (threadIdx.x < k) sh.buffer[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) sh.count = min(n, k);
  const Key last = sh.best[k - 1];
  __syncthreads();
  return last;
}

// The largest of v, and of every four.
__device__ __forceinline__ float maxima(const float (&v)[kPerThread], float (&four)[kPerThread / 4]) {
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < kPerThread / 4; ++i) {
    four[i] = fmaxf(fmaxf(v[4 * i], v[4 * i + 1]), fmaxf(v[4 * i + 2], v[4 * i + 3]));
    top = fmaxf(top, four[i]);
  }
  return top;
}

// Sum of exp(v - m), two elements an instruction but for the exponential.
__device__ __forceinline__ float exp_sum(const float (&v)[kPerThread], float m) {
  float even = 0.f, odd = 0.f;
#pragma unroll
  for (int i = 0; i < kPerThread; i += 2) {
    float a, b;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 y, {%5, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(a), "=f"(b)
        : "f"(v[i]), "f"(v[i + 1]), "f"(-m), "f"(kLog2e));
    a = ex2_approx(a);
    b = ex2_approx(b);
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(even), "+f"(odd)
        : "f"(a), "f"(b));
  }
  return even + odd;
}

// 16 bytes from byte `shift` (0 .. 15) of the 32 in lo and hi.
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, unsigned shift) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const unsigned bits = 8 * (shift & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// One block a segment of a row, in one pass: tiles of kTile elements in registers, the next
// tile's loads in flight.  Per thread a running maximum and the sum of exp against it,
// rescaled once a tile; a tile's elements are looked at one by one only in threads whose
// maximum reaches the block's threshold.  The first threshold comes from the tile's group
// maxima, later ones from the merges.
//
// A thread's elements are given by their index in the row alone, so equal rows have equal
// sums wherever they lie in memory.  Rows off the 16-byte grid (an odd vocabulary, kShifted)
// are read as the two pieces that cover 16 bytes; pieces that reach over the row's ends are
// read element by element.
template <int DT, bool kShifted>
__global__ void __launch_bounds__(kThreads) beam_segment_kernel(const BeamParams p) {
  using T = typename Elem<DT>::T;
  constexpr int kVec = 16 / Elem<DT>::bytes;      // elements of a 16-byte piece
  constexpr int kLoads = kPerThread / kVec;
  extern __shared__ __align__(16) unsigned char raw[];
  SegmentShared& sh = *reinterpret_cast<SegmentShared*>(raw);
  const int seg = blockIdx.x, k = p.num_candidates;
  const long long row = blockIdx.y;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  // the row's whole pieces, cut evenly; the elements behind the last go to the last segment
  const int pieces = p.vocab_size / kVec;
  const int first = static_cast<int>((long long)pieces * seg / p.num_segments);
  const int end = static_cast<int>((long long)pieces * (seg + 1) / p.num_segments);
  const unsigned shift = kShifted ? reinterpret_cast<uintptr_t>(x) % 16 : 0;
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x) - shift);
  // pieces [inner, inner_end) lie in the row with the 32 bytes that are read for them
  const int inner = shift ? 1 : 0;
  const int inner_end = (p.vocab_size - kVec + static_cast<int>(shift / sizeof(T))) / kVec;
  if (threadIdx.x == 0) sh.count = 0;

  float m = kNegInf, s = 0.f;
  Key threshold = 0;      // candidates below it are not among the segment's k best
  float least = kNegInf;  // its value
  int keys = 0;           // candidates at the buffer's start that are keys
  bool fresh = true;      // no threshold yet
  // index_of(i): the row's element that v[i] is
  auto take = [&](float (&v)[kPerThread], auto index_of) {
    float four[kPerThread / 4];  // maxima of four elements each; NaN is passed over
    float top = maxima(v, four);
    float m2 = fmaxf(m, top);
    float sum = m2 != kNegInf ? exp_sum(v, m2) : 0.f;
    if (top == INFINITY || sum != sum) {  // NaN and +inf: once more, as -inf and the largest finite value
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) v[i] = fminf(fmaxf(v[i], kNegInf), largest<DT>());
      top = maxima(v, four);
      m2 = fmaxf(m, top);
      sum = m2 != kNegInf ? exp_sum(v, m2) : 0.f;
    }
    if (m2 != kNegInf) {
      s = s * ex2_approx((m - m2) * kLog2e) + sum;
      m = m2;
    }
    if (fresh) {
      least = group_threshold(top, k, sh.float_groups, &sh.float_threshold);
      if (least != kNegInf) threshold = make_key(least, 0xffffffffu);
    }
    bool full = fresh;  // the first tile's candidates give a sharper threshold at once
    fresh = false;
    if (top >= least) {
#pragma unroll
      for (int q = 0; q < kPerThread / 4; ++q) {
        if (!(four[q] >= least)) continue;
#pragma unroll
        for (int i = 4 * q; i < 4 * q + 4; ++i) {
          if (!(v[i] >= least) || v[i] == kNegInf) continue;
          const unsigned index = index_of(i);
          if (v[i] == least && index > key_index(threshold)) continue;
          const int at = atomicAdd(&sh.count, 1);
          sh.buffer[at] = static_cast<Key>(__float_as_uint(v[i])) << 32 | index;
          full |= at >= kSpare;
        }
      }
    }
    if (__syncthreads_or(full)) {
      const int kept = sh.count;
      threshold = max(threshold, merge_candidates(sh, k, keys));
      if (threshold != 0) least = key_value(threshold);
      keys = min(k, kept);
    }
  };

  uint4 next[kLoads], over[kShifted ? kLoads : 1];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = base + i * kThreads + threadIdx.x;
      if (at >= end) continue;
      if (!kShifted || (at >= inner && at < inner_end)) {
        next[i] = src[at];
        if constexpr (kShifted) over[i] = src[at + 1];
      } else {
        T each[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) each[j] = x[(long long)at * kVec + j];
        memcpy(&next[i], each, 16);
      }
    }
  };
  load(first);
  for (int base = first; base < end; base += kLoads * kThreads) {
    const bool whole = base + kLoads * kThreads <= end;
    float v[kPerThread];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = base + i * kThreads + threadIdx.x;
      uint4 piece = next[i];
      if constexpr (kShifted) piece = shifted(piece, over[i], at >= inner && at < inner_end ? shift : 0);
      const uint32_t w[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == PA_F32) {
          v[i * kVec + j] = __uint_as_float(w[j]);
        } else {
          const float2 f = unpack2<DT>(w[j]);
          v[i * kVec + 2 * j] = f.x;
          v[i * kVec + 2 * j + 1] = f.y;
        }
      }
      if (!whole && at >= end) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i * kVec + j] = kNegInf;
      }
    }
    load(base + kLoads * kThreads);
    take(v, [&](int i) { return (base + i / kVec * kThreads + threadIdx.x) * kVec + i % kVec; });
  }
  const int tail = pieces * kVec;
  if (seg == p.num_segments - 1 && tail < p.vocab_size) {
    float v[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) v[j] = kNegInf;
    if (static_cast<int>(threadIdx.x) < p.vocab_size - tail) v[0] = Elem<DT>::load(x + tail + threadIdx.x);
    take(v, [&](int) { return tail + threadIdx.x; });
  }

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int o = 16; o; o >>= 1) join_state(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
  if (lane == 0) {
    sh.m[warp] = m;
    sh.s[warp] = s;
  }
  __syncthreads();
  if (fresh || sh.count > keys) merge_candidates(sh, k, keys);  // else `best` is up to date
  const long long part = row * p.num_segments + seg;
  if (warp == 0) {
    m = lane < kWarps ? sh.m[lane] : kNegInf;
    s = lane < kWarps ? sh.s[lane] : 0.f;
    for (int o = kWarps / 2; o; o >>= 1) join_state(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
    if (lane == 0) p.state[part] = make_float2(m, s);
  }
  if (threadIdx.x < k) p.keys[part * k + threadIdx.x] = sh.best[threadIdx.x];
}

// log of a sum of 1 or more, to 2^-25 or so: its power of two in fp64 and log1p of the rest
// (within -0.3 .. 0.42) in fp32.  fp64's own log took half of the join's time: the SM has two
// fp64 lanes.
__device__ __forceinline__ double log_of(double sum) {
  const long long bits = __double_as_longlong(sum);
  int power = static_cast<int>(bits >> 52) - 1023;
  long long rest = bits & 0xfffffffffffffll;  // the mantissa less one, times 2^52
  float f = static_cast<float>(rest) * 0x1p-52f;
  if (f > 0.41421356f) {
    ++power;
    f = static_cast<float>(rest - (1ll << 52)) * 0x1p-53f;
  }
  return power * 0.69314718055994530942 + static_cast<double>(log1pf(f));
}

// A beam of a sequence: its score, its row's maximum and the log of the sum against it.
struct Beam {
  double log_sum;
  float score, m;
};

// The fp64 score of a candidate, as an integer of the same order.
__device__ __forceinline__ long long score_of(const Beam& b, Key key) {
  const long long bits =
      __double_as_longlong(b.score + ((key_value(key) - static_cast<double>(b.m)) - b.log_sum));
  return bits ^ ((bits >> 63) & 0x7fffffffffffffffll);
}

// Candidates in order: by score, then the lower beam, then the key (larger logit, lower
// token).  Key 0 is none and comes last.
struct Candidate {
  long long score;
  Key key;
  int beam;
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  if (a.key == 0 || b.key == 0) return a.key != 0;
  if (a.score != b.score) return a.score > b.score;
  if (a.beam != b.beam) return a.beam < b.beam;
  return a.key > b.key;
}

__device__ __forceinline__ void write_out(const BeamParams& p, long long seq, int k, const Candidate& c) {
  const long long at = seq * p.num_candidates + k;
  const bool none = c.key == 0;
  const double score = __longlong_as_double(c.score ^ ((c.score >> 63) & 0x7fffffffffffffffll));
  p.out_scores[at] = none ? kNegInf : static_cast<float>(score);
  p.out_tokens[at] = none ? -1 : static_cast<int>(key_index(c.key));
  p.out_parents[at] = none ? -1 : static_cast<int>(seq * p.num_beams + c.beam);
}

constexpr int kJoin = 1024;  // candidates that are ranked at once
constexpr int kHeld = 4;     // keys a thread loads ahead

// One block a sequence: the rows' states are joined, then the segments' candidates.  Most
// fall to a threshold on their fp32 scores, held with the scores' error bounds so that
// none of the best can be lost; the rest are ranked by their fp64 scores.
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamParams p) {
  extern __shared__ Beam beams[];  // [num_beams]
  __shared__ long long scores[kJoin];
  __shared__ Key kept[kJoin];
  __shared__ int owner[kJoin];
  __shared__ __align__(16) float tops[kThreads];
  __shared__ float bound;
  __shared__ Candidate found[kThreads / 32];
  __shared__ int count;
  const long long seq = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per_beam = p.num_segments * p.num_candidates, n = p.num_beams * per_beam;
  const Key* keys = p.keys + seq * n;
  Key held[kHeld];  // on their way while the states are joined
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = threadIdx.x + i * kThreads;
    held[i] = c < n ? keys[c] : 0;
  }
  if (threadIdx.x == 0) count = 0;
  for (int w = warp; w < p.num_beams; w += kThreads / 32) {
    const float2* st = p.state + (seq * p.num_beams + w) * p.num_segments;
    const float cum = p.beam_scores[seq * p.num_beams + w];
    float m = kNegInf;
    for (int i = lane; i < p.num_segments; i += 32) m = fmaxf(m, st[i].x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    double sum = 0.0;
    if (m != kNegInf)
      for (int i = lane; i < p.num_segments; i += 32) sum += static_cast<double>(st[i].y * expf(st[i].x - m));
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) beams[w] = {log_of(sum), m == kNegInf ? kNegInf : fminf(fmaxf(cum, kNegInf), largest<PA_F32>()), m};
  }
  __syncthreads();
  // f(candidate's beam, its key) for this thread's candidates
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (held[i] != 0) f((threadIdx.x + i * kThreads) / per_beam, held[i]);
    for (int c = threadIdx.x + kHeld * kThreads; c < n; c += kThreads) {
      const Key key = keys[c];
      if (key != 0) f(c / per_beam, key);
    }
  };
  // fp32: each of the three terms and sums is rounded once, so a score is off by less than
  // 2^-22 of the terms' magnitudes
  auto score32 = [&](const Beam& b, Key key, float& error) {
    const float rel = key_value(key) - b.m, log_sum = static_cast<float>(b.log_sum);
    error = 0x1p-21f * (fabsf(b.score) + fabsf(rel) + fabsf(log_sum));
    return b.score + (rel - log_sum);
  };
  float top = kNegInf;
  each([&](int w, Key key) {
    const Beam b = beams[w];
    if (b.score == kNegInf) return;
    float error;
    const float score = score32(b, key, error);
    top = fmaxf(top, score - error);
  });
  const float threshold = thread_threshold(top, p.num_candidates, tops, &bound);
  each([&](int w, Key key) {
    const Beam b = beams[w];
    if (b.score == kNegInf) return;
    float error;
    const float score = score32(b, key, error);
    if (score + error < threshold) return;
    const int at = atomicAdd(&count, 1);
    if (at >= kJoin) return;
    scores[at] = score_of(b, key);
    kept[at] = key;
    owner[at] = w;
  });
  __syncthreads();
  const int m = count;
  if (m <= kJoin) {
    for (int i = warp; i < m; i += kThreads / 32) {
      const Candidate mine = {scores[i], kept[i], owner[i]};
      int rank = 0;
      for (int j = lane; j < m; j += 32) {
        const long long other = scores[j];
        if (other >= mine.score) rank += other > mine.score || before({other, kept[j], owner[j]}, mine);
      }
      rank = __reduce_add_sync(~0u, rank);
      if (lane == 0 && rank < p.num_candidates) write_out(p, seq, rank, mine);
    }
    for (int i = m + threadIdx.x; i < p.num_candidates; i += kThreads) write_out(p, seq, i, {0, 0, 0});
    return;
  }
  // more near-equal candidates than fit: one after the other
  Candidate last = {0x7fffffffffffffffll, ~0ull, -1};
  for (int k = 0; k < p.num_candidates; ++k) {
    Candidate best = {0, 0, 0};
    each([&](int w, Key key) {
      const Beam b = beams[w];
      if (b.score == kNegInf) return;
      const Candidate cand = {score_of(b, key), key, w};
      if (before(last, cand) && before(cand, best)) best = cand;
    });
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
    if (threadIdx.x == 0) write_out(p, seq, k, best);
    last = best;
  }
}

}  // namespace

// Segments of a row: rows are cut as long as the grid fits at once (four blocks an SM), but
// no finer than half a tile.
int beam_segments(long long rows, int vocab_size) {
  const long long fit = 152 * 4 / rows, most = (vocab_size + kTile / 2 - 1) / (kTile / 2);
  return static_cast<int>(fit < 1 ? 1 : fit < most ? fit : most);
}

template <int DT, bool kShifted>
static cudaError_t launch_segments(const BeamParams& p, cudaStream_t stream) {
  const int smem = sizeof(SegmentShared);
  const cudaError_t e = set_smem<beam_segment_kernel<DT, kShifted>>(smem);
  if (e != cudaSuccess) return e;
  beam_segment_kernel<DT, kShifted><<<dim3(p.num_segments, p.num_seqs * p.num_beams), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int DT>
static cudaError_t launch_type(const BeamParams& p, cudaStream_t stream) {
  const bool one = p.num_seqs * p.num_beams == 1;
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                       (one || p.row_stride * Elem<DT>::bytes % 16 == 0);
  return aligned ? launch_segments<DT, false>(p, stream) : launch_segments<DT, true>(p, stream);
}

cudaError_t launch_beam_select(const BeamParams& p, int dtype, cudaStream_t stream) {
  const cudaError_t e = dtype == PA_F32   ? launch_type<PA_F32>(p, stream)
                        : dtype == PA_F16 ? launch_type<PA_F16>(p, stream)
                                          : launch_type<PA_BF16>(p, stream);
  if (e != cudaSuccess) return e;
  beam_join_kernel<<<p.num_seqs, kThreads, p.num_beams * sizeof(Beam), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
