// Beam selection: the best continuations of every sequence's beams.
//
//   score(w, v) = beam_score[w] + (x[w][v] - m_w) - log sum_u exp(x[w][u] - m_w),   m_w = max_u x[w][u]
//
// (the maximum comes off first: log sum exp itself would be lost in a maximum of 1e30)
// keeps the num_candidates largest of a sequence's num_beams x vocab_size scores.  Within a
// row the order is the logits' own, so the rows are cut into segments; each gives its
// maximum and sum of the softmax and its best logits, and a second kernel joins the
// segments of a sequence's rows.
#include <type_traits>

#include "launch.cuh"
#include "pa_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 4;       // 16-byte pieces of a tile that one thread takes
constexpr int kTileBytes = kThreads * kLoads * 16;
constexpr int kWindow = 8;      // tiles between the block's barriers
constexpr int kRoom = 1024;     // candidates a block can hold
constexpr int kRescan = 2048;   // elements that are looked at again at a time
constexpr int kGroups = 64;     // of threads, for bounds
constexpr int kFew = 96;        // candidates that are ranked without a bound first
constexpr int kMaxKeep = PA_MAX_BEAM_CANDIDATES;
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kMaxKeep <= kGroups, "");

template <int DT>
constexpr float largest() {
  return DT == PA_F16 ? 65504.f : DT == PA_BF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f;
}

// A logit as fp32: NaN counts as -inf, +inf as the type's largest finite value.
template <int DT>
__device__ __forceinline__ float clean_logit(typename Elem<DT>::T raw) {
  return fminf(fmaxf(Elem<DT>::load(&raw), kNegInf), largest<DT>());
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
// The key of a candidate as it is pushed: its value's bits above its index.
__device__ __forceinline__ Key key_of(Key pushed) {
  return make_key(__uint_as_float(static_cast<unsigned>(pushed >> 32)), static_cast<unsigned>(pushed));
}

// The joined softmax state of a warp's lanes: s is sum exp(x - m), (-inf, 0) is empty.
__device__ __forceinline__ void warp_state(float& m, float& s) {
  float top = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (top != kNegInf) s *= ex2_approx((m - top) * kLog2e);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  m = top;
}

// A lower bound of the k-th largest of the block's values: the k-th largest of 64 groups of
// neighbouring threads, by each group's largest.  The values of k groups are at or above it,
// so the k largest of all are too.  Groups are ranked as whole numbers whose last six bits
// are the group's place, so that no two are equal; the bound has those bits off (2^-18 of
// the value lower at most).  `largest` gets a value at or above all but 2^-18 of the largest.
struct __align__(16) GroupShared {
  int order[kGroups];
  float values[kGroups], bound, largest;
};
__device__ __forceinline__ int float_order(float x) {  // whole numbers in the order of floats
  const int b = __float_as_int(x + 0.f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float group_bound(float v, int k, GroupShared& sh) {
  constexpr int kGroup = kThreads / kGroups;
#pragma unroll
  for (int o = 1; o < kGroup; o <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  if (threadIdx.x % kGroup == 0) {
    const int g = threadIdx.x / kGroup;
    sh.order[g] = (float_order(v) & ~63) | g;
    sh.values[g] = v;
  }
  __syncthreads();
  if (threadIdx.x < kGroups) {
    const int mine = sh.order[threadIdx.x];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kGroups; i += 4) {
      const int4 o = *reinterpret_cast<const int4*>(sh.order + i);
      rank += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    }
    if (rank == k - 1) {
      const int b = mine & ~63;
      sh.bound = sh.values[threadIdx.x] == kNegInf ? kNegInf : __int_as_float(b ^ ((b >> 31) & 0x7fffffff));
    }
    if (rank == 0) sh.largest = sh.values[threadIdx.x];
  }
  __syncthreads();
  return sh.bound;
}

struct __align__(16) SegmentShared {
  Key buffer[kRoom];  // candidates: the k best so far as keys, then (value, index) as they come
  Key pick[kRoom];    // merge: the keys that reach its bound
  Key best[kMaxKeep];
  GroupShared groups;
  float m[kWarps], s[kWarps];
  int count, picked;
};

// Reduce the block's candidates to the k best, in order, at the buffer's start and, with 0
// behind them, in `best`; the first `keys` entries are keys already.  Returns the k-th best
// key, or 0 where there are fewer.
__device__ Key merge_candidates(SegmentShared& sh, int k, int keys) {
  const int n = min(sh.count, kRoom);
  float bound = kNegInf;
  if (n > kFew) {  // only what reaches a bound is ranked
    float top = kNegInf;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const Key c = sh.buffer[i];
      top = fmaxf(top, i < keys ? key_value(c) : __uint_as_float(static_cast<unsigned>(c >> 32)));
    }
    bound = group_bound(top, k, sh.groups);
  }
  if (threadIdx.x < kMaxKeep) sh.best[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.picked = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    Key key = sh.buffer[i];
    if (i >= keys) key = key_of(key);
    if (key_value(key) >= bound) sh.pick[atomicAdd(&sh.picked, 1)] = key;
  }
  __syncthreads();
  const int m = sh.picked;
  for (int i = threadIdx.x; i < m; i += kThreads) {
    const Key key = sh.pick[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < m; ++j) rank += sh.pick[j] > key;  // keys are distinct
    if (rank < k) sh.buffer[rank] = sh.best[rank] = key;
  }
  if (threadIdx.x == 0) sh.count = min(n, k);
  __syncthreads();
  return sh.best[k - 1];
}

// Drop the candidates from element `start` on from the merged ones; returns how many stay.
__device__ int drop_candidates(SegmentShared& sh, int k, unsigned start) {
  if (threadIdx.x == 0) {
    int kept = 0;
    for (int i = 0; i < k; ++i) {
      const Key key = sh.best[i];
      if (key != 0 && key_index(key) < start) sh.buffer[kept++] = key;
    }
    sh.count = kept;
  }
  __syncthreads();
  const int kept = sh.count;
  __syncthreads();
  return kept;
}

// Push a candidate; returns whether they are to be merged.  One equal to the threshold's
// value counts up to the threshold's place.
__device__ __forceinline__ bool push_candidate(SegmentShared& sh, float value, unsigned index, float least,
                                               Key threshold, int spare) {
  if (value == kNegInf || (value == least && index > key_index(threshold))) return false;
  const int at = atomicAdd(&sh.count, 1);
  if (at < kRoom) sh.buffer[at] = static_cast<Key>(__float_as_uint(value)) << 32 | index;
  return at >= spare;
}

// 16 bytes from byte 4 kWord + bits / 8 of the 32 in lo and hi; kHalves: bits may be 16.
template <int kWord, bool kHalves>
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, unsigned bits) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if constexpr (kHalves)
    return make_uint4(__funnelshift_r(w[kWord], w[kWord + 1], bits), __funnelshift_r(w[kWord + 1], w[kWord + 2], bits),
                      __funnelshift_r(w[kWord + 2], w[kWord + 3], bits),
                      __funnelshift_r(w[kWord + 3], w[kWord + 4], bits));
  else return make_uint4(w[kWord], w[kWord + 1], w[kWord + 2], w[kWord + 3]);
}

// A thread's part of a tile: kLoads pieces as they lie in memory.
template <int DT>
struct Part {
  static constexpr int kWords = 4 * kLoads, n = 4 * kWords / Elem<DT>::bytes;
  uint32_t w[kWords];

  __device__ __forceinline__ float at(int i) const {
    if constexpr (DT == PA_F32) return __uint_as_float(w[i]);
    else if constexpr (DT == PA_BF16) return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(i % 2 ? w[i / 2] >> 16 : w[i / 2])));
  }
  __device__ __forceinline__ void put(int i, uint4 piece) {  // the i-th 16 bytes
    w[4 * i] = piece.x;
    w[4 * i + 1] = piece.y;
    w[4 * i + 2] = piece.z;
    w[4 * i + 3] = piece.w;
  }
  static __device__ __forceinline__ uint32_t empty() {  // a word of -inf
    return DT == PA_F32 ? 0xff800000u : DT == PA_F16 ? 0xfc00fc00u : 0xff80ff80u;
  }
  // The larger of two words, element by element; NaN is passed over.
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (DT == PA_F32) {
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (DT == PA_F16) {
      const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  __device__ __forceinline__ float maximum() const {  // +inf as the largest finite value
    uint32_t top = w[0];
#pragma unroll
    for (int i = 1; i < kWords; ++i) top = larger(top, w[i]);
    float2 f = make_float2(__uint_as_float(top), kNegInf);
    if constexpr (DT != PA_F32) f = unpack2<DT>(top);
    return fminf(fmaxf(fmaxf(f.x, f.y), kNegInf), largest<DT>());
  }
  // Bits of the elements that are at or above `least` and not -inf, of the fourths whose sum
  // is not below `bound`.
  __device__ __forceinline__ unsigned reach(float least, float4 sums, float bound) const {
    const float lowest = fmaxf(least, -largest<PA_F32>());
    const float sum[4] = {sums.x, sums.y, sums.z, sums.w};
    unsigned bits = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (sum[c] < bound) continue;
#pragma unroll
      for (int i = c; i < n; i += 4) bits |= (at(i) >= lowest ? 1u : 0u) << i;
    }
    return bits;
  }
  // Sums of exp(x - m), of every fourth element each.  m comes off before the product with
  // log2 e, so that an element that is m gives exactly 1 and a likely token's score loses
  // nothing.
  __device__ __forceinline__ float4 exp_sums(float m) const {
    const float2 off = make_float2(-m, -m), scale = make_float2(kLog2e, kLog2e);
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int i = 0; i < n; i += 4) {
      const float2 d = __fmul2_rn(__fadd2_rn(make_float2(at(i), at(i + 1)), off), scale);
      const float2 e = __fmul2_rn(__fadd2_rn(make_float2(at(i + 2), at(i + 3)), off), scale);
      a = __fadd2_rn(a, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
      b = __fadd2_rn(b, make_float2(ex2_approx(e.x), ex2_approx(e.y)));
    }
    return make_float4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void clean() {  // NaN to -inf, +inf to the largest finite value
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (DT == PA_F32) {
        w[i] = __float_as_uint(fminf(fmaxf(__uint_as_float(w[i]), kNegInf), largest<DT>()));
      } else {
        const float2 f = unpack2<DT>(w[i]);
        w[i] = pack2<DT>(fminf(fmaxf(f.x, kNegInf), largest<DT>()), fminf(fmaxf(f.y, kNegInf), largest<DT>()));
      }
    }
  }
};

__device__ __forceinline__ void async_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Tiles on their way, and the pieces of one that a warp fetches (with a shift also those
// behind its runs of 32).
constexpr int kStages = 2;
template <bool kShifted>
constexpr int ring_slots() { return kLoads * (kShifted ? 33 : 32); }

// One block a segment of a row, in one pass: tiles of kTileBytes, the next one on its
// way to shared memory while one is in registers.  Per thread the sum of exp against a
// reference m: the first tile's maximum, later the thread's own where it is larger, so that
// m of the largest element's thread is that element.  Where the sums of a part's
// exponentials stay below the threshold's, no element can have reached it; only else is the
// part's maximum taken and its elements looked at one by one and pushed to the block's
// candidates.  The first tile's group maxima give the first threshold, merges give sharper
// ones.  The warps run freely for a window of tiles before they meet to merge (a barrier a
// tile cost a third of the time).
//
// A thread's elements are given by their index in the row alone, so equal rows have equal
// sums wherever they lie in memory.  In rows off the 16-byte grid (an odd vocabulary,
// kShifted) 16 bytes of elements are put together from the two aligned pieces they lie in.
//
// Bound by memory with fp32 logits (256 rows of 262,144: 48 us with the join, 5.6 TB/s), by
// the issue of instructions with 16-bit ones (600 rows of 131,072 bf16: 36 us, 4.3 TB/s; four
// pieces a thread and tile for every type, as what a tile costs besides its elements is half of
// it: two pieces, 4,096 elements a tile, took 39 us), and by the way of the first tile and the
// merges in short segments (128 rows of 131,072 bf16, four segments each: 20 us with the
// join).
template <int DT, bool kShifted>
__global__ void __launch_bounds__(kThreads, 4) beam_segment_kernel(const BeamParams p) {
  using T = typename Elem<DT>::T;
  constexpr int kVec = 16 / Elem<DT>::bytes;  // elements of a 16-byte piece
  constexpr int kStep = kLoads * kThreads;    // pieces of a tile
  constexpr int kSlots = ring_slots<kShifted>();
  previous_done();
  next_may_start();  // the join's blocks come up while the last segments run
  extern __shared__ __align__(16) unsigned char raw[];
  SegmentShared& sh = *reinterpret_cast<SegmentShared*>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int seg = blockIdx.x, k = p.num_candidates;
  const int spare = 2 * k;  // candidates that do not force a merge
  const long long row = blockIdx.y;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  // the row's whole pieces, cut evenly; the elements behind the last go to the last segment
  const int pieces = p.vocab_size / kVec;
  const int first = static_cast<int>((long long)pieces * seg / p.num_segments);
  const int end = static_cast<int>((long long)pieces * (seg + 1) / p.num_segments);
  const unsigned shift = kShifted ? reinterpret_cast<uintptr_t>(x) % 16 : 0;
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x) - shift);

  // a thread's pieces of a tile lie kThreads apart, and a warp alone reads what it fetches
  constexpr int kRun = kSlots / kLoads;  // slots of 32 neighbouring pieces
  const int own = threadIdx.x;
  uint4* ring = reinterpret_cast<uint4*>(raw + sizeof(SegmentShared)) + warp * kSlots + lane;
  auto fetch = [&](uint4* dst, int at) {
    if constexpr (kShifted) {  // a piece that reaches over the row's ends: its elements alone
      const long long start = (long long)at * kVec - static_cast<int>(shift / sizeof(T));
      if (start < 0 || start + kVec > p.vocab_size) {
        T* out = reinterpret_cast<T*>(dst);
        for (int j = 0; j < kVec; ++j)
          if (start + j >= 0 && start + j < p.vocab_size) out[j] = x[start + j];
        return;
      }
    }
    async_copy16(dst, src + at);
  };
  auto load = [&](int base, int stage) {
    uint4* slot = ring + stage * (kSlots * kWarps);
    const int at = base + own, stop = end + (kShifted ? 1 : 0);
    // a whole tile inside the row: no piece is asked for its place (without a shift this gained nothing)
    if (kShifted && base > 0 && base + kStep < pieces && base + kStep <= end) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) async_copy16(slot + i * kRun, src + at + i * kThreads);
      if (lane < kLoads) async_copy16(slot - lane + lane * kRun + 32, src + (at - lane + lane * kThreads + 32));
      async_commit();
      return;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (at + i * kThreads < stop) fetch(slot + i * kRun, at + i * kThreads);
    if constexpr (kShifted) {  // the pieces behind the runs: lane i fetches run i's
      const int behind = at - lane + lane * kThreads + 32;
      if (lane < kLoads && behind < stop) fetch(slot - lane + lane * kRun + 32, behind);
    }
    async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) load(first + i * kStep, i);
  if (threadIdx.x == 0) sh.count = 0;

  float m = kNegInf, s = 0.f;
  Key threshold = 0;      // candidates below it are not among the segment's k best
  float least = kNegInf;  // its value
  float bound = 0.f;      // four sums of a part's exponentials below this: no element at the threshold
  int keys = 0;           // candidates at the buffer's start that are keys
  bool merged = false;
  auto set_bound = [&]() {
    bound = least != kNegInf && m != kNegInf ? fminf(ex2_approx((least - m) * kLog2e) * (1.f - 0x1p-10f), 0x1p64f) : 0.f;
  };
  auto merge = [&]() {
    const int count = sh.count;
    threshold = max(threshold, merge_candidates(sh, k, keys));
    if (threshold != 0) least = key_value(threshold);
    keys = min(k, count);
    merged = true;
    return count <= kRoom;
  };

  int stage = 0;
  for (int base = first; base < end;) {
    // windows double up to kWindow tiles: a threshold from as many elements as came before
    // lets some k of a window pass
    const int stop = min(end, base + min(kWindow * kStep, max(kStep, base - first)));
    bool full = false;
    for (int tile = base; tile < stop; tile += kStep) {
      const int mine = tile + own;
      async_wait<kStages - 1>();
      if constexpr (kShifted) __syncwarp();
      const uint4* slot = ring + stage * (kSlots * kWarps);
      Part<DT> v;
      auto read = [&](auto word) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          if constexpr (kShifted)
            v.put(i, shifted<word.value, sizeof(T) < 4>(slot[i * kRun], slot[i * kRun + 1], 8 * (shift % 4)));
          else v.put(i, slot[i * kRun]);
        }
      };
      if constexpr (kShifted) {  // the same way for the whole block, so no word is chosen by data
        switch (shift / 4) {
          case 0: read(std::integral_constant<int, 0>()); break;
          case 1: read(std::integral_constant<int, 1>()); break;
          case 2: read(std::integral_constant<int, 2>()); break;
          default: read(std::integral_constant<int, 3>());
        }
      } else {
        read(std::integral_constant<int, 0>());
      }
      if (tile + kStep > end) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (mine + i * kThreads >= end) v.put(i, make_uint4(v.empty(), v.empty(), v.empty(), v.empty()));
      }
      if (tile == first) {
        least = group_bound(v.maximum(), k, sh.groups);
        if (least != kNegInf) threshold = make_key(least, 0xffffffffu);
        m = sh.groups.largest;
        set_bound();
      }
      float4 sums = m != kNegInf ? v.exp_sums(m) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (!(sums.x < bound && sums.y < bound && sums.z < bound && sums.w < bound)) {
        constexpr float kBelow = 1.f - 0x1p-10f;  // of no element above m
        // without a reference yet (a first tile of -inf and NaN alone) the sums say nothing
        if (m == kNegInf || !(sums.x < kBelow && sums.y < kBelow && sums.z < kBelow && sums.w < kBelow)) {
          const float top = v.maximum();
          if (top > m || !((sums.x + sums.y) + (sums.z + sums.w) < INFINITY)) {  // a new reference; or NaN or +inf
            const float m2 = fmaxf(m, top);
            v.clean();
            s *= m2 != kNegInf ? ex2_approx((m - m2) * kLog2e) : 0.f;
            m = m2;
            set_bound();
            sums = m != kNegInf ? v.exp_sums(m) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        for (unsigned left = v.reach(least, sums, bound); left; left &= left - 1) {
          const int i = __ffs(left) - 1;  // its value comes from the ring: registers have no index
          const T* at =
              reinterpret_cast<const T*>(reinterpret_cast<const unsigned char*>(slot + i / kVec * kRun) + shift);
          full |= push_candidate(sh, clean_logit<DT>(at[i % kVec]), (mine + i / kVec * kThreads) * kVec + i % kVec, least,
                                 threshold, spare);
        }
      }
      s += (sums.x + sums.y) + (sums.z + sums.w);
      __syncwarp();  // the stage has been read
      load(tile + kStages * kStep, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if (__syncthreads_or(full) && !merge()) {
      // The window held more candidates than the block has room for: it is looked at again,
      // kRescan elements at a time.  Where these overflow too, the threshold (the k-th best
      // of those that fitted) leaves at least kRoom - 3 k of them below.
      keys = drop_candidates(sh, k, base * kVec);
      for (int e0 = base * kVec; e0 < stop * kVec; e0 += kRescan) {
        bool again = true;
        while (again) {
          bool over = false;
          for (int e = e0 + threadIdx.x; e < min(stop * kVec, e0 + kRescan); e += kThreads) {
            const float value = clean_logit<DT>(x[e]);
            if (value >= least) over |= push_candidate(sh, value, e, least, threshold, spare);
          }
          again = __syncthreads_or(over) && !merge();
          if (again) keys = drop_candidates(sh, k, e0);
        }
      }
    }
    set_bound();
    base = stop;
  }
  async_wait<0>();
  const int tail = pieces * kVec;
  if (seg == p.num_segments - 1 && tail < p.vocab_size) {  // one element a thread
    __syncthreads();                                       // the count has been set
    if (static_cast<int>(threadIdx.x) < p.vocab_size - tail) {
      const float value = clean_logit<DT>(x[tail + threadIdx.x]);
      if (value != kNegInf) {
        const float m2 = fmaxf(m, value);
        s = s * ex2_approx((m - m2) * kLog2e) + ex2_approx((value - m2) * kLog2e);
        m = m2;
        if (value >= least) push_candidate(sh, value, tail + threadIdx.x, least, threshold, spare);
      }
    }
  }

  warp_state(m, s);
  if (lane == 0) {
    sh.m[warp] = m;
    sh.s[warp] = s;
  }
  __syncthreads();
  if (!merged || sh.count > keys) merge_candidates(sh, k, keys);  // else `best` is up to date
  const long long part = row * p.num_segments + seg;
  if (warp == 0) {
    m = lane < kWarps ? sh.m[lane] : kNegInf;
    s = lane < kWarps ? sh.s[lane] : 0.f;
    warp_state(m, s);
    if (lane == 0) p.state[part] = make_float2(m, s);
  }
  if (threadIdx.x < k) p.keys[part * k + threadIdx.x] = sh.best[threadIdx.x];
}

// A beam of a sequence: its score, its row's maximum and the log of the sum against it, as
// log_sum = power x log 2 + rest.
struct Beam {
  float score, m;
  int power;
  float rest;
};

// Sums are joined as whole numbers of 2^-32 (exact in any order; their sum is 1 or more, so
// the rounding of each costs 2^-33 of it at most), and their logarithm is kept in the two parts of struct Beam, each to
// 2^-25 or so: the SM has two fp64 lanes, and fp64 sums and logarithms took half the join's
// time.
__device__ __forceinline__ void set_log(Beam& b, unsigned long long sum) {
  const int top = 63 - __clzll(static_cast<long long>(sum | 1));
  // sum = 2^top (1 + f), f in [0, 1); above sqrt 2 as 2^(top + 1) (1 - g)
  const unsigned long long f = sum << (63 - top) & 0x7fffffffffffffffull;  // f x 2^63
  const bool upper = f > 0x3504f333f9de6484ull;
  b.power = top - 32 + (upper ? 1 : 0);
  b.rest = log1pf(upper ? static_cast<float>(0x8000000000000000ull - f) * -0x1p-64f : static_cast<float>(f) * 0x1p-63f);
}

// Candidates in order: by score, then the lower beam, then the key (larger logit, lower
// token).  Scores are fp64 bits as integers of the same order.  Key 0 is none and comes last.
struct Candidate {
  long long score;
  Key key;
  int beam;
};
__device__ __forceinline__ long long order_of(double score) {
  const long long bits = __double_as_longlong(score);
  return bits ^ ((bits >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ Candidate candidate_of(const Beam* beams, Key key, int beam) {
  const Beam b = beams[beam];
  const double log_sum = b.power * 0.69314718055994530942 + static_cast<double>(b.rest);
  return {order_of(b.score + ((key_value(key) - static_cast<double>(b.m)) - log_sum)), key, beam};
}
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

constexpr int kJoin = 1024;  // candidates that pass the first threshold
constexpr int kHeld = 4;     // keys a thread loads ahead

// One block a sequence: the rows' states are joined, then the segments' candidates.  Most
// fall to a threshold on their fp32 scores, held with the scores' error bounds so that
// none of the best can be lost; the rest are ranked by their fp64 scores.  Bound by latency:
// loads, two ranked bounds and the last ranking follow one another, 3 to 6 us behind the
// segments; its blocks are brought up while these still run (as a launch of its own behind
// them it cost 2 us more).
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamParams p) {
  previous_done();  // the segments are done and their results there
  extern __shared__ Beam beams[];  // [num_beams]
  __shared__ Key kept[kJoin];
  __shared__ float2 bounds[kJoin];
  __shared__ unsigned short owner[kJoin];
  __shared__ Candidate last[kThreads];
  __shared__ long long scores[kThreads];
  __shared__ GroupShared groups;
  __shared__ Candidate found[kWarps];
  __shared__ int count, few;
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
  if (threadIdx.x == 0) count = few = 0;
  for (int w = warp; w < p.num_beams; w += kWarps) {
    const float2* st = p.state + (seq * p.num_beams + w) * p.num_segments;
    const float cum = p.beam_scores[seq * p.num_beams + w];
    float2 own = lane < p.num_segments ? st[lane] : make_float2(kNegInf, 0.f);
    float m = own.x;
    for (int i = lane + 32; i < p.num_segments; i += 32) m = fmaxf(m, st[i].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    unsigned long long sum = 0;
    for (int i = lane; i < p.num_segments; i += 32) {
      if (i != lane) own = st[i];
      if (m != kNegInf) sum += __float2ull_rn(own.y * ex2_approx((own.x - m) * kLog2e) * 0x1p32f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) {
      Beam b;
      b.score = m == kNegInf ? kNegInf : fminf(fmaxf(cum, kNegInf), largest<PA_F32>());
      b.m = m;
      set_log(b, sum);
      beams[w] = b;
    }
  }
  __syncthreads();
  // the beam of candidate c: c + 0.5 is exact and n far below 2^21, so the quotient's error
  // cannot reach a whole number
  const float inverse = 1.f / static_cast<float>(per_beam);
  auto beam_of = [&](int c) { return static_cast<int>((static_cast<float>(c) + 0.5f) * inverse); };
  // fp32 score of a candidate less and plus what it may be off: every term and sum is rounded
  // once, so that is less than 2^-22 of the terms' magnitudes
  auto range_of = [&](int w, Key key) {
    const Beam b = beams[w];
    const float rel = key_value(key) - b.m, log_sum = b.power * 0.69314718f + b.rest;
    const float score = b.score + (rel - log_sum);
    const float error = 0x1p-21f * (fabsf(b.score) + fabsf(rel) + fabsf(log_sum) + 1.f);
    return key == 0 || b.score == kNegInf ? make_float2(kNegInf, kNegInf) : make_float2(score - error, score + error);
  };
  float top = kNegInf;
  float2 range[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    range[i] = make_float2(kNegInf, kNegInf);
    if (held[i] != 0) range[i] = range_of(beam_of(threadIdx.x + i * kThreads), held[i]);
    top = fmaxf(top, range[i].x);
  }
  for (int c = threadIdx.x + kHeld * kThreads; c < n; c += kThreads) top = fmaxf(top, range_of(beam_of(c), keys[c]).x);
  const float bound = group_bound(top, p.num_candidates, groups);
  auto keep = [&](int c, Key key, float2 r) {
    if (r.y == kNegInf || r.y < bound) return;
    const int at = atomicAdd(&count, 1);
    if (at >= kJoin) return;
    kept[at] = key;
    owner[at] = beam_of(c);
    bounds[at] = r;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) keep(threadIdx.x + i * kThreads, held[i], range[i]);
  for (int c = threadIdx.x + kHeld * kThreads; c < n; c += kThreads) {
    const Key key = keys[c];
    keep(c, key, range_of(beam_of(c), key));
  }
  __syncthreads();
  const int m = count;
  if (m <= kJoin) {
    // Long sorted lists side by side make uneven groups; where much is left, a second
    // threshold on what lies in no order now.  fp64 scores are for the few behind it.
    float least = kNegInf;
    if (m > kFew) {
      float best = kNegInf;
      for (int i = threadIdx.x; i < m; i += kThreads) best = fmaxf(best, bounds[i].x);
      least = group_bound(best, p.num_candidates, groups);
    }
    for (int i = threadIdx.x; i < m; i += kThreads) {
      if (bounds[i].y < least) continue;
      const int at = atomicAdd(&few, 1);
      if (at >= kThreads) continue;
      const Candidate c = candidate_of(beams, kept[i], owner[i]);
      last[at] = c;
      scores[at] = c.score;
    }
    __syncthreads();
    if (few <= kThreads) {
      const int i = threadIdx.x;
      if (i < few) {
        const long long mine = scores[i];
        int rank = 0, equal = 0;
#pragma unroll 4
        for (int j = 0; j < few; ++j) {
          const long long other = scores[j];
          rank += other > mine;
          equal += other == mine;
        }
        if (equal > 1) {
          const Candidate me = last[i];
#pragma unroll 4
          for (int j = 0; j < few; ++j) {
            const Candidate c = last[j];
            rank += (c.score == mine) & ((c.beam < me.beam) | ((c.beam == me.beam) & (c.key > me.key)));
          }
        }
        if (rank < p.num_candidates) write_out(p, seq, rank, last[i]);
      } else if (i < p.num_candidates) {
        write_out(p, seq, i, {0, 0, 0});
      }
      return;
    }
  }
  // more near-equal candidates than fit: one after the other
  Candidate given = {0x7fffffffffffffffll, ~0ull, -1};
  for (int k = 0; k < p.num_candidates; ++k) {
    Candidate best = {0, 0, 0};
    for (int c = threadIdx.x; c < n; c += kThreads) {
      const Key key = keys[c];
      const int w = beam_of(c);
      if (key == 0 || beams[w].score == kNegInf) continue;
      const Candidate cand = candidate_of(beams, key, w);
      if (before(given, cand) && before(cand, best)) best = cand;
    }
    for (int o = 16; o; o >>= 1) {
      const Candidate other = {__shfl_xor_sync(~0u, best.score, o), __shfl_xor_sync(~0u, best.key, o),
                               __shfl_xor_sync(~0u, best.beam, o)};
      if (before(other, best)) best = other;
    }
    if (lane == 0) found[warp] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
      if (before(found[w], best)) best = found[w];
    __syncthreads();
    if (threadIdx.x == 0) write_out(p, seq, k, best);
    given = best;
  }
}

}  // namespace

// Segments of a row: rows are cut as long as the grid fits at once (four blocks an SM), but
// no finer than a tile.  (128 rows of 131,072 bf16, 256 of 262,144 fp32: 20 and 48 us, with as
// many as six blocks an SM would take 30 and 63.  16 rows of 131,072 bf16: 8.3 us, with half
// tiles 9.7; four of 32,000 fp32: 7.1, with two tiles 8.1.)
int beam_segments(long long rows, int vocab_size, int elem_bytes) {
  const long long fit = 152 * 4 / rows, least = kTileBytes / elem_bytes, most = (vocab_size + least - 1) / least;
  return static_cast<int>(fit < 1 ? 1 : fit < most ? fit : most);
}

template <int DT, bool kShifted>
static cudaError_t launch_segments(const BeamParams& p, cudaStream_t stream) {
  const int smem = sizeof(SegmentShared) + kStages * kWarps * ring_slots<kShifted>() * 16;
  const cudaError_t e = set_smem<beam_segment_kernel<DT, kShifted>>(smem);
  if (e != cudaSuccess) return e;
  return launch_early(beam_segment_kernel<DT, kShifted>, dim3(p.num_segments, p.num_seqs * p.num_beams), kThreads,
                      smem, 1, p, stream);
}

template <int DT>
static cudaError_t launch_type(const BeamParams& p, cudaStream_t stream) {
  const bool one = p.num_seqs * p.num_beams == 1;
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                       (one || p.row_stride * Elem<DT>::bytes % 16 == 0);
  // rows on the grid are read as they lie (256 rows of 262,144 fp32 48 us, of 262,143 58; 600 of
  // 131,072 bf16 37, of 131,071 42)
  return aligned ? launch_segments<DT, false>(p, stream) : launch_segments<DT, true>(p, stream);
}

cudaError_t launch_beam_select(const BeamParams& p, int dtype, cudaStream_t stream) {
  const cudaError_t e = dtype == PA_F32   ? launch_type<PA_F32>(p, stream)
                        : dtype == PA_F16 ? launch_type<PA_F16>(p, stream)
                                          : launch_type<PA_BF16>(p, stream);
  if (e != cudaSuccess) return e;
  return launch_early(beam_join_kernel, dim3(p.num_seqs), kThreads, p.num_beams * sizeof(Beam), 1, p, stream);
}

}  // namespace pa
