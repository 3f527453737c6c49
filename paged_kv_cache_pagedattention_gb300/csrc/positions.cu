// Positions and cache slots of a step's new tokens, from request lengths, block tables and the
// grids of the media in the sequences.
//
//   token i of a sequence (i counts from its start) whose media are (s, F, R, C, e): first
//   token, frames, rows, columns, positions from one frame to the next.  A medium has
//   S = F R C tokens and takes X = max((F - 1) e + 1, R, C) positions, so what stands behind
//   it is D = S - X positions nearer:
//     text             i - sum of D over the media before it, on every axis
//     token (f, r, c)  b + (f e, r, c), b = s - sum of D over the media before this one
//   slot = table[i / block_size] * block_size + i % block_size
//
// Bound by latency: some bytes a token, and a chain of starts -> lengths and media -> sums ->
// stores.  A warp serves up to 128 tokens of one request (four a lane).  It looks all media of the
// request through once, 128 on their way together, for their order and for the sum of D before its
// tokens; then it steps through those that its tokens lie in, 32 a time, a prefix sum over the warp
// giving D before each (15 prompts of 8,191 tokens with some 525 media each: 14.5 us when every warp
// took prefix sums over all of them).  A step's tokens and requests need at most requests + tokens / 128 warps, and
// warp w finds its piece by itself: request r's pieces begin at r + start(r) / 128, which no
// other request's pieces reach, so no launch has to count first.
#include <limits.h>

#include "launch.cuh"
#include "pa_common.cuh"

namespace pa {

namespace {

constexpr int kPerLane = 4, kPiece = 32 * kPerLane;
constexpr int kThreads = 128;
constexpr int kBatch = 4;

// One medium, as lanes hold it.
struct Medium {
  int first, rows, cols, step;
  long long size;  // tokens, 0 where there is no medium
  long long extent;
  bool ok;
};

__device__ __forceinline__ Medium load_medium(const int32_t* media, long long i, long long end) {
  Medium m = {INT_MAX, 1, 1, 0, 0, 0, true};
  if (i >= end) return m;
  const int32_t* r = media + 5 * i;
  const int frames = r[1];
  m.first = r[0];
  m.rows = r[2];
  m.cols = r[3];
  m.step = r[4];
  // all in range where the products are: none passes 2^62
  m.ok = m.first >= 0 && frames >= 1 && m.rows >= 1 && m.cols >= 1 && m.step >= 0;
  const long long plane = (long long)m.rows * m.cols;
  m.ok = m.ok && plane <= INT_MAX;
  m.size = plane * frames;
  m.extent = max((long long)(frames - 1) * m.step + 1, (long long)max(m.rows, m.cols));
  m.ok = m.ok && m.size <= INT_MAX && m.first + m.size <= INT_MAX && m.extent <= INT_MAX;
  if (!m.ok) m.size = m.extent = 0;
  return m;
}

__device__ __forceinline__ void write_token(const PositionsParams& p, int row, long long a, long long b, long long c,
                                            long long slot) {
  if (p.positions) {
    p.positions[row] = static_cast<int>(a);
    if (p.num_axes == 3) {
      p.positions[(long long)p.total_tokens + row] = static_cast<int>(b);
      p.positions[2ll * p.total_tokens + row] = static_cast<int>(c);
    }
  }
  if (p.slot_mapping) p.slot_mapping[row] = slot;
}

__global__ void __launch_bounds__(kThreads) positions_kernel(const PositionsParams p) {
  const int n = p.num_seqs, lane = threadIdx.x & 31;
  previous_done();
  // every block looks at all starts: where one is wrong, no token is placed
  int bad = 0;
  for (int i = threadIdx.x; i <= n; i += kThreads) {
    const int v = p.query_start_loc[i];
    bad |= i == 0 ? v != 0 : v < p.query_start_loc[i - 1];
    bad |= i == n && v != p.total_tokens;
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PA_ERRFLAG_QUERY);
    for (long long t = (long long)blockIdx.x * kThreads + threadIdx.x; t < p.total_tokens;
         t += (long long)gridDim.x * kThreads)
      write_token(p, static_cast<int>(t), 0, 0, 0, -1);
    return;
  }
  // the last request whose pieces begin at or before this warp's place
  const int w = static_cast<int>(((long long)blockIdx.x * kThreads + threadIdx.x) >> 5);
  int r = 0;
  for (int hi = n; hi - r > 1;) {
    const int mid = r + (hi - r) / 2;
    if (mid + p.query_start_loc[mid] / kPiece <= w) r = mid; else hi = mid;
  }
  const int q0 = p.query_start_loc[r], q_len = p.query_start_loc[r + 1] - q0;
  const long long first_row = (long long)(w - r - q0 / kPiece) * kPiece;  // in the request
  if (first_row >= q_len) return;
  const int count = min(kPiece, q_len - static_cast<int>(first_row));
  const int seq_len = p.seq_lens[r];
  const bool len_ok = seq_len >= q_len &&
                      (!p.slot_mapping || seq_len <= (long long)p.max_blocks_per_seq * p.block_size);
  const int i0 = len_ok ? seq_len - q_len + static_cast<int>(first_row) : 0;  // the piece's first token
  const int i1 = i0 + count - 1;
  unsigned flags = len_ok ? 0u : seq_len < q_len ? PA_ERRFLAG_QUERY : PA_ERRFLAG_SEQ_LEN;

  // the tokens' table entries come while the media are looked through
  int entry[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    entry[j] = -1;
    if (len_ok && p.slot_mapping && lane + 32 * j < count)
      entry[j] = p.block_tables[(long long)r * p.max_blocks_per_seq + (i0 + lane + 32 * j) / p.block_size];
  }

  long long at[kPerLane][3];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) at[j][0] = at[j][1] = at[j][2] = i0 + min(lane + 32 * j, count - 1);
  if (len_ok && p.media_start) {
    const long long m0 = p.media_start[r], m1 = p.media_start[r + 1];
    bool ok = 0 <= m0 && m0 <= m1 && m1 <= p.num_media;
    // All media once, kBatch tiles of 32 on their way together: whether they are in order and range, how
    // many begin at or before the piece's first token, and the positions that those leave out.
    long long saved = 0, end = 0;
    int begun = 0;
    for (long long k = m0; ok && k < m1; k += 32 * kBatch) {
      Medium m[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) m[u] = load_medium(p.media, k + 32 * u + lane, m1);
      bool good = true;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const long long behind = m[u].first + m[u].size;  // the lanes behind the last medium: INT_MAX
        long long prev = __shfl_up_sync(0xffffffffu, behind, 1);
        if (lane == 0) prev = end;
        good = good && m[u].ok && m[u].first >= prev;
        end = __shfl_sync(0xffffffffu, behind, 31);
        if (m[u].size > 0 && m[u].first <= i0) {
          saved += m[u].size - m[u].extent;
          ++begun;
        }
      }
      ok = __all_sync(0xffffffffu, good);
    }
    for (int o = 16; o >= 1; o >>= 1) {
      saved += __shfl_xor_sync(0xffffffffu, saved, o);
      begun += __shfl_xor_sync(0xffffffffu, begun, o);
    }
    // From the last of those on, media that some token of the piece lies in or behind
    const long long from = m0 + max(begun - 1, 0);
    Medium m = load_medium(p.media, ok ? from + lane : 0, ok ? m1 : 0);
    if (begun > 0) saved -= __shfl_sync(0xffffffffu, m.size - m.extent, 0);
    for (long long k = from; ok && k < m1; k += 32) {
      if (__shfl_sync(0xffffffffu, m.first, 0) > i1) break;
      const Medium next = load_medium(p.media, k + 32 + lane, m1);
      long long sum = m.size - m.extent;
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const long long before = saved + sum - (m.size - m.extent);
      const int highest = __shfl_sync(0xffffffffu, m.first, 31);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        const int i = i0 + min(lane + 32 * j, count - 1);
        int c = 0;  // media of the tile that begin at or before token i
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
          if (__shfl_sync(0xffffffffu, m.first, c + o - 1) <= i) c += o;
        if (highest <= i) c = 32;
        const int src = max(c - 1, 0);
        const long long s_before = __shfl_sync(0xffffffffu, before, src);
        const int s_first = __shfl_sync(0xffffffffu, m.first, src), s_rows = __shfl_sync(0xffffffffu, m.rows, src);
        const int s_cols = __shfl_sync(0xffffffffu, m.cols, src), s_step = __shfl_sync(0xffffffffu, m.step, src);
        const int s_size = __shfl_sync(0xffffffffu, static_cast<int>(m.size), src);
        const int s_extent = __shfl_sync(0xffffffffu, static_cast<int>(m.extent), src);
        const int inside = i - s_first;
        if (c > 0 && inside < s_size) {
          const long long base = s_first - s_before;
          const int plane = s_rows * s_cols, f = inside / plane, cell = inside - f * plane;
          at[j][0] = base + (long long)f * s_step;
          at[j][1] = base + cell / s_cols;
          at[j][2] = base + cell % s_cols;
        } else if (c > 0) {
          at[j][0] = at[j][1] = at[j][2] = i - s_before - s_size + s_extent;
        }
      }
      saved += __shfl_sync(0xffffffffu, sum, 31);
      m = next;
    }
    if (!ok) flags |= PA_ERRFLAG_MEDIA;
  }
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    if (lane + 32 * j >= count) continue;
    const int row = q0 + static_cast<int>(first_row) + lane + 32 * j;
    const bool reach = max(at[j][0], max(at[j][1], at[j][2])) <= INT_MAX && at[j][0] >= 0;
    if (flags || !reach) {
      if (!reach) flag_error(p.err, PA_ERRFLAG_MEDIA);
      write_token(p, row, 0, 0, 0, -1);
      continue;
    }
    long long slot = -1;
    if (p.slot_mapping) {
      if (entry[j] >= 0 && entry[j] < p.num_blocks)
        slot = (long long)entry[j] * p.block_size + (i0 + lane + 32 * j) % p.block_size;
      else
        flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
    }
    write_token(p, row, at[j][0], at[j][1], at[j][2], slot);
  }
  if (flags && lane == 0) flag_error(p.err, flags);
}

}  // namespace

cudaError_t launch_positions(const PositionsParams& p, cudaStream_t stream) {
  const long long warps = (long long)p.num_seqs + p.total_tokens / kPiece;
  return launch_early(positions_kernel, dim3(static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads)), kThreads,
                      0, 1, p, stream);
}

}  // namespace pa
