// Pages of sequences: fork (children take their parents' blocks), append (blocks and slots
// of the next tokens, copy-on-write of shared tails) and release.  [AGENTIC] "統一分頁 +
// 共用池": one pool, reference counts, copy-on-write; [LINEAGE] "Prefix reuse": a shared
// block that is not yet full is copied before a branch writes into it.
//
// ref_counts[b] is the number of table rows that hold block b; a block is free at 0.
// Everything is whole numbers and every choice goes by row order and block number, so a
// call's result does not depend on which thread comes first.
#include "pa_common.cuh"

namespace pa {

namespace {

constexpr int kTableThreads = 256;

__device__ __forceinline__ int blocks_of(int tokens, int block_size) {
  return static_cast<int>(((long long)tokens + block_size - 1) / block_size);
}

__device__ __forceinline__ bool length_ok(const SequenceParams& p, int len) {
  return len >= 0 && len <= (long long)p.max_blocks_per_seq * p.block_size;
}

// Grid: x = child, y = slice of its row.
__global__ void __launch_bounds__(kTableThreads) fork_kernel(const SequenceParams p) {
  const int child = blockIdx.x;
  const int parent = p.parents[child];
  int len = 0;
  if (parent >= p.num_parents) {
    if (blockIdx.y == 0 && threadIdx.x == 0) flag_error(p.err, PA_ERRFLAG_PARENT);
  } else if (parent >= 0) {
    len = p.parent_lens[parent];
    if (!length_ok(p, len)) {
      if (blockIdx.y == 0 && threadIdx.x == 0) flag_error(p.err, PA_ERRFLAG_SEQ_LEN);
      len = 0;
    }
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.seq_lens[child] = len;
  if (len == 0) return;
  const int blocks = blocks_of(len, p.block_size);
  const int32_t* src = p.parent_tables + (long long)parent * p.max_blocks_per_seq;
  int32_t* dst = p.block_tables + (long long)child * p.max_blocks_per_seq;
  for (int j = blockIdx.y * kTableThreads + threadIdx.x; j < blocks; j += gridDim.y * kTableThreads) {
    const int b = src[j];
    dst[j] = b;
    if (b >= p.num_blocks) flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
    else if (b >= 0) atomicAdd(p.ref_counts + b, 1);
  }
}

// One block a row: its length is read by every thread before one of them writes it.
__global__ void __launch_bounds__(1024) release_kernel(const SequenceParams p) {
  const int row = blockIdx.x;
  const int len = p.seq_lens[row];
  const int keep = p.keep_lens ? p.keep_lens[row] : 0;
  __syncthreads();
  if (!length_ok(p, len) || keep < 0) {
    if (threadIdx.x == 0) flag_error(p.err, PA_ERRFLAG_SEQ_LEN);
    return;
  }
  if (keep >= len) return;
  if (threadIdx.x == 0) p.seq_lens[row] = keep;
  const int32_t* table = p.block_tables + (long long)row * p.max_blocks_per_seq;
  const int last = blocks_of(len, p.block_size);
  for (int j = blocks_of(keep, p.block_size) + threadIdx.x; j < last; j += blockDim.x) {
    const int b = table[j];
    if (b >= p.num_blocks) {
      flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
    } else if (b >= 0 && atomicSub(p.ref_counts + b, 1) <= 0) {  // held by no row: put it back
      atomicAdd(p.ref_counts + b, 1);
      flag_error(p.err, PA_ERRFLAG_REF_COUNT);
    }
  }
}

constexpr int kAppendThreads = 1024;

// Exclusive prefix sum of v over the block, and the block's total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int incl = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kAppendThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  __syncthreads();
  return before + incl - v;
}

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const SequenceParams p) {
  __shared__ int warp_sums[kAppendThreads / 32];
  __shared__ int bad;
  const int n = p.num_rows, bs = p.block_size;
  int32_t* tail = p.ws_tail;    // block that row i would write into and shares, else -1
  int32_t* need = p.ws_need;    // blocks row i takes, times two, plus one if the first replaces its tail
  int32_t* first = p.ws_first;  // where they start in `fresh`
  int32_t* fresh = p.ws_fresh;  // the blocks given out, in order
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  unsigned flags = 0;
  if (threadIdx.x == 0 && (p.query_start_loc[0] != 0 || p.query_start_loc[n] != p.total_tokens))
    flags |= PA_ERRFLAG_QUERY;
  for (int i = threadIdx.x; i < n; i += kAppendThreads) {
    const int len = p.seq_lens[i];
    const long long add = (long long)p.query_start_loc[i + 1] - p.query_start_loc[i];
    tail[i] = -1;
    need[i] = 0;
    if (add < 0) {
      flags |= PA_ERRFLAG_QUERY;
      continue;
    }
    if (!length_ok(p, len) || len + add > (long long)p.max_blocks_per_seq * bs || len + add > 0x7fffffff) {
      flags |= PA_ERRFLAG_SEQ_LEN;
      continue;
    }
    if (add == 0) continue;
    need[i] = 2 * (blocks_of(static_cast<int>(len + add), bs) - blocks_of(len, bs));
    if (len % bs) {
      const int b = p.block_tables[(long long)i * p.max_blocks_per_seq + len / bs];
      if (b < 0 || b >= p.num_blocks) flags |= PA_ERRFLAG_BLOCK_TABLE;
      else if (p.ref_counts[b] < 1) flags |= PA_ERRFLAG_REF_COUNT;
      else if (p.ref_counts[b] > 1) tail[i] = b;
    }
  }
  if (flags) {
    flag_error(p.err, flags);
    atomicOr(&bad, 1);
  }
  __syncthreads();
  if (!bad) {
    // a shared tail is copied by every row that writes it but, where they are all of its
    // holders, the last
    for (int i = threadIdx.x; i < n; i += kAppendThreads) {
      const int b = tail[i];
      if (b < 0) continue;
      int lower = 0;
      for (int j = 0; j < i; ++j) lower += tail[j] == b;
      if (lower < p.ref_counts[b] - 1) need[i] += 1;
    }
  }
  __syncthreads();
  int base = 0;
  if (!bad) {
    for (int i0 = 0; i0 < n; i0 += kAppendThreads) {
      const int i = i0 + threadIdx.x;
      const int v = i < n ? (need[i] >> 1) + (need[i] & 1) : 0;
      int total;
      const int before = block_scan(v, warp_sums, total);
      if (i < n) first[i] = base + before;
      base += total;
    }
    int found = 0;
    for (int b0 = 0; b0 < p.num_blocks && found < base; b0 += kAppendThreads) {
      const int b = b0 + threadIdx.x;
      const int v = b < p.num_blocks && p.ref_counts[b] == 0;
      int total;
      const int at = found + block_scan(v, warp_sums, total);
      if (v && at < base) fresh[at] = b;
      found += total;
    }
    if (found < base) {
      if (threadIdx.x == 0) {
        flag_error(p.err, PA_ERRFLAG_POOL);
        bad = 1;
      }
    }
  }
  __syncthreads();
  const bool refused = bad != 0;
  for (int i = threadIdx.x; i < n; i += kAppendThreads) {
    long long src = 0, dst = 0;
    if (!refused) {
      int32_t* table = p.block_tables + (long long)i * p.max_blocks_per_seq;
      const int len = p.seq_lens[i];
      int at = first[i];
      if (need[i] & 1) {
        src = tail[i];
        dst = fresh[at++];
        table[len / bs] = static_cast<int32_t>(dst);
        atomicSub(p.ref_counts + src, 1);
        p.ref_counts[dst] = 1;
      }
      int j = blocks_of(len, bs);
      for (int k = need[i] >> 1; k; --k, ++j) {
        const int b = fresh[at++];
        table[j] = b;
        p.ref_counts[b] = 1;
      }
    }
    p.block_mapping[2 * (long long)i] = src;
    p.block_mapping[2 * (long long)i + 1] = dst;
  }
  __syncthreads();
  for (int t = threadIdx.x; t < p.total_tokens; t += kAppendThreads) {
    long long slot = -1;
    if (!refused) {
      int lo = 0, hi = n;  // first row with query_start_loc[row + 1] > t
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (p.query_start_loc[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
      }
      const int pos = p.seq_lens[lo] + (t - p.query_start_loc[lo]);
      slot = (long long)p.block_tables[(long long)lo * p.max_blocks_per_seq + pos / bs] * bs + pos % bs;
    }
    p.slot_mapping[t] = slot;
  }
  __syncthreads();
  if (!refused)
    for (int i = threadIdx.x; i < n; i += kAppendThreads)
      p.seq_lens[i] += p.query_start_loc[i + 1] - p.query_start_loc[i];
}

}  // namespace

cudaError_t launch_fork_blocks(const SequenceParams& p, cudaStream_t stream) {
  const int slices = (p.max_blocks_per_seq + 4 * kTableThreads - 1) / (4 * kTableThreads);
  fork_kernel<<<dim3(p.num_rows, slices < 1024 ? slices : 1024), kTableThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_release_blocks(const SequenceParams& p, cudaStream_t stream) {
  release_kernel<<<p.num_rows, 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_append_blocks(const SequenceParams& p, cudaStream_t stream) {
  append_kernel<<<1, kAppendThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
