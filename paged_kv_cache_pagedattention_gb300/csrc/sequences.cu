// Pages of sequences: fork (children take their parents' blocks), append (blocks and slots
// of the next tokens, copy-on-write of shared tails) and release.  [AGENTIC] "統一分頁 +
// 共用池": one pool, reference counts, copy-on-write; [LINEAGE] "Prefix reuse": a shared
// block that is not yet full is copied before a branch writes into it.
//
// ref_counts[b] is the number of table rows that hold block b; a block is free at 0.
// Everything is whole numbers and every choice goes by row order and block number, so a
// call's result does not depend on which thread comes first.
#include <cooperative_groups.h>

#include <algorithm>

#include "launch.cuh"
#include "pa_common.cuh"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kTableThreads = 256;
constexpr int kTableUnroll = 4;

__device__ __forceinline__ int blocks_of(int tokens, int block_size) {
  return static_cast<int>((static_cast<unsigned>(tokens) + static_cast<unsigned>(block_size) - 1u) /
                          static_cast<unsigned>(block_size));
}

__device__ __forceinline__ bool length_ok(const SequenceParams& p, int len) {
  return len >= 0 && len <= (long long)p.max_blocks_per_seq * p.block_size;
}

// Grid: x = child, y = slice of its row.  Four entries a thread on their way at once.  Bound by
// latency in short rows (2 us), by the counts' atomics in long ones (1,024 children of 8,192
// blocks: 13 us).
__global__ void __launch_bounds__(kTableThreads) fork_kernel(const SequenceParams p) {
  previous_done();
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
  const int blocks = blocks_of(len, p.block_size);
  const int32_t* src = p.parent_tables + (long long)parent * p.max_blocks_per_seq;
  int32_t* dst = p.block_tables + (long long)child * p.max_blocks_per_seq;
  const int step = gridDim.y * kTableThreads;
  for (int j0 = blockIdx.y * kTableThreads + threadIdx.x; j0 < blocks; j0 += kTableUnroll * step) {
    int b[kTableUnroll];
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) b[u] = j0 + u * step < blocks ? src[j0 + u * step] : -1;
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) {
      if (j0 + u * step < blocks) dst[j0 + u * step] = b[u];
      if (b[u] >= p.num_blocks) flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
      else if (b[u] >= 0) atomicAdd(p.ref_counts + b[u], 1);
    }
  }
}

// The same by parents, grid: x = parent, y = slice of its row, z = part of the children, each
// of p.fork_part.  A parent's entries are read once for all of a part's children and counted
// up once, by the number of them, so there are as many fewer atomics.
constexpr int kForkPart = 1024;  // children of a part at most
constexpr int kForkMost = 1 << 20;
__global__ void __launch_bounds__(kTableThreads) fork_parents_kernel(const SequenceParams p) {
  __shared__ int children[kForkPart];
  __shared__ int count;
  const int parent = blockIdx.x;
  if (threadIdx.x == 0) count = 0;
  previous_done();
  const int len_given = p.parent_lens[parent];
  __syncthreads();
  const int first = blockIdx.z * p.fork_part, past = min(p.num_rows, first + p.fork_part);
  for (int c = first + threadIdx.x; c < past; c += kTableThreads) {
    const int from = p.parents[c];
    if (from == parent) {
      children[atomicAdd(&count, 1)] = c;
    } else if (parent == 0 && blockIdx.y == 0 && (from < 0 || from >= p.num_parents)) {
      p.seq_lens[c] = 0;
      if (from >= 0) flag_error(p.err, PA_ERRFLAG_PARENT);
    }
  }
  __syncthreads();
  const int held = count;
  if (held == 0) return;
  const int len = length_ok(p, len_given) ? len_given : 0;
  if (blockIdx.y == 0) {
    if (threadIdx.x == 0 && len != len_given) flag_error(p.err, PA_ERRFLAG_SEQ_LEN);
    for (int c = threadIdx.x; c < held; c += kTableThreads) p.seq_lens[children[c]] = len;
  }
  const int blocks = blocks_of(len, p.block_size);
  const int32_t* src = p.parent_tables + (long long)parent * p.max_blocks_per_seq;
  const int step = gridDim.y * kTableThreads;
  for (int j0 = blockIdx.y * kTableThreads + threadIdx.x; j0 < blocks; j0 += kTableUnroll * step) {
    int b[kTableUnroll];
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) b[u] = j0 + u * step < blocks ? src[j0 + u * step] : -1;
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) {
      if (b[u] >= p.num_blocks) flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
      else if (b[u] >= 0) atomicAdd(p.ref_counts + b[u], held);
    }
    for (int c = 0; c < held; ++c) {
      int32_t* dst = p.block_tables + (long long)children[c] * p.max_blocks_per_seq;
#pragma unroll
      for (int u = 0; u < kTableUnroll; ++u)
        if (j0 + u * step < blocks) dst[j0 + u * step] = b[u];
    }
  }
}

// A cluster of blocks a row: every one reads the row's length before one of them writes it.
// Bound by the L2's atomics: 256 rows of 2K to 8K blocks (1.3 M atomics at places of no order)
// take 15 us, 20 with one block a row.  Without their results they took 12, but a count that is
// 0 already would go below it.
__global__ void __launch_bounds__(kTableThreads) release_kernel(const SequenceParams p) {
  const cg::cluster_group cluster = cg::this_cluster();
  const int row = blockIdx.x / cluster.num_blocks(), part = cluster.block_rank();
  previous_done();
  const int len = p.seq_lens[row];
  const int keep = p.keep_lens ? p.keep_lens[row] : 0;
  cluster.sync();
  if (!length_ok(p, len) || keep < 0) {
    if (part == 0 && threadIdx.x == 0) flag_error(p.err, PA_ERRFLAG_SEQ_LEN);
    return;
  }
  if (keep >= len) return;
  if (part == 0 && threadIdx.x == 0) p.seq_lens[row] = keep;
  const int32_t* table = p.block_tables + (long long)row * p.max_blocks_per_seq;
  const int last = blocks_of(len, p.block_size), step = cluster.num_blocks() * kTableThreads;
  for (int j0 = blocks_of(keep, p.block_size) + part * kTableThreads + threadIdx.x; j0 < last;
       j0 += kTableUnroll * step) {
    int b[kTableUnroll], held[kTableUnroll];
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) b[u] = j0 + u * step < last ? table[j0 + u * step] : -1;
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) {
      held[u] = 1;
      if (b[u] >= p.num_blocks) flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
      else if (b[u] >= 0) held[u] = atomicSub(p.ref_counts + b[u], 1);
    }
#pragma unroll
    for (int u = 0; u < kTableUnroll; ++u) {
      if (held[u] > 0) continue;  // else held by no row: put it back
      atomicAdd(p.ref_counts + b[u], 1);
      flag_error(p.err, PA_ERRFLAG_REF_COUNT);
    }
  }
}

// ---------------------------------------------------------------- append

constexpr int kAppendThreads = 1024;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendParts = 8;
static_assert(kAppendThreads * kAppendParts == PA_MAX_APPEND_SEQS, "one row a thread");
constexpr int kScan = 8;                                // 32-block groups of the pool that a warp looks at at once
constexpr int kLook = kAppendWarps * 32 * kScan;        // blocks that all warps look at at once
constexpr int kFewBlocks = 2;                           // new blocks of a row that its thread writes alone
constexpr int kInline = 8;                              // new tokens of a row whose slots its thread writes itself

// Bits of the 32 blocks from b0 + 32 u on that are free (count 0) and below `end`.
__device__ __forceinline__ void free_masks(const int32_t* refs, int b0, int end, unsigned (&masks)[kScan]) {
  const int lane = threadIdx.x % 32;
  int r[kScan];
#pragma unroll
  for (int u = 0; u < kScan; ++u) r[u] = b0 + u * 32 + lane < end ? refs[b0 + u * 32 + lane] : 1;
#pragma unroll
  for (int u = 0; u < kScan; ++u) masks[u] = __ballot_sync(~0u, r[u] == 0);
}

// Exclusive prefix sum over the block of v, which every lane of a warp gives as its warp's
// (kWarp) or each thread as its own; `total` is the block's sum.
template <bool kWarp>
__device__ __forceinline__ int block_prefix(int v, int* sums, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int upto = v;
  if constexpr (!kWarp) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += up;
    }
  }
  __syncthreads();  // sums may still be read
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int before = lane < warp ? sums[lane] : 0;
  total = sums[lane];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(~0u, before, o);
    total += __shfl_xor_sync(~0u, total, o);
  }
  return before + upto - v;
}

struct __align__(16) AppendShared {
  int tails[kAppendThreads];  // block that a row would write into and shares, else -1
  int sums[kAppendWarps];
  unsigned flags;             // errors, and the two below
  int needed;                 // blocks of this part's rows
  int enough;                 // part 0: whether the pool has what all parts need
};
constexpr unsigned kSharedTail = 1u << 30, kLargeRow = 1u << 31;

// One row a thread: one block up to kAppendThreads rows, a cluster of them above.  What a row
// needs stays in its thread's registers.  The first block's warps look through the pool from
// its lowest block on, until as many free ones are found as all rows need.  All of it is
// latency, some six dependent trips to memory (256 rows that share tails, a pool of 17,000
// blocks with free ones all over it: 7.7 us), as long as the pool's first kLook blocks have
// enough free ones.  Each kLook blocks more that are looked through are one more trip behind
// the others, about 1.1 us: 256 rows of one new block each, with their release, take 5.7 us
// where every second block is free, whatever the pool's size, but 6.8, 23 and 142 us where only
// the last twentieth of 16,384, 131,072 and 1,048,576 blocks is.  Above kAppendThreads rows:
// 2,048 take 13 us, 8,192 20 us.  Where a row grows by more than kInline tokens, these blocks
// alone write every slot behind a search for its row: a prompt of 131,072 tokens takes 73 us, 16
// chunks of 512 among 128 decodes 14.
template <bool kCluster>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const SequenceParams p) {
  __shared__ AppendShared sh;
  __shared__ __align__(16) int other[kCluster ? kAppendThreads : 4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int parts = kCluster ? gridDim.x : 1, part = kCluster ? blockIdx.x : 0;
  auto meet = [&]() {
    if constexpr (kCluster) cg::this_cluster().sync();
    else __syncthreads();
  };
  auto part_of = [&](int r) -> AppendShared* {
    if constexpr (kCluster) return cg::this_cluster().map_shared_rank(&sh, r);
    else return &sh;
  };
  const int n = p.num_rows, i = part * kAppendThreads + threadIdx.x;
  const unsigned bs = p.block_size;
  const bool mine = i < n;
  int len = 0, start = 0, stop = 0;
  previous_done();
  if (mine) {
    len = p.seq_lens[i];
    start = p.query_start_loc[i];
    stop = p.query_start_loc[i + 1];
  }
  unsigned masks[kScan];  // the pool's first kLook blocks, on their way with the rows
  if (part == 0) free_masks(p.ref_counts, warp * 32 * kScan, p.num_blocks, masks);
  if (threadIdx.x == 0) sh.flags = 0;
  __syncthreads();

  // the row: its last block if that is partly filled, who holds it, and the blocks it grows by
  unsigned flags = 0;
  const long long add = (long long)stop - start;
  int last = -1, held = 0, grows = 0, grown = 0, offset = 0;
  if (mine) {
    if ((i == 0 && start != 0) || (i == n - 1 && stop != p.total_tokens) || add < 0) {
      flags = PA_ERRFLAG_QUERY;
    } else if (!length_ok(p, len) || len + add > (long long)p.max_blocks_per_seq * p.block_size ||
               len + add > 0x7fffffff) {
      flags = PA_ERRFLAG_SEQ_LEN;
    } else if (add > 0) {
      grown = blocks_of(len, bs);
      grows = blocks_of(static_cast<int>(len + add), bs) - grown;
      offset = static_cast<int>(static_cast<unsigned>(len) % bs);
      if (offset) {
        last = p.block_tables[(long long)i * p.max_blocks_per_seq + grown - 1];
        if (last < 0 || last >= p.num_blocks) {
          flags = PA_ERRFLAG_BLOCK_TABLE;
        } else {
          held = p.ref_counts[last];
          if (held < 1) flags = PA_ERRFLAG_REF_COUNT;
        }
      }
    }
    if (flags) flag_error(p.err, flags);
    if (held > 1) flags |= kSharedTail;
    if (add > kInline) flags |= kLargeRow;
  }
  flags = __reduce_or_sync(~0u, flags);
  if (flags && lane == 0) atomicOr(&sh.flags, flags);
  sh.tails[threadIdx.x] = held > 1 ? last : -1;
  meet();

  unsigned all_flags = 0;
  for (int r = 0; r < parts; ++r) all_flags |= part_of(r)->flags;
  bool refused = (all_flags & ~(kSharedTail | kLargeRow)) != 0;
  // A shared tail is copied by every row that writes it but, where these are all of its
  // holders, the last: by those with fewer rows before them than the others that hold it.
  bool copies = false;
  if (all_flags & kSharedTail) {
    int lower = 0;
    for (int r = 0; r <= part; ++r) {
      const int* tails = sh.tails;
      if constexpr (kCluster) {
        __syncthreads();
        other[threadIdx.x] = part_of(r)->tails[threadIdx.x];
        __syncthreads();
        tails = other;
      }
      const int until = r < part ? kAppendThreads : static_cast<int>(threadIdx.x);
      if (held > 1) {
        int j = 0;
        for (; j + 4 <= until; j += 4) {
          const int4 t = *reinterpret_cast<const int4*>(tails + j);
          lower += (t.x == last) + (t.y == last) + (t.z == last) + (t.w == last);
        }
        for (; j < until; ++j) lower += tails[j] == last;
      }
    }
    copies = held > 1 && lower < held - 1;
  }
  // where the row's blocks start among all that are given out
  int needed;
  int at = block_prefix<false>(refused ? 0 : grows + (copies ? 1 : 0), sh.sums, needed);
  if constexpr (kCluster) {
    if (threadIdx.x == 0) sh.needed = needed;
    meet();
    needed = 0;
    for (int r = 0; r < parts; ++r) {
      const int theirs = part_of(r)->needed;
      if (r < part) at += theirs;
      needed += theirs;
    }
  }
  // the free blocks by ascending number, as many as are needed
  int32_t* fresh = p.ws_fresh;
  if (part == 0) {
    int found = 0;
    for (int look = 0; !refused && found < needed && look < p.num_blocks; look += kLook) {
      const int b0 = look + warp * 32 * kScan;
      if (look > 0) free_masks(p.ref_counts, b0, p.num_blocks, masks);
      int count = 0, sum;
#pragma unroll
      for (int u = 0; u < kScan; ++u) count += __popc(masks[u]);
      int place = found + block_prefix<true>(count, sh.sums, sum);
#pragma unroll
      for (int u = 0; u < kScan; ++u) {
        const int to = place + __popc(masks[u] & ((1u << lane) - 1));
        if ((masks[u] >> lane & 1) && to < needed) fresh[to] = b0 + u * 32 + lane;
        place += __popc(masks[u]);
      }
      found += sum;
    }
    if (threadIdx.x == 0) sh.enough = found >= needed;
  }
  meet();
  if (!refused && !part_of(0)->enough) {
    if (i == 0) flag_error(p.err, PA_ERRFLAG_POOL);
    refused = true;
  }

  int32_t* table = p.block_tables + (long long)i * p.max_blocks_per_seq;
  if (mine) {
    long long src = 0, dst = 0;
    if (!refused) {
      if (copies) {
        src = last;
        last = fresh[at++];
        dst = last;
        table[grown - 1] = last;
        atomicSub(p.ref_counts + src, 1);
        p.ref_counts[last] = 1;
      }
      if (!(all_flags & kLargeRow)) {  // the slots: the last block's rest, then the new blocks
        unsigned slot_at = offset;
        int block = last, next = at;
        for (int t = start; t < stop; ++t, ++slot_at) {
          if (slot_at == bs || (t == start && offset == 0)) {
            block = fresh[next++];
            slot_at = 0;
          }
          p.slot_mapping[t] = (long long)block * bs + slot_at;
        }
      }
      p.seq_lens[i] = stop - start + len;
    }
    p.block_mapping[2 * (long long)i] = src;
    p.block_mapping[2 * (long long)i + 1] = dst;
  }
  // the new blocks into the tables: a thread its own, a warp together those of a long prompt
  if (refused) grows = 0;
  if (grows <= kFewBlocks)
    for (int k = 0; k < grows; ++k) {
      const int block = fresh[at + k];
      table[grown + k] = block;
      p.ref_counts[block] = 1;
    }
  for (unsigned left = __ballot_sync(~0u, grows > kFewBlocks); left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    const int many = __shfl_sync(~0u, grows, from), first = __shfl_sync(~0u, at, from);
    int32_t* to = p.block_tables + (long long)__shfl_sync(~0u, i, from) * p.max_blocks_per_seq +
                  __shfl_sync(~0u, grown, from);
#pragma unroll 4
    for (int k = lane; k < many; k += 32) {
      const int block = fresh[first + k];
      to[k] = block;
      p.ref_counts[block] = 1;
    }
  }
  meet();  // a part's shared memory is read until here, the tables below
  if (!(all_flags & kLargeRow) && !refused) return;

  for (int t = i; t < p.total_tokens; t += parts * kAppendThreads) {
    long long slot = -1;
    if (!refused) {
      int row = 0, past = n;  // first row with query_start_loc[row + 1] > t
      while (row < past) {
        const int mid = (row + past) / 2;
        if (p.query_start_loc[mid + 1] <= t) row = mid + 1;
        else past = mid;
      }
      const unsigned pos = p.seq_lens[row] - (p.query_start_loc[row + 1] - t);  // the lengths count the new tokens
      slot = (long long)p.block_tables[(long long)row * p.max_blocks_per_seq + pos / bs] * bs + pos % bs;
    }
    p.slot_mapping[t] = slot;
  }
}

}  // namespace

cudaError_t launch_fork_blocks(const SequenceParams& p, cudaStream_t stream) {
  const int slices = (p.max_blocks_per_seq + 4 * kTableThreads - 1) / (4 * kTableThreads);
  const int rows = p.num_rows, y = slices < 1024 ? slices : 1024;
  // By parents where at least two children on average share a parent and the rows are long, else
  // the look for a parent's children costs more than its atomics (by parents against by
  // children: 128 parents and 1,024 children of 131,072 tokens 8.3 against 13.4 us, one parent
  // 7.6 against 36; of 1,024 tokens in tables of 64 blocks 3.5 against 2.5, and 1,024 parents
  // of 131,072 tokens with as many children 19 against 14).  Lengths are on the device, so the
  // tables' width stands for them: 128 parents and 1,024 children of 1,024 tokens take 2.6 us in
  // tables of 64 blocks, 3.3 in tables of 8,192.
  if (p.num_parents > 0 && rows / 2 >= p.num_parents && rows <= kForkMost &&
      (long long)rows * p.max_blocks_per_seq >= 1 << 19) {
    // parts of the children until the grid fills the device, of eight for each parent or more
    const long long blocks = (long long)p.num_parents * y;
    const int least = (rows + kForkPart - 1) / kForkPart, most = rows / 8 / p.num_parents;
    const int fill = static_cast<int>(152 * 8 / blocks);
    SequenceParams q = p;
    const int parts = std::max(least, std::min(fill, most));
    q.fork_part = (rows + parts - 1) / parts;
    return launch_early(fork_parents_kernel, dim3(p.num_parents, y, parts), kTableThreads, 0, 1, q, stream);
  }
  return launch_early(fork_kernel, dim3(rows, y), kTableThreads, 0, 1, p, stream);
}

cudaError_t launch_release_blocks(const SequenceParams& p, cudaStream_t stream) {
  // blocks a row: enough for the longest row its table has room for, at kTableUnroll entries a
  // thread.  Rows far shorter than that pay for blocks with nothing to do: 1,024 rows of 1,024
  // tokens take 3 us in tables of 64 blocks and 13.5 in tables of 8,192.
  int cluster = 1;
  while (cluster < 8 && p.num_rows < (1 << 27) && cluster * kTableThreads * kTableUnroll < p.max_blocks_per_seq) cluster *= 2;
  return launch_early(release_kernel, dim3(p.num_rows * cluster), kTableThreads, 0, cluster, p, stream);
}

cudaError_t launch_append_blocks(const SequenceParams& p, cudaStream_t stream) {
  // one block where it has a thread for every row: a cluster of one takes 3 us longer
  if (p.num_rows <= kAppendThreads) return launch_early(append_kernel<false>, dim3(1), kAppendThreads, 0, 1, p, stream);
  const int parts = (p.num_rows + kAppendThreads - 1) / kAppendThreads;
  return launch_early(append_kernel<true>, dim3(parts), kAppendThreads, 0, parts, p, stream);
}

}  // namespace pa
