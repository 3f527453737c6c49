// Differential attention without matrix instructions, and the joining of partial states:
//  * diff_generic_kernel -- one warp per (query row, head, partition), fp32 throughout: fp32 caches,
//    NVFP4 caches and every shape that the tensor-core kernels do not take;
//  * diff_merge_kernel -- a row's partial states of both maps -> their difference, norm and output.
#include "diff.cuh"
#include "kv_rows.cuh"
#include "launch.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// 32 keys at a time: lane j scores key j under both maps, then every lane adds the 32 value rows,
// elements 64 k + 2 lane and the next of each, into both maps' sums: a value row is read once.
template <int QDT, int KVDT>
__global__ void __launch_bounds__(128) diff_generic_kernel(const DiffParams p, int only_multi_token) {
  using QE = Elem<QDT>;
  const AttnParams& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.num_q_heads / 2, d = a.head_size, width = 2 * d;
  const int head = blockIdx.y * 4 + warp;
  const int row = blockIdx.x, z = blockIdx.z;
  if (head >= heads || plan_rejected(a)) return;
  const RowInfo ri = row_info(a, row);
  float2 acc[2][kDiffPairs];
#pragma unroll
  for (int k = 0; k < kDiffPairs; ++k) acc[0][k] = acc[1][k] = make_float2(0.f, 0.f);
  if (!ri.ok) {
    if (z == 0) {
      typename QE::T* out = static_cast<typename QE::T*>(a.out) + ((long long)row * heads + head) * width;
      for (int i = lane; i < width; i += 32) out[i] = QE::from_float(0.f);
      if (lane == 0 && a.query_start_loc == nullptr) flag_error(a.err, PA_ERRFLAG_SEQ_LEN);
    }
    return;
  }
  if (a.query_start_loc != nullptr && only_multi_token >= 0 && (ri.q_len > 1) != (only_multi_token != 0)) return;
  if (z >= ri.parts_row) return;

  const int kvh = head / a.group * 2;
  const int t0 = ri.origin + z * ri.part, t1 = min(t0 + ri.part, ri.kv_len);
  float c[2], vscale[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    c[j] = a.scale * kLog2e;
    vscale[j] = 1.f;
    if (is_scaled<KVDT>()) {
      c[j] *= a.k_scale[(kvh + j) * a.scale_stride];
      vscale[j] = a.v_scale[(kvh + j) * a.scale_stride];
    }
  }
  __shared__ float sq[4][2][kDiffMaxHead];
  const typename QE::T* qrow =
      static_cast<const typename QE::T*>(a.q) + ((long long)row * a.num_q_heads + 2 * head) * d;
  for (int i = lane; i < width; i += 32) sq[warp][i / d][i % d] = QE::load(qrow + i);
  __syncwarp();

  const int32_t* table = a.block_tables + (long long)ri.request * a.max_blocks_per_seq;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int tb = max(t0, ri.lo); tb < t1; tb += 32) {
    const int tt = tb + lane, off = tt % a.block_size;
    long long tile = -1;
    float s[2] = {-INFINITY, -INFINITY};
    if (tt < t1) {
      const int phys = table[tt / a.block_size];
      if (phys < 0 || phys >= a.num_blocks) {
        flag_error(a.err, PA_ERRFLAG_BLOCK_TABLE);
      } else {
        tile = (long long)phys * a.num_kv_heads + kvh;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const KvRow kr = kv_row<KVDT>(a.k_cache, tile + j, a.block_size, d, off);
          const float* q = sq[warp][j];
          float dot[4] = {0.f, 0.f, 0.f, 0.f};
          int dd = 0;
          for (; dd + 32 <= d; dd += 32) {
            float kv[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) kv[e] = kv_elem<KVDT>(kr, dd + e);
#pragma unroll
            for (int e = 0; e < 32; ++e) dot[e & 3] = fmaf(q[dd + e], kv[e], dot[e & 3]);
          }
          for (; dd < d; ++dd) dot[0] = fmaf(q[dd], kv_elem<KVDT>(kr, dd), dot[0]);
          s[j] = ((dot[0] + dot[1]) + (dot[2] + dot[3])) * c[j];
        }
      }
    }
    float w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float top = fmaxf(m[j], warp_max_xor(s[j], 1, 16));
      const float u = top == -INFINITY ? 0.f : top;
      const float alpha = exp2f(m[j] - u);  // 0 before the first key
      w[j] = exp2f(s[j] - u);
      l[j] = l[j] * alpha + warp_sum_xor(w[j], 1, 16);
      m[j] = top;
#pragma unroll
      for (int k = 0; k < kDiffPairs; ++k) {
        acc[j][k].x *= alpha;
        acc[j][k].y *= alpha;
      }
    }
    const int n = min(32, t1 - tb);
    const long long place = tile < 0 ? -1 : tile * a.block_size + off;  // of the first half's row
    for (int i = 0; i < n; ++i) {
      const float w0 = __shfl_sync(0xffffffffu, w[0], i), w1 = __shfl_sync(0xffffffffu, w[1], i);
      const long long at = __shfl_sync(0xffffffffu, place, i);
      if (at < 0) continue;  // an unreadable block, flagged above
      const long long vt = at / a.block_size;
      const int vo = static_cast<int>(at - vt * a.block_size);
      const KvRow r0 = kv_row<KVDT>(a.v_cache, vt, a.block_size, d, vo);
      const KvRow r1 = kv_row<KVDT>(a.v_cache, vt + 1, a.block_size, d, vo);
#pragma unroll
      for (int k = 0; k < kDiffPairs; ++k) {
        const int e = 64 * k + 2 * lane;
        if (e < width) {  // d is no multiple of 2 everywhere: each element by itself
          const float x = e < d ? kv_elem<KVDT>(r0, e) : kv_elem<KVDT>(r1, e - d);
          const float y = e + 1 < d ? kv_elem<KVDT>(r0, e + 1) : kv_elem<KVDT>(r1, e + 1 - d);
          acc[0][k].x = fmaf(w0, x, acc[0][k].x);
          acc[0][k].y = fmaf(w0, y, acc[0][k].y);
          acc[1][k].x = fmaf(w1, x, acc[1][k].x);
          acc[1][k].y = fmaf(w1, y, acc[1][k].y);
        }
      }
    }
  }
  if constexpr (is_scaled<KVDT>()) {
#pragma unroll
    for (int k = 0; k < kDiffPairs; ++k) {
      const int e = 64 * k + 2 * lane;
      const float x = vscale[e >= d], y = vscale[e + 1 >= d];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[j][k].x *= x;
        acc[j][k].y *= y;
      }
    }
  }
  if (ri.parts_row == 1) {
    const float w0 = diff_weight(l[0]), w1 = diff_weight(l[1]) * diff_lambda(p, row, head);
#pragma unroll
    for (int k = 0; k < kDiffPairs; ++k) {
      acc[0][k].x = acc[0][k].x * w0 - acc[1][k].x * w1;
      acc[0][k].y = acc[0][k].y * w0 - acc[1][k].y * w1;
    }
    diff_finish<QDT>(p, row, head, width, acc[0]);
  } else {
    const long long pi = row_partial_base(a, ri, row) + z;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* wa = a.ws_acc + (pi * a.num_q_heads + 2 * head + j) * width;
#pragma unroll
      for (int k = 0; k < kDiffPairs; ++k) {
        const int e = 64 * k + 2 * lane;
        if (e < width) *reinterpret_cast<float2*>(wa + e) = acc[j][k];
      }
      if (lane == 0) a.ws_ml[pi * a.num_q_heads + 2 * head + j] = make_float2(m[j], l[j]);
    }
  }
}

struct DiffMergeArgs {
  DiffParams p;
  int single;  // of a flattened batch: the single-token rows, an item a request; else the others, an item a row
};

// Rows with partial states: kWarps warps a head share its partitions.  Lane i sums elements
// 64 k + 2 i and the next of both maps, every partition weighted by 2^(m_j - M) of its map.
template <int QDT, int kWarps, int N>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps) diff_merge_kernel(const DiffMergeArgs args) {
  const DiffParams& p = args.p;
  const AttnParams& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.num_q_heads / 2, width = 2 * a.head_size;
  const long long item = kWarps == 1 ? (long long)blockIdx.x * 4 + warp : blockIdx.x;
  const int part = kWarps == 1 ? 0 : warp;  // this warp's place among its head's
  previous_done();
  if (item >= (long long)(args.single ? a.num_seqs : a.num_rows) * heads || plan_rejected(a)) return;
  int row = static_cast<int>(item / heads);
  const int head = static_cast<int>(item % heads);
  if (args.single && a.query_start_loc) {
    const int q0 = a.query_start_loc[row];
    if (a.query_start_loc[row + 1] - q0 != 1) return;
    row = q0;
  }
  const RowInfo ri = row_info(a, row);
  if (!ri.ok || (ri.q_len > 1) == (args.single != 0)) return;
  const int np = ri.parts_row;
  if (np <= 1) return;  // written by the attention kernel
  const long long base = row_partial_base(a, ri, row);
  const int hq = a.num_q_heads;
  const float2* ml = a.ws_ml + base * hq + 2 * head;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int z = lane; z < np; z += 32) {
    const float4 v = *reinterpret_cast<const float4*>(ml + (long long)z * hq);
    combine_ml(m[0], l[0], v.x, v.y);
    combine_ml(m[1], l[1], v.z, v.w);
  }
  for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[j], o), l2 = __shfl_xor_sync(0xffffffffu, l[j], o);
      combine_ml(m[j], l[j], m2, l2);
    }
  }
  // weights of the difference: 1 / l1 and -lambda / l2
  const float f0 = diff_weight(l[0]), f1 = -diff_weight(l[1]) * diff_lambda(p, row, head);
  float2 o[N];
#pragma unroll
  for (int k = 0; k < N; ++k) o[k] = make_float2(0.f, 0.f);
  const float* acc = a.ws_acc + (base * hq + 2 * head) * width;
  for (int z0 = part; z0 < np; z0 += 2 * kWarps) {
    float2 x[2][2][N];
    float w[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int z = z0 + u * kWarps;
      const bool in = z < np;
      const float4 v = in ? *reinterpret_cast<const float4*>(ml + (long long)z * hq)
                          : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      w[u][0] = v.y > 0.f ? f0 * exp2f(v.x - m[0]) : 0.f;
      w[u][1] = v.w > 0.f ? f1 * exp2f(v.z - m[1]) : 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int e = 64 * k + 2 * lane;
          x[u][j][k] = in && e < width
                           ? *reinterpret_cast<const float2*>(acc + ((long long)z * hq + j) * width + e)
                           : make_float2(0.f, 0.f);
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          o[k].x = fmaf(x[u][j][k].x, w[u][j], o[k].x);
          o[k].y = fmaf(x[u][j][k].y, w[u][j], o[k].y);
        }
  }
  if constexpr (kWarps > 1) {
    __shared__ float2 red[kWarps][N][32];
#pragma unroll
    for (int k = 0; k < N; ++k) red[warp][k][lane] = o[k];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      for (int v = 1; v < kWarps; ++v) {
        o[k].x += red[v][k][lane].x;
        o[k].y += red[v][k][lane].y;
      }
    }
  }
  diff_finish<QDT>(p, row, head, width, o);
}

template <int QDT, int KVDT>
cudaError_t launch_generic_t(const DiffParams& p, int grid_z, int only_multi, cudaStream_t s) {
  const dim3 grid(p.a.num_rows, (p.a.num_q_heads / 2 + 3) / 4, grid_z);
  diff_generic_kernel<QDT, KVDT><<<grid, 128, 0, s>>>(p, only_multi);
  return cudaGetLastError();
}

// Single-token rows may have many partitions: eight warps a head then.  Rows of chunks have few, and there are many of them.
template <int QDT, int N>
cudaError_t launch_merge_t(const DiffParams& p, int single, int partitions, cudaStream_t s) {
  DiffMergeArgs args;
  args.p = p;
  args.single = single;
  const long long items = (long long)(single ? p.a.num_seqs : p.a.num_rows) * (p.a.num_q_heads / 2);
  if (partitions > 16)
    return launch_early<DiffMergeArgs>(diff_merge_kernel<QDT, 8, N>, dim3(static_cast<unsigned>(items)), 256, 0, 1, args,
                                       s);
  return launch_early<DiffMergeArgs>(diff_merge_kernel<QDT, 1, N>, dim3(static_cast<unsigned>((items + 3) / 4)), 128, 0,
                                     1, args, s);
}

template <int QDT>
cudaError_t launch_merge_width(const DiffParams& p, int single, int partitions, cudaStream_t s) {
  if (p.a.head_size <= 64) return launch_merge_t<QDT, 2>(p, single, partitions, s);
  if (p.a.head_size <= 128) return launch_merge_t<QDT, 4>(p, single, partitions, s);
  return launch_merge_t<QDT, 8>(p, single, partitions, s);
}

}  // namespace

cudaError_t launch_diff_generic(const DiffParams& p, int q_dtype, int kv_dtype, int grid_z, int only_multi_token,
                                cudaStream_t stream) {
#define PA_DIFF(Q, KV) \
  if (q_dtype == Q && kv_dtype == KV) return launch_generic_t<Q, KV>(p, grid_z, only_multi_token, stream);
  PA_DIFF(PA_F32, PA_F32)
  PA_DIFF(PA_F16, PA_F16)
  PA_DIFF(PA_BF16, PA_BF16)
  PA_DIFF(PA_F32, PA_FP8_E4M3)
  PA_DIFF(PA_F16, PA_FP8_E4M3)
  PA_DIFF(PA_BF16, PA_FP8_E4M3)
  PA_DIFF(PA_F32, PA_FP8_E5M2)
  PA_DIFF(PA_F16, PA_FP8_E5M2)
  PA_DIFF(PA_BF16, PA_FP8_E5M2)
  PA_DIFF(PA_F32, PA_NVFP4)
  PA_DIFF(PA_F16, PA_NVFP4)
  PA_DIFF(PA_BF16, PA_NVFP4)
#undef PA_DIFF
  return cudaErrorInvalidValue;
}

cudaError_t launch_diff_merge(const DiffParams& p, int q_dtype, int single, int partitions, cudaStream_t stream) {
  if (q_dtype == PA_F32) return launch_merge_width<PA_F32>(p, single, partitions, stream);
  if (q_dtype == PA_F16) return launch_merge_width<PA_F16>(p, single, partitions, stream);
  if (q_dtype == PA_BF16) return launch_merge_width<PA_BF16>(p, single, partitions, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
