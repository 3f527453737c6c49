// Differential attention without matrix instructions, and the joining of partial states:
//  * diff_generic_kernel -- one CTA per (query row, head, partition), fp32 throughout: fp32 caches,
//    NVFP4 caches and every shape that the tensor-core kernels do not take;
//  * diff_merge_kernel -- a row's partial states of both maps -> their difference, norm and output.
#include "diff.cuh"
#include "kv_rows.cuh"
#include "launch.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Warps of a generic CTA: 256 keys in one or two rounds of them (N pairs of output elements a lane).
template <int N>
constexpr int generic_warps() { return N <= 4 ? 16 : 8; }

struct DiffGenericArgs {
  DiffParams p;
  int only_multi_token;  // -1: every row; 0, 1: of single-token requests, of the others
};

// Element pairs of cached rows.
template <int KVDT>
__device__ __forceinline__ float2 kv_pair(const KvRow& r, int e) {
  if constexpr (KVDT == PA_F32) {
    return *reinterpret_cast<const float2*>(r.row + 4 * e);
  } else if constexpr (KVDT == PA_F16 || KVDT == PA_BF16) {
    return unpack2<KVDT>(*reinterpret_cast<const uint32_t*>(r.row + 2 * e));
  } else {
    return make_float2(kv_elem<KVDT>(r, e), kv_elem<KVDT>(r, e + 1));
  }
}

// One CTA a (query row, head, partition); its warps deal the keys out in groups of kKeys.  Of a
// group, eight lanes share a key's dot products, four keys at once; then lane i adds elements
// 64 k + 2 i and the next of the value rows, which were fetched before the scores were known, to both
// maps' sums.  The warps' states meet in shared memory, so that a context of one partition (256 tokens
// at least) takes one launch.
//
// Latency is what bounds the calls that come here (table, rows, two sums over the warp, the meeting):
// loads are in flight together, 64 registers of values a lane.  4 fp32 sequences of 17 to 200 tokens:
// 8.9 us (11.9 with eight warps, two rounds of keys), where a warp a head that took the keys one after
// the other in partitions of 64, and a second launch to join them, took 61.
template <int QDT, int KVDT, int N>
__global__ void __launch_bounds__(32 * generic_warps<N>()) diff_generic_kernel(const DiffGenericArgs args) {
  using QE = Elem<QDT>;
  constexpr int kKeys = 32 / N, kWarps = generic_warps<N>();
  const DiffParams& p = args.p;
  const AttnParams& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.num_q_heads / 2, d = a.head_size, width = 2 * d;
  const int head = blockIdx.y, row = blockIdx.x, z = blockIdx.z;
  previous_done();
  if (plan_rejected(a)) return;
  const RowInfo ri = row_info(a, row);
  if (!diff_row_ok(a, ri)) {
    if (z == 0 && ri.q_len == 1) {  // as the tiles, which no such request of several tokens has
      typename QE::T* out = static_cast<typename QE::T*>(a.out) + ((long long)row * heads + head) * width;
      for (int i = threadIdx.x; i < width; i += 32 * kWarps) out[i] = QE::from_float(0.f);
      if (threadIdx.x == 0 && a.query_start_loc == nullptr) flag_error(a.err, PA_ERRFLAG_SEQ_LEN);
    }
    return;
  }
  if (a.query_start_loc != nullptr && args.only_multi_token >= 0 && (ri.q_len > 1) != (args.only_multi_token != 0)) return;
  if (z >= ri.parts_row) return;

  const int kvh = head / a.group * 2;
  const int t0 = max(ri.origin + z * ri.part, ri.lo), t1 = min(ri.origin + (z + 1) * ri.part, ri.kv_len);
  __shared__ __align__(16) float sq[2][64 * N];            // read four at a time
  __shared__ __align__(16) float red[kWarps][2][64 * N];   // two
  __shared__ float2 red_ml[kWarps][2];
  const typename QE::T* qrow = static_cast<const typename QE::T*>(a.q) + ((long long)row * a.num_q_heads + 2 * head) * d;
  for (int i = threadIdx.x; i < width; i += 32 * kWarps) sq[i >= d][i >= d ? i - d : i] = QE::load(qrow + i);
  __syncthreads();
  const float lam = diff_lambda(p, row, head);  // on its way before it is needed
  float c[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    c[j] = a.scale * kLog2e * (is_scaled<KVDT>() ? a.k_scale[(kvh + j) * a.scale_stride] : 1.f);

  const int32_t* table = a.block_tables + (long long)ri.request * a.max_blocks_per_seq;
  const bool even = d % 2 == 0, quads = KVDT == PA_F32 && d % 4 == 0;
  const int sub = lane & 7;  // this lane's place among the eight of a key
  float2 acc[2][N];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < N; ++k) acc[0][k] = acc[1][k] = make_float2(0.f, 0.f);
  for (int tb = t0 + warp * kKeys; tb < t1; tb += kWarps * kKeys) {
    // lane i of the first kKeys holds where key tb + i lies
    const int mine = tb + lane;
    long long my_tile = -1;
    int my_off = 0;
    if (lane < kKeys && mine < t1) {
      const int phys = table[mine / a.block_size];
      my_off = mine % a.block_size;
      if (phys < 0 || phys >= a.num_blocks) flag_error(a.err, PA_ERRFLAG_BLOCK_TABLE);
      else my_tile = (long long)phys * a.num_kv_heads + kvh;
    }
    // scores: s[j] of key tb + lane ends up in lane (of the first kKeys)
    float s[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int k0 = 0; k0 < kKeys; k0 += 4) {
      const int key = k0 + (lane >> 3);
      const long long tile = __shfl_sync(0xffffffffu, my_tile, key);
      const int off = __shfl_sync(0xffffffffu, my_off, key);
      float dot[2] = {0.f, 0.f};
      if (tile >= 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const KvRow kr = kv_row<KVDT>(a.k_cache, tile + j, a.block_size, d, off);
          if (quads) {
#pragma unroll
            for (int e = 0; e < 64 * N / 2; e += 32) {
              if (e + 4 * sub < d) {
                const float4 x = *reinterpret_cast<const float4*>(kr.row + 4 * (e + 4 * sub));
                const float4 y = *reinterpret_cast<const float4*>(&sq[j][e + 4 * sub]);
                dot[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot[j]))));
              }
            }
          } else if (even) {
#pragma unroll 4
            for (int e = 2 * sub; e < d; e += 16) {
              const float2 x = kv_pair<KVDT>(kr, e);
              dot[j] = fmaf(x.x, sq[j][e], fmaf(x.y, sq[j][e + 1], dot[j]));
            }
          } else {
            for (int e = sub; e < d; e += 8) dot[j] = fmaf(kv_elem<KVDT>(kr, e), sq[j][e], dot[j]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float x = warp_sum_xor(dot[j], 1, 4);
        const float got = __shfl_sync(0xffffffffu, x, (lane & 3) * 8);  // of key k0 + lane % 4
        if ((lane & ~3) == k0 && my_tile >= 0) s[j] = got * c[j];
      }
    }
    // the values, before the weights are known
    float2 v[kKeys][N];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const long long tile = __shfl_sync(0xffffffffu, my_tile, i);
      const int off = __shfl_sync(0xffffffffu, my_off, i);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int e = 64 * k + 2 * lane;
        v[i][k] = make_float2(0.f, 0.f);
        if (tile >= 0 && e < width) {
          if (even) {
            v[i][k] = kv_pair<KVDT>(kv_row<KVDT>(a.v_cache, tile + (e >= d), a.block_size, d, off), e >= d ? e - d : e);
          } else {  // a pair may lie in both halves
            const KvRow r0 = kv_row<KVDT>(a.v_cache, tile, a.block_size, d, off);
            const KvRow r1 = kv_row<KVDT>(a.v_cache, tile + 1, a.block_size, d, off);
            v[i][k].x = e < d ? kv_elem<KVDT>(r0, e) : kv_elem<KVDT>(r1, e - d);
            v[i][k].y = e + 1 < d ? kv_elem<KVDT>(r0, e + 1) : kv_elem<KVDT>(r1, e + 1 - d);
          }
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
      for (int k = 0; k < N; ++k) {
        acc[j][k].x *= alpha;
        acc[j][k].y *= alpha;
      }
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = __shfl_sync(0xffffffffu, w[j], i);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          acc[j][k].x = fmaf(f, v[i][k].x, acc[j][k].x);
          acc[j][k].y = fmaf(f, v[i][k].y, acc[j][k].y);
        }
      }
    }
  }
  // ---- the warps' states; the first warp joins them
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int k = 0; k < N; ++k) *reinterpret_cast<float2*>(&red[warp][j][64 * k + 2 * lane]) = acc[j][k];
    if (lane == 0) red_ml[warp][j] = make_float2(m[j], l[j]);
  }
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
    for (int v = 0; v < kWarps; ++v) combine_ml(m[j], l[j], red_ml[v][j].x, red_ml[v][j].y);
#pragma unroll
    for (int k = 0; k < N; ++k) acc[j][k] = make_float2(0.f, 0.f);
    for (int v = 0; v < kWarps; ++v) {
      const float2 ml = red_ml[v][j];
      const float f = ml.y > 0.f ? exp2f(ml.x - m[j]) : 0.f;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float2 x = *reinterpret_cast<const float2*>(&red[v][j][64 * k + 2 * lane]);
        acc[j][k].x = fmaf(x.x, f, acc[j][k].x);
        acc[j][k].y = fmaf(x.y, f, acc[j][k].y);
      }
    }
    if constexpr (is_scaled<KVDT>()) {
      const float vs[2] = {a.v_scale[kvh * a.scale_stride], a.v_scale[(kvh + 1) * a.scale_stride]};
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int e = 64 * k + 2 * lane;
        acc[j][k].x *= vs[e >= d];
        acc[j][k].y *= vs[e + 1 >= d];
      }
    }
  }
  if (ri.parts_row == 1) {
    const float w0 = diff_weight(l[0]), w1 = diff_weight(l[1]) * lam;
#pragma unroll
    for (int k = 0; k < N; ++k) {
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
      for (int k = 0; k < N; ++k) {
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
  if (a.query_start_loc && !a.plan_ok && (a.query_start_loc[0] != 0 || a.query_start_loc[1] != a.num_rows)) return;
  int row = static_cast<int>(item / heads);
  const int head = static_cast<int>(item % heads);
  if (args.single && a.query_start_loc) {
    const int q0 = a.query_start_loc[row];
    if (a.query_start_loc[row + 1] - q0 != 1) return;
    row = q0;
  }
  const RowInfo ri = row_info(a, row);
  if (!diff_row_ok(a, ri) || (ri.q_len > 1) == (args.single != 0)) return;
  const int np = ri.parts_row;
  if (np <= 1) return;  // written by the attention kernel
  const long long base = row_partial_base(a, ri, row);
  const int hq = a.num_q_heads;
  const float2* ml = a.ws_ml + base * hq + 2 * head;
  const float lam = diff_lambda(p, row, head);
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
  const float f0 = diff_weight(l[0]), f1 = -diff_weight(l[1]) * lam;
  float2 o[N];
#pragma unroll
  for (int k = 0; k < N; ++k) o[k] = make_float2(0.f, 0.f);
  const float* acc = a.ws_acc + (base * hq + 2 * head) * width;
  constexpr int kAhead = N == 8 ? 2 : 4;  // partitions whose loads are on their way together
  for (int z0 = part; z0 < np; z0 += kAhead * kWarps) {
    float2 x[kAhead][2][N];
    float w[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
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
    for (int u = 0; u < kAhead; ++u)
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
  DiffGenericArgs args;
  args.p = p;
  args.only_multi_token = only_multi;
  const dim3 grid(p.a.num_rows, p.a.num_q_heads / 2, grid_z);
  if (p.a.head_size <= 64)
    return launch_early<DiffGenericArgs>(diff_generic_kernel<QDT, KVDT, 2>, grid, 32 * generic_warps<2>(), 0, 1, args, s);
  if (p.a.head_size <= 128)
    return launch_early<DiffGenericArgs>(diff_generic_kernel<QDT, KVDT, 4>, grid, 32 * generic_warps<4>(), 0, 1, args, s);
  return launch_early<DiffGenericArgs>(diff_generic_kernel<QDT, KVDT, 8>, grid, 32 * generic_warps<8>(), 0, 1, args, s);
}

// Single-token rows may have many partitions: eight warps a head then.  Rows of chunks have few, and
// there are many of them (8,192 tokens of 16 heads with eight warps each: 234 us to find nothing to do).
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
