// Differential attention of single-token rows on tensor cores.
//
// One CTA handles (request, KV group, up to 4 or 8 of its heads, partition of the context); each
// of its warps takes every other unit of kTok tokens: the group's two key tiles and two value
// tiles, four TMA copies into a ring of the warp's own (layout [128-byte piece][token], 128-byte
// swizzle).  m16n8k16 products with the keys' tokens (then the values' dims) as the 16 rows:
//   S^T[token][col]   = K_j[token] . q_j       O^T[dim][col] += V^T[dim][token] P^T[token][col]
// Up to four heads: the columns are map 1's heads, then map 2's, of one tile.  Both key tiles are
// multiplied by all eight queries and the half that belongs together is kept, which costs no more
// products than one tile a map would, and the values, twice as wide as the keys, meet both maps'
// weights in one product each.  Up to eight heads: a tile of columns a map; every value fragment
// serves two products.  Either way each cached byte is read once for all heads.
//
// Bound by memory: the bytes of K and V.  What counts is bytes on their way: units of 16 KB, two a warp,
// two warps a CTA, three CTAs an SM (192 KB).  Measured on the card's 6.7 TB/s (copy): 64 rows of 512 to
// 4,096 tokens, 32/8 heads of 128 bf16, 102 us, 5.9 TB/s with the joining of the partitions; 3 rows of
// 98,304 to 131,072, 64/8 heads f16, 220 us, 6.4 TB/s; 256 rows of a 4,096-token window on an e4m3 cache
// 328 us, 6.3 TB/s.  16% of the issue slots, so the second product of each weight (see kSplit) takes
// nothing: 102.9 and 103.3 us without and with it.
#include "diff.cuh"
#include "launch.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 2;

struct DiffDecodeArgs {
  DiffParams p;
  int heads_cta;    // heads of a CTA: 4 or 8
  int head_groups;  // CTAs a KV group
  CUtensorMap tk, tv;
};

template <int QDT, int KVDT, int HEAD, int TOK, int NT>
struct Geom {
  static constexpr bool kFp8 = is_fp8<KVDT>();
  static constexpr int kRow = HEAD * (kFp8 ? 1 : 2);
  static constexpr int kTile = TOK * kRow;      // one head's unit of K or V
  static constexpr int kStage = 4 * kTile;      // K_1, K_2, V_1, V_2
  static constexpr int kStages = 2;
  // Weights meet V as two 16-bit numbers, the second what the first leaves out, so that they are good to
  // 2^-16 (bf16) or 2^-21 of themselves: memory bounds these rows, the second product is free.  The f16
  // weights of an FP8 cache are far finer than a bf16 output already.
  static constexpr bool kSplit = !(kFp8 && QDT == PA_BF16);
  static constexpr int kMTiles = TOK / 16, kSteps = HEAD / 16;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kRedRow = 2 * HEAD + 8;  // a state's row, off the banks of its neighbours
  static constexpr int kRed = kWarps * NT * 8 * (kRedRow + 2) * 4;
  static constexpr int kSmem = 1024 + (kRing > kRed ? kRing : kRed);
  static_assert(kRow % 128 == 0 && kTile % 1024 == 0, "pieces of whole swizzle patterns");
  static __device__ __forceinline__ uint32_t off(int tok, int chunk) {
    return static_cast<uint32_t>((chunk >> 3) * TOK * 128) + swz128(tok, chunk & 7);
  }
};

template <int HEAD, int NT>
struct State {
  float acc[NT][HEAD / 8][4];  // both value halves: 2 HEAD / 16 tiles of 16 dims
  float m[NT][2], l[NT][2];
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < HEAD / 8; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
  }
};

// The queries as B fragments and the score multipliers (log2 units) of this thread's columns.
// FP8 caches: q scaled by a power of two a head, so that f16 holds it (the multiplier takes it back).
template <int QDT, int KVDT, int HEAD, int NT>
__device__ __forceinline__ void load_queries(const DiffParams& p, long long row, int h0, int nh, int kvh,
                                             uint32_t (&qb)[NT][HEAD / 16][2], float (&c)[NT][2]) {
  using QE = Elem<QDT>;
  constexpr int KS = HEAD / 16;
  const AttnParams& a = p.a;
  const int lane = threadIdx.x & 31, qn = lane >> 2, qq = lane & 3;
  const float base = a.scale * kLog2e;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int map = NT == 1 ? qn >> 2 : t, n = NT == 1 ? qn & 3 : qn;
    const bool live = n < nh;
    const typename QE::T* q =
        static_cast<const typename QE::T*>(a.q) + (row * a.num_q_heads + 2 * (h0 + (live ? n : 0)) + map) * HEAD;
    if constexpr (!is_fp8<KVDT>()) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(q);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[t][ks][0] = live ? w[8 * ks + qq] : 0u;
        qb[t][ks][1] = live ? w[8 * ks + 4 + qq] : 0u;
      }
      c[t][0] = c[t][1] = base;
    } else {
      // step ks: rows 2 qq, 2 qq + 1 are dims 32 qq + 4 ks + {0, 1}, rows 8 behind them + {2, 3}
      float x[KS][4], top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[ks][e] = live ? QE::load(q + 32 * qq + 4 * ks + e) : 0.f;
          top = fmaxf(top, fabsf(x[ks][e]));
        }
      top = warp_max_xor(top, 1, 2);
      int ex = 0;
      frexpf(top, &ex);
      const int sh = max(-100, min(100, 15 - ex));
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[t][ks][0] = pack2<PA_F16>(ldexpf(x[ks][0], sh), ldexpf(x[ks][1], sh));
        qb[t][ks][1] = pack2<PA_F16>(ldexpf(x[ks][2], sh), ldexpf(x[ks][3], sh));
      }
      const float mine = ldexpf(base * a.k_scale[(kvh + map) * a.scale_stride], -sh);
      c[t][0] = __shfl_sync(0xffffffffu, mine, 8 * qq);
      c[t][1] = __shfl_sync(0xffffffffu, mine, 8 * qq + 4);
    }
  }
}

// Key tile `k` (16 tokens from 16 mt on) times the queries of column tile t, into s.
template <int QDT, int KVDT, int HEAD, int TOK, int NT>
__device__ __forceinline__ void score_tile(const uint8_t* k, int mt, const uint32_t (&qb)[HEAD / 16][2], float (&s)[4]) {
  using G = Geom<QDT, KVDT, HEAD, TOK, NT>;
  const int lane = threadIdx.x & 31, qq = lane & 3;
  float s2[4] = {0.f, 0.f, 0.f, 0.f};  // a second, independent chain
  s[0] = s[1] = s[2] = s[3] = 0.f;
  if constexpr (!G::kFp8) {
    const uint32_t kb = smem_u32(k);
#pragma unroll
    for (int ks = 0; ks < G::kSteps; ++ks) {
      const int tok = 16 * mt + (lane & 7) + 8 * ((lane >> 3) & 1);
      uint32_t a0, a1, a2, a3;
      ldsm_x4(kb + G::off(tok, 2 * ks + (lane >> 4)), a0, a1, a2, a3);
      mma_16816<QDT>(ks & 1 ? s2 : s, a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
    }
  } else {
    const int tA = 16 * mt + (lane >> 2), tB = tA + 8;
    const uint4 a0 = *reinterpret_cast<const uint4*>(k + swz128(tA, 2 * qq));
    const uint4 a1 = *reinterpret_cast<const uint4*>(k + swz128(tA, 2 * qq + 1));
    const uint4 b0 = *reinterpret_cast<const uint4*>(k + swz128(tB, 2 * qq));
    const uint4 b1 = *reinterpret_cast<const uint4*>(k + swz128(tB, 2 * qq + 1));
    const uint32_t wa[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    const uint32_t wb[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
    for (int ks = 0; ks < G::kSteps; ++ks) {
      uint32_t f0, f1, f2, f3;
      fp8x4_to_f16x2x2<KVDT>(wa[ks], f0, f2);
      fp8x4_to_f16x2x2<KVDT>(wb[ks], f1, f3);
      mma_16816<PA_F16>(ks & 1 ? s2 : s, f0, f1, f2, f3, qb[ks][0], qb[ks][1]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] += s2[e];
}

// One unit of tokens into a warp's state; its tokens lo .. rem - 1 are attended.
template <int QDT, int KVDT, int HEAD, int TOK, int NT>
__device__ __forceinline__ void attend_unit(const uint8_t* stage, int rem, int lo,
                                            const uint32_t (&qb)[NT][HEAD / 16][2], const float (&c)[NT][2],
                                            State<HEAD, NT>& w) {
  using G = Geom<QDT, KVDT, HEAD, TOK, NT>;
  constexpr int MDT = G::kFp8 ? PA_F16 : QDT;
  const int lane = threadIdx.x & 31, qq = lane & 3;
  const bool part = rem < TOK || lo > 0;

  float sc[NT][G::kMTiles][4];
#pragma unroll
  for (int mt = 0; mt < G::kMTiles; ++mt) {
    if constexpr (NT == 1) {
      float s2[4];
      score_tile<QDT, KVDT, HEAD, TOK, NT>(stage, mt, qb[0], sc[0][mt]);
      score_tile<QDT, KVDT, HEAD, TOK, NT>(stage + G::kTile, mt, qb[0], s2);
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[0][mt][e] = qq < 2 ? sc[0][mt][e] : s2[e];  // columns 4 on are map 2's
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) score_tile<QDT, KVDT, HEAD, TOK, NT>(stage + t * G::kTile, mt, qb[t], sc[t][mt]);
    }
  }
  if (part) {
#pragma unroll
    for (int mt = 0; mt < G::kMTiles; ++mt) {
      const int t0 = 16 * mt + (lane >> 2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t0 >= rem || t0 < lo) sc[t][mt][0] = sc[t][mt][1] = -INFINITY;
        if (t0 + 8 >= rem || t0 + 8 < lo) sc[t][mt][2] = sc[t][mt][3] = -INFINITY;
      }
    }
  }

  // online softmax, fp32; the maximum is raised only past a slack (see kRescaleSlack)
  uint32_t pb[NT][G::kMTiles][2], pr[NT][G::kMTiles][2];  // weights, and what they leave out
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int mt = 0; mt < G::kMTiles; ++mt) {
      top[0] = fmaxf(top[0], fmaxf(sc[t][mt][0], sc[t][mt][2]));
      top[1] = fmaxf(top[1], fmaxf(sc[t][mt][1], sc[t][mt][3]));
    }
    top[0] = warp_max_xor(top[0], 4, 16) * c[t][0];
    top[1] = warp_max_xor(top[1], 4, 16) * c[t][1];
    if (__any_sync(0xffffffffu, top[0] > w.m[t][0] + kRescaleSlack || top[1] > w.m[t][1] + kRescaleSlack)) {
      float al[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float nm = fmaxf(w.m[t][k], top[k]);
        al[k] = nm == -INFINITY ? 1.f : ex2_approx(w.m[t][k] - nm);
        w.m[t][k] = nm;
        w.l[t][k] *= al[k];
      }
#pragma unroll
      for (int i = 0; i < HEAD / 8; ++i) {
        w.acc[t][i][0] *= al[0];
        w.acc[t][i][1] *= al[1];
        w.acc[t][i][2] *= al[0];
        w.acc[t][i][3] *= al[1];
      }
    }
    const float u0 = w.m[t][0] == -INFINITY ? 0.f : w.m[t][0], u1 = w.m[t][1] == -INFINITY ? 0.f : w.m[t][1];
#pragma unroll
    for (int mt = 0; mt < G::kMTiles; ++mt) {
      const float e0 = ex2_approx(fmaf(sc[t][mt][0], c[t][0], -u0)), e1 = ex2_approx(fmaf(sc[t][mt][1], c[t][1], -u1));
      const float e2 = ex2_approx(fmaf(sc[t][mt][2], c[t][0], -u0)), e3 = ex2_approx(fmaf(sc[t][mt][3], c[t][1], -u1));
      const uint32_t x = pack2<MDT>(e0, e1), y = pack2<MDT>(e2, e3);
      const float2 fx = unpack2<MDT>(x), fy = unpack2<MDT>(y);
      pb[t][mt][0] = movmatrix_trans(x);
      pb[t][mt][1] = movmatrix_trans(y);
      if constexpr (G::kSplit) {
        w.l[t][0] += e0 + e2;
        w.l[t][1] += e1 + e3;
        pr[t][mt][0] = movmatrix_trans(pack2<MDT>(e0 - fx.x, e1 - fx.y));
        pr[t][mt][1] = movmatrix_trans(pack2<MDT>(e2 - fy.x, e3 - fy.y));
      } else {  // the sums are of the rounded weights that meet V
        w.l[t][0] += fx.x + fy.x;
        w.l[t][1] += fx.y + fy.y;
      }
    }
  }

  // O^T += V^T P^T; values that no row attends may hold anything and are taken as 0
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint8_t* v = stage + (2 + half) * G::kTile;
#pragma unroll
    for (int kt = 0; kt < G::kMTiles; ++kt) {
      const int tk = 16 * kt + 2 * qq;  // tokens of this thread's A halves: tk, tk + 1, tk + 8, tk + 9
      auto in = [&](int tok) { return tok < rem && tok >= lo; };
      if constexpr (!G::kFp8) {
        const uint32_t m01 = (in(tk) ? 0xffffu : 0u) | (in(tk + 1) ? 0xffff0000u : 0u);
        const uint32_t m89 = (in(tk + 8) ? 0xffffu : 0u) | (in(tk + 9) ? 0xffff0000u : 0u);
        const uint32_t vb = smem_u32(v);
#pragma unroll
        for (int dt = 0; dt < G::kSteps; ++dt) {
          const int tok = 16 * kt + (lane & 7) + 8 * (lane >> 4);
          uint32_t a0, a1, a2, a3;
          ldsm_x4_trans(vb + G::off(tok, 2 * dt + ((lane >> 3) & 1)), a0, a1, a2, a3);
          if (part) {
            a0 &= m01;
            a1 &= m01;
            a2 &= m89;
            a3 &= m89;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_16816<MDT>(w.acc[t][half * G::kSteps + dt], a0, a1, a2, a3, pb[t][kt][0], pb[t][kt][1]);
            if constexpr (G::kSplit)
              mma_16816<MDT>(w.acc[t][half * G::kSteps + dt], a0, a1, a2, a3, pr[t][kt][0], pr[t][kt][1]);
          }
        }
      } else {
        // dims 16 (lane >> 2) .. + 15 of those tokens
        const int rr = lane >> 2;
        uint4 x[4];
        x[0] = *reinterpret_cast<const uint4*>(v + swz128(tk, rr));
        x[1] = *reinterpret_cast<const uint4*>(v + swz128(tk + 1, rr));
        x[2] = *reinterpret_cast<const uint4*>(v + swz128(tk + 8, rr));
        x[3] = *reinterpret_cast<const uint4*>(v + swz128(tk + 9, rr));
        if (part) {
          if (!in(tk)) x[0] = make_uint4(0, 0, 0, 0);
          if (!in(tk + 1)) x[1] = make_uint4(0, 0, 0, 0);
          if (!in(tk + 8)) x[2] = make_uint4(0, 0, 0, 0);
          if (!in(tk + 9)) x[3] = make_uint4(0, 0, 0, 0);
        }
        const uint32_t w0[4] = {x[0].x, x[0].y, x[0].z, x[0].w}, w1[4] = {x[1].x, x[1].y, x[1].z, x[1].w};
        const uint32_t w2[4] = {x[2].x, x[2].y, x[2].z, x[2].w}, w3[4] = {x[3].x, x[3].y, x[3].z, x[3].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // dims 16 rr + 4 k .. + 3: dim tiles 2 k, 2 k + 1
          uint32_t c01[4], c89[4];
          fp8x4_to_f16x2x2<KVDT>(__byte_perm(w0[k], w1[k], 0x5140), c01[0], c01[1]);
          fp8x4_to_f16x2x2<KVDT>(__byte_perm(w0[k], w1[k], 0x7362), c01[2], c01[3]);
          fp8x4_to_f16x2x2<KVDT>(__byte_perm(w2[k], w3[k], 0x5140), c89[0], c89[1]);
          fp8x4_to_f16x2x2<KVDT>(__byte_perm(w2[k], w3[k], 0x7362), c89[2], c89[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_16816<PA_F16>(w.acc[t][half * G::kSteps + 2 * k], c01[0], c01[1], c89[0], c89[1], pb[t][kt][0],
                              pb[t][kt][1]);
            mma_16816<PA_F16>(w.acc[t][half * G::kSteps + 2 * k + 1], c01[2], c01[3], c89[2], c89[3], pb[t][kt][0],
                              pb[t][kt][1]);
            if constexpr (G::kSplit) {
              mma_16816<PA_F16>(w.acc[t][half * G::kSteps + 2 * k], c01[0], c01[1], c89[0], c89[1], pr[t][kt][0],
                                pr[t][kt][1]);
              mma_16816<PA_F16>(w.acc[t][half * G::kSteps + 2 * k + 1], c01[2], c01[3], c89[2], c89[3], pr[t][kt][0],
                                pr[t][kt][1]);
            }
          }
        }
      }
    }
  }
}

template <int QDT, int KVDT, int HEAD, int TOK, int NT>
__global__ void __launch_bounds__(kWarps * 32) diff_decode_kernel(const __grid_constant__ DiffDecodeArgs args) {
  using G = Geom<QDT, KVDT, HEAD, TOK, NT>;
  using QE = Elem<QDT>;
  constexpr int ST = G::kStages, W = 2 * HEAD;
  const DiffParams& p = args.p;
  const AttnParams& a = p.a;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bars[kWarps * ST];
  __shared__ int stage_ok[kWarps * ST];
  __shared__ int s_failed;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x, z = blockIdx.z;
  const int g = blockIdx.y / args.head_groups, hg = blockIdx.y % args.head_groups;
  const int kvh = 2 * g;
  const int heads = a.num_q_heads / 2;
  const int h0 = g * a.group + hg * args.heads_cta, nh = min(args.heads_cta, a.group - hg * args.heads_cta);
  const int bs = a.block_size;

  if (threadIdx.x == 0) {
    s_failed = 0;
    tma_prefetch_desc(&args.tk);
    tma_prefetch_desc(&args.tv);
    for (int i = 0; i < kWarps * ST; ++i) mbar_init(bars + i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  previous_done();

  int row = r;
  if (a.query_start_loc != nullptr) {
    if (plan_rejected(a)) return;
    const int q0 = a.query_start_loc[r];
    if (a.query_start_loc[r + 1] - q0 != 1) return;  // rows of several tokens go elsewhere
    row = q0;
  }
  const int seq_len = a.seq_lens[r];
  if (seq_len < 1 || seq_len > a.max_seq_len || (long long)seq_len > (long long)a.max_blocks_per_seq * bs) {
    if (z == 0) {
      typename QE::T* out = static_cast<typename QE::T*>(a.out) + ((long long)row * heads + h0) * W;
      for (int i = threadIdx.x; i < nh * W; i += kWarps * 32) out[i] = QE::from_float(0.f);
      if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err, PA_ERRFLAG_SEQ_LEN);
    }
    return;
  }
  const int origin = window_origin(a, seq_len, 1);
  const int first = a.window > 0 ? max(0, seq_len - a.window) : 0;  // first key attended
  const int t0 = origin + z * a.part, t1 = min(t0 + a.part, seq_len);
  if (t0 >= seq_len) return;
  const int nparts = (seq_len - origin + a.part - 1) / a.part;
  const int u0 = max(t0, first) / TOK, u1 = (t1 + TOK - 1) / TOK;  // units of this CTA (none if all before the window)

  const int32_t* table = a.block_tables + (long long)r * a.max_blocks_per_seq;
  const int nmine = u1 - u0 > warp ? (u1 - u0 - warp + kWarps - 1) / kWarps : 0;
  uint8_t* ring = smem + warp * ST * G::kStage;
  uint64_t* wbars = bars + warp * ST;
  int* wok = stage_ok + warp * ST;
  // table entries of this warp's units, 32 at a time in registers, the next 32 on their way
  auto load_window = [&](int base) {
    const int i = base + lane;
    return i < nmine ? table[(u0 + warp + i * kWarps) * TOK / bs] : -1;
  };
  int tbl = load_window(0), tbl_next = load_window(32);
  auto issue = [&](int i, int phys) {
    if (lane == 0) {
      const int s = i % ST;
      const bool valid = phys >= 0 && phys < a.num_blocks;
      wok[s] = valid;
      if (!valid) {
        flag_error(a.err, PA_ERRFLAG_BLOCK_TABLE);
        mbar_arrive(wbars + s);  // a phase without data: the unit is skipped
      } else {
        uint8_t* st = ring + s * G::kStage;
        const int y = kvh * bs + (u0 + warp + i * kWarps) * TOK % bs;
        mbar_arrive_expect_tx(wbars + s, G::kStage);
        tma_load_4d(st, &args.tk, 0, y, 0, phys, wbars + s);
        tma_load_4d(st + G::kTile, &args.tk, 0, y + bs, 0, phys, wbars + s);
        tma_load_4d(st + 2 * G::kTile, &args.tv, 0, y, 0, phys, wbars + s);
        tma_load_4d(st + 3 * G::kTile, &args.tv, 0, y + bs, 0, phys, wbars + s);
      }
    }
  };
  for (int i = 0; i < min(ST, nmine); ++i) issue(i, __shfl_sync(0xffffffffu, tbl, i));

  uint32_t qb[NT][HEAD / 16][2];
  float c[NT][2];
  load_queries<QDT, KVDT, HEAD, NT>(p, row, h0, nh, kvh, qb, c);
  State<HEAD, NT> w;
  w.init();
  bool failed = false;
  int consumed = 0;
  for (int i = 0; i < nmine; ++i) {
    const int s = i % ST;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(wbars + s, (i / ST) & 1))) {
      failed = true;
      break;
    }
    consumed = i + 1;
    if (wok[s]) {
      const int at = (u0 + warp + i * kWarps) * TOK;
      attend_unit<QDT, KVDT, HEAD, TOK, NT>(ring + s * G::kStage, seq_len - at, first - at, qb, c, w);
    }
    __syncwarp();
    const int j = i + ST;
    if (j < nmine) {
      if ((j & 31) == 0) {
        tbl = tbl_next;
        tbl_next = load_window(j + 32);
      }
      const int phys = __shfl_sync(0xffffffffu, tbl, j & 31);
      if (lane == 0) fence_proxy_async();
      issue(j, phys);
    }
  }
  if (failed) {
    // a copy never completed: note it, let the ones in flight land (with a limit), write nothing
    if (lane == 0) {
      flag_error(a.err, PA_ERRFLAG_TIMEOUT);
      for (int i = consumed; i < min(consumed + ST, nmine); ++i)
        (void)mbar_wait_bounded(wbars + (i % ST), (i / ST) & 1, 100000000ull);
    }
    s_failed = 1;
  }

  // ---- the warps' states meet in shared memory: [warp][column][2 HEAD], maxima and sums behind
  __syncthreads();
  if (s_failed) return;
  float* red = reinterpret_cast<float*>(smem);
  float2* red_ml = reinterpret_cast<float2*>(red + kWarps * NT * 8 * G::kRedRow);
  {
    const int qq = lane & 3, rr = lane >> 2;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float l = warp_sum_xor(w.l[t][k], 4, 16);
        const int col = (warp * NT + t) * 8 + 2 * qq + k;
        if (lane < 4) red_ml[col] = make_float2(w.m[t][k], l);
#pragma unroll
        for (int i = 0; i < HEAD / 8; ++i) {
          const int dt = i % G::kSteps, half = i / G::kSteps * HEAD;
          const int dA = half + (G::kFp8 ? 16 * rr + 2 * dt : 16 * dt + rr);
          red[col * G::kRedRow + dA] = w.acc[t][i][k];
          red[col * G::kRedRow + (G::kFp8 ? dA + 1 : dA + 8)] = w.acc[t][i][2 + k];
        }
      }
    }
  }
  __syncthreads();
  const bool direct = nparts == 1;
  const long long pi = (a.part_off ? (long long)a.part_off[r] : (long long)row * a.max_partitions) + z;
  float vs[2] = {1.f, 1.f};
  if constexpr (G::kFp8) {
    vs[0] = a.v_scale[kvh * a.scale_stride];
    vs[1] = a.v_scale[(kvh + 1) * a.scale_stride];
  }
  for (int n = warp; n < nh; n += kWarps) {
    float2 o[2][W / 64];
    float M[2], L[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = NT == 1 ? 4 * j + n : 8 * j + n;
      M[j] = -INFINITY;
      L[j] = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float2 ml = red_ml[v * NT * 8 + col];
        if (ml.y > 0.f) M[j] = fmaxf(M[j], ml.x);
      }
#pragma unroll
      for (int k = 0; k < W / 64; ++k) o[j][k] = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float2 ml = red_ml[v * NT * 8 + col];
        if (!(ml.y > 0.f)) continue;
        const float f = exp2f(ml.x - M[j]);
        L[j] = fmaf(ml.y, f, L[j]);
        const float2* x = reinterpret_cast<const float2*>(red + (v * NT * 8 + col) * G::kRedRow);
#pragma unroll
        for (int k = 0; k < W / 64; ++k) {
          const float2 y = x[32 * k + lane];
          o[j][k].x = fmaf(y.x, f, o[j][k].x);
          o[j][k].y = fmaf(y.y, f, o[j][k].y);
        }
      }
#pragma unroll
      for (int k = 0; k < W / 64; ++k) {
        o[j][k].x *= vs[k >= W / 128];
        o[j][k].y *= vs[k >= W / 128];
      }
    }
    const int h = h0 + n;
    if (direct) {
      const float w0 = diff_weight(L[0]), w1 = diff_weight(L[1]) * diff_lambda(p, row, h);
#pragma unroll
      for (int k = 0; k < W / 64; ++k) {
        o[0][k].x = o[0][k].x * w0 - o[1][k].x * w1;
        o[0][k].y = o[0][k].y * w0 - o[1][k].y * w1;
      }
      diff_finish<QDT>(p, row, h, W, o[0]);
    } else {
      if (n + kWarps >= nh) next_may_start();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const long long at = pi * a.num_q_heads + 2 * h + j;
#pragma unroll
        for (int k = 0; k < W / 64; ++k) reinterpret_cast<float2*>(a.ws_acc + at * W)[32 * k + lane] = o[j][k];
        if (lane == 0) a.ws_ml[at] = make_float2(M[j], L[j]);
      }
    }
  }
}

template <int QDT, int KVDT, int HEAD, int TOK, int NT>
cudaError_t launch_t(const DiffParams& p, int grid_z, const CUtensorMap* tk, const CUtensorMap* tv,
                     cudaStream_t stream) {
  constexpr auto kernel = diff_decode_kernel<QDT, KVDT, HEAD, TOK, NT>;
  constexpr int smem = Geom<QDT, KVDT, HEAD, TOK, NT>::kSmem;
  const cudaError_t e = set_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  DiffDecodeArgs args;
  args.p = p;
  args.heads_cta = NT == 1 ? 4 : 8;
  args.head_groups = (p.a.group + args.heads_cta - 1) / args.heads_cta;
  args.tk = *tk;
  args.tv = *tv;
  return launch_early<DiffDecodeArgs>(kernel, dim3(p.a.num_seqs, p.a.num_kv_heads / 2 * args.head_groups, grid_z),
                                      kWarps * 32, smem, 1, args, stream);
}

// One column tile for up to four heads a group, a tile a map for more.
template <int QDT, int KVDT, int HEAD, int TOK>
cudaError_t launch_heads(const DiffParams& p, int grid_z, const CUtensorMap* tk, const CUtensorMap* tv,
                         cudaStream_t s) {
  return p.a.group <= 4 ? launch_t<QDT, KVDT, HEAD, TOK, 1>(p, grid_z, tk, tv, s)
                        : launch_t<QDT, KVDT, HEAD, TOK, 2>(p, grid_z, tk, tv, s);
}

template <int QDT>
cudaError_t launch_query(const DiffParams& p, int kv_dtype, int grid_z, const CUtensorMap* tk, const CUtensorMap* tv,
                         cudaStream_t s) {
  const int d = p.a.head_size, tok = diff_decode_unit(kv_dtype, d, p.a.block_size);
  if (kv_dtype == QDT && d == 128) return launch_heads<QDT, QDT, 128, 16>(p, grid_z, tk, tv, s);
  if (kv_dtype == QDT && d == 64)
    return tok == 32 ? launch_heads<QDT, QDT, 64, 32>(p, grid_z, tk, tv, s)
                     : launch_heads<QDT, QDT, 64, 16>(p, grid_z, tk, tv, s);
  if (kv_dtype == PA_FP8_E4M3 && d == 128)
    return tok == 32 ? launch_heads<QDT, PA_FP8_E4M3, 128, 32>(p, grid_z, tk, tv, s)
                     : launch_heads<QDT, PA_FP8_E4M3, 128, 16>(p, grid_z, tk, tv, s);
  if (kv_dtype == PA_FP8_E5M2 && d == 128)
    return tok == 32 ? launch_heads<QDT, PA_FP8_E5M2, 128, 32>(p, grid_z, tk, tv, s)
                     : launch_heads<QDT, PA_FP8_E5M2, 128, 16>(p, grid_z, tk, tv, s);
  return cudaErrorInvalidValue;
}

}  // namespace

bool diff_decode_supported(int q_dtype, int kv_dtype, int head_size, int block_size) {
  if (q_dtype != PA_BF16 && q_dtype != PA_F16) return false;
  if (block_size % 16) return false;
  if (kv_dtype == q_dtype) return head_size == 64 || head_size == 128;
  return (kv_dtype == PA_FP8_E4M3 || kv_dtype == PA_FP8_E5M2) && head_size == 128;
}

// Tokens of a unit: 16 KB of the four tiles, where blocks hold that many.
int diff_decode_unit(int kv_dtype, int head_size, int block_size) {
  const int row = head_size * (kv_dtype == PA_FP8_E4M3 || kv_dtype == PA_FP8_E5M2 ? 1 : 2);
  return row == 128 && block_size % 32 == 0 ? 32 : 16;
}

cudaError_t launch_diff_decode(const DiffParams& p, int q_dtype, int kv_dtype, int grid_z, const CUtensorMap* tmap_k,
                               const CUtensorMap* tmap_v, cudaStream_t stream) {
  if (q_dtype == PA_BF16) return launch_query<PA_BF16>(p, kv_dtype, grid_z, tmap_k, tmap_v, stream);
  if (q_dtype == PA_F16) return launch_query<PA_F16>(p, kv_dtype, grid_z, tmap_k, tmap_v, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
