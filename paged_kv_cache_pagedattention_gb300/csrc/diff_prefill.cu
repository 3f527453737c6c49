// Differential attention of multi-token rows on the 5th-generation tensor cores.
//
// A persistent grid, one CTA per SM; a CTA works on one map of a tile: a work item of the varlen
// plan (request, first query row, partition of the keys) for one (KV group, group of <= 8 heads).
// A tile's rows are (token, head) pairs, token-major (row = token * GP + head, GP = the head group
// padded to a power of two), 128 to a row tile; row r lives in TMEM lane r.  The value row is twice
// as wide as a key, so a map's accumulators take 2 head_size columns: one row tile with head_size
// 128, two with 64.  Keys stream in chunks of 64 tokens (whole paged blocks).  Per chunk i:
//   S(i)  = Q_j K_j(i)^T    M = 128 rows, N = 64 keys, K = head_size         -> TMEM (2 buffers)
//   P(i)  = softmax numerators of S(i), 16-bit, over S(i)                    -> TMEM
//   O    += P(i) [V_1 V_2](i)   M = 128, N = 2 head_size, K = 64 keys        -> TMEM
// Warps: four for the softmax of a row tile (a row a thread), two TMA producers (K; V), one issuer
// of MMAs a row tile, and for FP8 caches six that widen codes to f16.
#include <algorithm>

#include "diff.cuh"
#include "tcgen05.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;   // rows of a row tile = TMEM lanes
constexpr int kChunk = 64;   // keys of a chunk
constexpr int kSBufs = 2;    // S / P buffers of a row tile, 64 TMEM columns each
constexpr int kOCol = kSBufs * 64;
constexpr int kConvThreads = 192;
constexpr int kValidRing = 16;

template <int HEAD, int BS, bool F8>
struct DiffTc {
  static constexpr int kTiles = HEAD == 128 ? 1 : 2;
  static constexpr int kTileCols = HEAD == 128 ? 512 : 256;  // kOCol + 2 HEAD used
  static constexpr int kWide = 2 * HEAD;
  static constexpr int kPieces = HEAD / 64;                  // 128-byte pieces of a 16-bit key
  static constexpr int kBlocks = kChunk / BS;
  static constexpr int kPiece = kChunk * 128;
  static constexpr int kKBytes = kPieces * kPiece;           // keys of a chunk
  static constexpr int kVBytes = 2 * kKBytes;                // values of a chunk
  static constexpr int kStageBytes = kKBytes + kVBytes;
  static constexpr int kStages = F8 ? 3 : HEAD == 128 ? 4 : 7;
  static constexpr int kQPiece = kRows * 128;
  static constexpr int kQTile = kPieces * kQPiece;
  // FP8: codes land in a staging ring, [K | V_1 | V_2][block][token][head_size bytes]
  static constexpr int kStg = F8 ? 2 : 0;
  static constexpr int kStgBlock = BS * HEAD;
  static constexpr int kStgTensor = kBlocks * kStgBlock;
  static constexpr int kStgOff = kTiles * kQTile + kStages * kStageBytes;
  static constexpr int kBarOff = kStgOff + kStg * 3 * kStgTensor;
  static constexpr int kNumBars = 2 * kStages + 3 * kSBufs * kTiles + 1 + 2 * kStg;
  static constexpr int kSmem = 1024 + kBarOff + 8 * kNumBars + 16;
  static constexpr int kProducer = 4 * kTiles, kMma = kProducer + 2, kConv = kMma + kTiles;
  static constexpr int kThreads = (kConv + (F8 ? kConvThreads / 32 : 0)) * 32;
  static_assert(kBlocks * BS == kChunk, "block size must divide the chunk");
  static_assert(kOCol + kWide <= kTileCols && kTiles * kTileCols <= 512, "TMEM columns");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(!F8 || HEAD == 128, "FP8 rows are one 128-byte piece");
};

// Byte offset, inside a chunk's V, of key `key`'s row in piece `pc` (the pieces of both halves).
template <int HEAD, int BS>
__device__ __forceinline__ uint32_t v_row_off(int key, int pc) {
  return (uint32_t)((key / BS) * (HEAD / 32) * BS * 128 + pc * BS * 128 + (key % BS) * 128);
}

struct DiffPrefillArgs {
  DiffParams p;
  CUtensorMap tk, tv;
};

template <int QDT, int KVDT, int HEAD, int BS>
__global__ void __launch_bounds__(DiffTc<HEAD, BS, is_fp8<KVDT>()>::kThreads, 1)
    diff_prefill_kernel(const __grid_constant__ DiffPrefillArgs args) {
  constexpr bool kCvt = is_fp8<KVDT>();
  constexpr int ODT = kCvt ? PA_F16 : QDT;
  using G = DiffTc<HEAD, BS, kCvt>;
  using QE = Elem<QDT>;
  constexpr int ST = G::kStages, NB = G::kBlocks, NT = G::kTiles;
  const AttnParams& p = args.p.a;

  if (plan_rejected(p)) return;
  const int nwork = *p.work_count;
  const int nfull = *p.work_full;
  const int num_groups = (p.group + 7) / 8;
  const int ny = p.num_kv_heads * num_groups;  // (KV group, head group, map)
  const int total = nwork * ny;
  const int total_full = nfull * ny;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + NT * G::kQTile;
  uint8_t* sStg = smem + G::kStgOff;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kBarOff);
  uint64_t* empty = full + ST;
  // Row tile t, buffer b (chunk i: b = i % 2, phase i / 2): S(i) is in TMEM, P(i) is, PV(i) is done
  uint64_t* s_full = empty + ST;
  uint64_t* p_full = s_full + NT * kSBufs;
  uint64_t* o_done = p_full + NT * kSBufs;
  uint64_t* mma_fin = o_done + NT * kSBufs;
  uint64_t* stg_full = mma_fin + 1;
  uint64_t* stg_empty = stg_full + G::kStg;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stg_empty + G::kStg);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int s_next, s_abort;
  // bit b: block b of a chunk can be read; chunks are at most ST + kStg apart
  __shared__ int s_valid[kValidRing];
  static_assert(ST + G::kStg < kValidRing, "a chunk's word outlives its stage");
  constexpr int RS = kCvt ? G::kStg : ST;  // the copies' ring
  uint64_t* rfull = kCvt ? stg_full : full;
  uint64_t* rempty = kCvt ? stg_empty : empty;

  if (tid == 0) {
    tma_prefetch_desc(&args.tk);
    tma_prefetch_desc(&args.tv);
    for (int i = 0; i < ST; ++i) {
      mbar_init(full + i, kCvt ? kConvThreads : 2);
      mbar_init(empty + i, NT);
    }
    for (int i = 0; i < G::kStg; ++i) {
      mbar_init(stg_full + i, 2);
      mbar_init(stg_empty + i, kConvThreads);
    }
    for (int i = 0; i < NT * kSBufs; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, kRows);
      mbar_init(o_done + i, 1);
    }
    mbar_init(mma_fin, NT);
    fence_mbar_init();
    s_next = atomicAdd(p.work_claim, 1);
    s_abort = 0;
  }
  __syncthreads();
  int L = s_next;
  if (L >= total) return;
  if (warp == G::kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  int gch = 0;               // ring chunks of earlier tiles
  int tch[NT] = {};          // a row tile's chunks of earlier tiles
  int g_issued = 0;
  for (;;) {
    const int lc = L < total_full ? L : L - total_full;
    const int nc = L < total_full ? nfull : nwork - nfull;
    // (item, map) pairs run fastest but for the group, so that both maps of a tile are in flight together
    const int x = (L < total_full ? 0 : nfull) + (lc >> 1) % nc, y = (lc >> 1) / nc, map = lc & 1;
    const int4 item = p.work[x];
    const int r = item.x, row0 = item.y, z = item.z;
    const int g = y / num_groups, hg = y % num_groups, kvh = 2 * g;
    const int h0 = g * p.group + hg * 8;
    const int nh = min(8, p.group - hg * 8);
    int gp = 1;
    while (gp < min(p.group, 8)) gp <<= 1;
    const int tile_tokens = kRows / gp;
    const int qs = p.query_start_loc[r];
    const int q_len = p.query_start_loc[r + 1] - qs;
    const int seq_len = p.seq_lens[r];
    const int t0 = row0 - qs;
    const int ntok = min(NT * tile_tokens, q_len - t0);
    const int pos0 = seq_len - q_len + t0;
    const int part = p.part_pf;
    const int origin = window_origin(p, seq_len, q_len);
    const int parts_req = (seq_len - origin + part - 1) / part;
    const int k0 = origin + z * part;
    const int klo = p.window > 0 ? max(k0, max(0, pos0 - p.window + 1) / BS * BS) : k0;
    auto tile_chunks = [&](int t) {
      const int nt = min(ntok, (t + 1) * tile_tokens) - t * tile_tokens;
      if (nt <= 0) return 0;
      const int k1t = min(k0 + part, p.causal ? pos0 + t * tile_tokens + nt : seq_len);
      return k1t > klo ? (k1t - klo + kChunk - 1) / kChunk : 0;
    };
    int nch_t[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) nch_t[t] = tile_chunks(t);
    const int k1 = min(k0 + part, p.causal ? pos0 + ntok : seq_len);
    const int nch = k1 > klo ? (k1 - klo + kChunk - 1) / kChunk : 0;
    const int kb_first = klo / BS;
    // V rows past the sequence's tokens are zeroed before they meet P: only the last chunk has such,
    // and the last row tile that reads it zeroes them
    const int kv_loaded_end = min(seq_len, (k1 + BS - 1) / BS * BS);
    const bool tail_chunk = nch > 0 && klo + nch * kChunk > kv_loaded_end;
    const int zero_tile = nch_t[NT - 1] == nch ? NT - 1 : 0;

    const int row_tok = tid / gp, row_head = tid % gp;
    const bool row_valid = tid < NT * kRows && row_tok < ntok && row_head < nh;
    const int row_pos = pos0 + row_tok;
    const int q_head = 2 * (h0 + row_head) + map;
    int q_shift = 0;  // FP8 caches: the row times 2^q_shift fits f16
    if (tid < NT * kRows) {
      const uint4* src = row_valid ? reinterpret_cast<const uint4*>(
                                         static_cast<const typename QE::T*>(p.q) +
                                         ((long long)(row0 + row_tok) * p.num_q_heads + q_head) * HEAD)
                                   : nullptr;
      uint8_t* dst = sQ + (tid / kRows) * G::kQTile;
      if constexpr (!kCvt) {
#pragma unroll
        for (int c = 0; c < HEAD / 8; ++c) {
          const uint4 v = src ? src[c] : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * G::kQPiece + swz128(tid % kRows, c & 7)) = v;
        }
      } else {
        float amax = 0.f;
        for (int c = 0; c < HEAD / 8 && src; ++c) {
          const uint4 v = src[c];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QDT>(w[e]);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        int ex = 0;
        frexpf(amax, &ex);
        q_shift = max(-100, min(100, 15 - ex));
#pragma unroll 4
        for (int c = 0; c < HEAD / 8; ++c) {
          const uint4 v = src ? src[c] : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QDT>(w[e]);
            h[e] = pack2<PA_F16>(ldexpf(f.x, q_shift), ldexpf(f.y, q_shift));
          }
          *reinterpret_cast<uint4*>(dst + (c >> 3) * G::kQPiece + swz128(tid % kRows, c & 7)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();  // the Q rows are in place; every role of the previous tile is done
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int32_t* table = p.block_tables + (long long)r * p.max_blocks_per_seq;

    if (warp == G::kProducer || warp == G::kProducer + 1) {
      // ------------------------------------------------------------ TMA producers
      const bool is_v = warp != G::kProducer;
      const int kb_end = (k1 + BS - 1) / BS;
      auto load_window = [&](int w) {
        const int kb = kb_first + 32 * w + lane;
        return kb < kb_end ? table[kb] : -1;
      };
      int cur_w = 0;
      int win = load_window(0);
      int win_next = load_window(1);
      for (int i = 0; i < nch; ++i) {
        const int gi = gch + i, s = gi % RS;
        if (gi >= RS && !__all_sync(0xffffffffu, mbar_wait_bounded(rempty + s, ((gi / RS) - 1) & 1))) {
          if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
          s_abort = 1;
          break;
        }
        const int w = (i * NB) >> 5;  // NB divides 32: a chunk's blocks share a window
        if (w != cur_w) {
          win = win_next;
          win_next = load_window(w + 1);
          cur_w = w;
        }
        // A block out of range, and the chunk's end behind the last one, is copied from behind the
        // cache's last block: zeros.  Scores of the former are masked by its bit.
        int phys[NB];
        int valid = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int e = __shfl_sync(0xffffffffu, win, (i * NB + b) & 31);
          const bool in_range = kb_first + i * NB + b < kb_end;
          const bool ok_b = e >= 0 && e < p.num_blocks;
          if (in_range && !ok_b && lane == 0 && !is_v) flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
          phys[b] = in_range && ok_b ? e : p.num_blocks;
          valid |= (ok_b || !in_range) << b;
        }
        if (elect_one()) {
          if (!is_v) s_valid[gi % kValidRing] = valid;
          if constexpr (kCvt) {
            uint8_t* sg = sStg + s * 3 * G::kStgTensor;
            mbar_arrive_expect_tx(rfull + s, G::kStgTensor * (is_v ? 2 : 1));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (is_v) {
                for (int h = 0; h < 2; ++h)
                  tma_load_4d(sg + (1 + h) * G::kStgTensor + b * G::kStgBlock, &args.tv, 0, (kvh + h) * BS, 0, phys[b],
                              rfull + s);
              } else {
                tma_load_4d(sg + b * G::kStgBlock, &args.tk, 0, (kvh + map) * BS, 0, phys[b], rfull + s);
              }
            }
          } else {
            uint8_t* sk = sKV + s * G::kStageBytes;
            mbar_arrive_expect_tx(full + s, is_v ? G::kVBytes : G::kKBytes);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (is_v) {
                uint8_t* sv = sk + G::kKBytes + v_row_off<HEAD, BS>(b * BS, 0);
                for (int h = 0; h < 2; ++h)
                  tma_load_4d(sv + h * G::kPieces * BS * 128, &args.tv, 0, (kvh + h) * BS, 0, phys[b], full + s);
              } else {
#pragma unroll
                for (int pc = 0; pc < G::kPieces; ++pc)
                  tma_load_4d(sk + pc * G::kPiece + b * BS * 128, &args.tk, 0, (kvh + map) * BS, pc, phys[b], full + s);
              }
            }
          }
        }
        __syncwarp();
        g_issued = gi + 1;
      }
    } else if (kCvt && warp >= G::kConv) {
      // ------------------------------------------------------------ FP8 converters: a row a thread
      if constexpr (kCvt) {
        const int ct = tid - G::kConv * 32;
        const int tensor = ct / kChunk, key = ct % kChunk;  // K, V_1, V_2
        const int blk = key / BS, tok = key % BS, sw = key & 7;
        for (int i = 0; i < nch; ++i) {
          const int gi = gch + i, s = gi % ST, ss = gi % G::kStg;
          bool ok = mbar_wait_bounded(stg_full + ss, (gi / G::kStg) & 1);
          if (gi >= ST) ok = ok && mbar_wait_bounded(empty + s, ((gi / ST) - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
            s_abort = 1;
            break;
          }
          const uint8_t* srow = sStg + (ss * 3 + tensor) * G::kStgTensor + blk * G::kStgBlock + tok * 128;
          uint8_t* sk = sKV + s * G::kStageBytes;
          uint8_t* drow = tensor == 0 ? sk + key * 128
                                      : sk + G::kKBytes + v_row_off<HEAD, BS>(key, (tensor - 1) * G::kPieces);
          const int piece_stride = tensor == 0 ? G::kPiece : BS * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint4 codes = *reinterpret_cast<const uint4*>(srow + ((q ^ sw) << 4));
            const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) fp8x4_to_f16x2x2<KVDT>(cw[e], h[2 * e], h[2 * e + 1]);
            uint8_t* row = drow + (q >> 2) * piece_stride;
            const int cc = (2 * q) & 7;
            *reinterpret_cast<uint4*>(row + ((cc ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(row + (((cc + 1) ^ sw) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          fence_proxy_async();
          mbar_arrive(stg_empty + ss);
          mbar_arrive(full + s);
        }
      }
    } else if (warp >= G::kMma && warp < G::kConv) {
      // ------------------------------------------------------------ MMA issuers, one warp a row tile
      const int t = NT == 1 ? 0 : warp - G::kMma;
      const int my_nch = NT == 1 ? nch_t[0] : t == 0 ? nch_t[0] : nch_t[NT - 1];
      const int tc = NT == 1 ? tch[0] : t == 0 ? tch[0] : tch[NT - 1];
      const uint32_t fmt = ODT == PA_BF16 ? 1u : 0u;
      const uint32_t id_s = umma_idesc(kRows, kChunk, fmt, 0);
      const uint32_t id_o = umma_idesc(kRows, G::kWide, fmt, 1);
      const uint64_t qd = umma_desc(smem_u32(sQ) + t * G::kQTile, 16, 1024);
      const uint64_t kd0 = umma_desc(smem_u32(sKV), 16, 1024);
      const uint64_t vd0 = umma_desc(smem_u32(sKV) + G::kKBytes, BS * 128, 1024);
      const uint32_t tT = tmem + t * G::kTileCols;
      uint64_t* my_p_full = p_full + t * kSBufs;
      auto issue_s = [&](int j) {
        const uint64_t kd = kd0 + (uint64_t)((((gch + j) % ST) * G::kStageBytes) >> 4);
        const uint32_t d = tT + ((tc + j) % kSBufs) * 64;
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < HEAD / 16; ++ks) {
            const uint32_t qo = ((ks >> 2) * G::kQPiece + (ks & 3) * 32) >> 4;
            const uint32_t ko = ((ks >> 2) * G::kPiece + (ks & 3) * 32) >> 4;
            umma(d, qd + qo, kd + ko, id_s, ks > 0 ? 1u : 0u);
          }
          umma_commit(s_full + t * kSBufs + (tc + j) % kSBufs);
        }
        __syncwarp();
      };
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
      };
      bool ok = true;
      for (int j = 0; ok && j < kSBufs && j < my_nch; ++j) {
        ok = wait_all(full + (gch + j) % ST, ((gch + j) / ST) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_s(j);
      }
      for (int i = 0; ok && i < nch; ++i) {
        const int gi = gch + i, ci = tc + i;
        if (i >= my_nch) {
          // a chunk that this row tile does not read: its stage is released once it has landed
          if (!(ok = wait_all(full + gi % ST, (gi / ST) & 1))) break;
          if (elect_one()) mbar_arrive(empty + gi % ST);
          __syncwarp();
          continue;
        }
        // the last chunk's V is read only after the row tile that zeroes its end has written P
        if (NT > 1 && tail_chunk && i == nch - 1 && t != zero_tile) {
          const int cz = (zero_tile == 0 ? tch[0] : tch[NT - 1]) + i;
          if (!(ok = wait_all(p_full + zero_tile * kSBufs + cz % kSBufs, (cz / kSBufs) & 1))) break;
        }
        if (!(ok = wait_all(my_p_full + ci % kSBufs, (ci / kSBufs) & 1))) break;
        tc_fence_after();
        const uint64_t vd = vd0 + (uint64_t)(((gi % ST) * G::kStageBytes) >> 4);
        const uint32_t pt = tT + (ci % kSBufs) * 64;
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < kChunk / 16; ++ks)
            umma_tmem_a(tT + kOCol, pt + ks * 8, vd + (uint64_t)(v_row_off<HEAD, BS>(16 * ks, 0) >> 4), id_o,
                        (i > 0 || ks > 0) ? 1u : 0u);
          umma_commit(o_done + t * kSBufs + ci % kSBufs);
          umma_commit(empty + gi % ST);
        }
        __syncwarp();
        const int j = i + kSBufs;
        if (j < my_nch) {
          if (!(ok = wait_all(full + (gch + j) % ST, ((gch + j) / ST) & 1))) break;
          tc_fence_after();
          issue_s(j);
        }
      }
      if (!ok) {
        if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
        s_abort = 1;
      }
    } else if (warp < 4 * NT) {
      // ------------------------------------------------------------ softmax: a row a thread
      const int t = NT == 1 ? 0 : warp >> 2;
      const int my_nch = NT == 1 ? nch_t[0] : t == 0 ? nch_t[0] : nch_t[NT - 1];
      const int tc = NT == 1 ? tch[0] : t == 0 ? tch[0] : tch[NT - 1];
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tT = tmem + t * G::kTileCols;
      const uint32_t tO = tT + kOCol;
      uint64_t* my_s_full = s_full + t * kSBufs;
      uint64_t* my_p_full = p_full + t * kSBufs;
      uint64_t* my_o_done = o_done + t * kSBufs;
      const float c = kCvt ? ldexpf(p.scale * kLog2e * p.k_scale[(kvh + map) * p.scale_stride], -q_shift)
                           : p.scale * kLog2e;
      const int row_limit = p.causal ? min(k1, row_pos + 1) : k1;
      const int row_lo = p.window > 0 ? max(0, row_pos - p.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      bool fail = false;
      for (int i = 0; i < my_nch; ++i) {
        const int base = klo + i * kChunk;
        const int ci = tc + i, gi = gch + i;
        const uint32_t tS = tT + (ci % kSBufs) * 64;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(my_s_full + ci % kSBufs, (ci / kSBufs) & 1))) {
          fail = true;
          break;
        }
        tc_fence_after();
        uint32_t sr[kChunk];
        tmem_ld32(tS + lane_base, sr);
        tmem_ld32(tS + 32 + lane_base, sr + 32);
        tmem_wait_ld();
        float sc[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) sc[j] = __uint_as_float(sr[j]);
        const int rem = row_limit - base, lo_rem = row_lo - base;
        if (rem < kChunk || lo_rem > 0) {
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
            if (j >= rem || j < lo_rem) sc[j] = -INFINITY;
        }
        // the chunk has long landed: its word is there to be read
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(full + gi % ST, (gi / ST) & 1))) {
          fail = true;
          break;
        }
        const int valid = s_valid[gi % kValidRing];
        if (valid != (1 << NB) - 1) {
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
            if (!(valid >> (j / BS) & 1)) sc[j] = -INFINITY;
        }
        float mq[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float v = max3(sc[8 * q], sc[8 * q + 1], sc[8 * q + 2]);
          v = max3(v, sc[8 * q + 3], sc[8 * q + 4]);
          v = max3(v, sc[8 * q + 5], sc[8 * q + 6]);
          mq[q] = fmaxf(v, sc[8 * q + 7]);
        }
        const float mx = max3(max3(mq[0], mq[1], mq[2]), max3(mq[3], mq[4], mq[5]), fmaxf(mq[6], mq[7])) * c;
        const bool need = mx > m + kRescaleSlack;
        float al = 1.f;
        if (need) {
          const float nm = fmaxf(m, mx);
          al = ex2_approx(m - nm);
          m = nm;
          l *= al;
        }
        const float u = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = f2_pack(c, c), nu2 = f2_pack(-u, -u);
        uint32_t pk[kChunk / 2];
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int j = 0; j < kChunk / 2; ++j) {
          const float2 v = f2_unpack(f2_fma(f2_pack(sc[2 * j], sc[2 * j + 1]), c2, nu2));
          const float e0 = ex2_approx(v.x), e1 = ex2_approx(v.y);
          acc2[j & 3] = f2_add(acc2[j & 3], f2_pack(e0, e1));
          pk[j] = pack2<ODT>(e0, e1);
        }
        const float2 lsum = f2_unpack(f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3])));
        l += lsum.x + lsum.y;
        // O is rescaled only once PV(i - 1) has completed
        if (__any_sync(0xffffffffu, need) && i > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(my_o_done + (ci - 1) % kSBufs, ((ci - 1) / kSBufs) & 1))) {
            fail = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cb = 0; cb < G::kWide; cb += 32) {
            uint32_t o[32];
            tmem_ld32(tO + cb + lane_base, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
            tmem_st32(tO + cb + lane_base, o);
          }
        }
        tmem_st32(tS + lane_base, pk);  // P(i) over the first half of S(i)'s columns
        // V rows past the loaded keys may hold any bits: zeroed, to keep 0 * V finite
        if (tail_chunk && t == zero_tile && i == nch - 1) {
          const int vrem = kv_loaded_end - base;
          for (int q = tid % kRows; q < 2 * G::kPieces * kChunk; q += kRows) {
            const int key = q % kChunk;
            if (key < vrem) continue;
            uint4* d = reinterpret_cast<uint4*>(sKV + (gi % ST) * G::kStageBytes + G::kKBytes +
                                                v_row_off<HEAD, BS>(key, q / kChunk));
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        tmem_wait_st();
        // PV(i - 2) is observed, so that no phase of o_done is ever two behind
        if (i >= kSBufs &&
            !__all_sync(0xffffffffu, mbar_wait_bounded(my_o_done + ci % kSBufs, ((ci - kSBufs) / kSBufs) & 1))) {
          fail = true;
          break;
        }
        tc_fence_before();
        mbar_arrive(my_p_full + ci % kSBufs);
      }
      if (!fail && my_nch > 0) {
        const int cl = tc + my_nch - 1;
        fail = !__all_sync(0xffffffffu, mbar_wait_bounded(my_o_done + cl % kSBufs, (cl / kSBufs) & 1));
        tc_fence_after();
      }
      if (fail) {
        if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
        s_abort = 1;
      } else {
        // ---- epilogue: the row's partial state (unnormalised O, maximum in log2 units, sum)
        const int kv_len = p.causal ? row_pos + 1 : seq_len;
        const int parts_row = (kv_len - origin + part - 1) / part;
        const bool write = row_valid && z < parts_row;
        const long long pi = (long long)p.part_off[r] + (long long)(t0 + row_tok) * parts_req + z;
        const long long at = pi * p.num_q_heads + q_head;
        float* w_row = p.ws_acc + at * G::kWide;
#pragma unroll 1
        for (int cb = 0; cb < G::kWide; cb += 32) {
          const float vs = kCvt ? p.v_scale[(kvh + cb / HEAD) * p.scale_stride] : 1.f;
          uint32_t o[32];
          if (my_nch > 0) {
            tmem_ld32(tO + cb + lane_base, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
          }
          if (!write) continue;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(w_row + cb + 4 * q) =
                make_float4(__uint_as_float(o[4 * q]) * vs, __uint_as_float(o[4 * q + 1]) * vs,
                            __uint_as_float(o[4 * q + 2]) * vs, __uint_as_float(o[4 * q + 3]) * vs);
        }
        if (write) p.ws_ml[at] = make_float2(m, l);
      }
    }

    gch += nch;
#pragma unroll
    for (int t = 0; t < NT; ++t) tch[t] += nch_t[t];
    if (tid == 0) s_next = atomicAdd(p.work_claim, 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    L = s_next;
    if (L >= total || s_abort) break;
  }

  // ---- every MMA completes and every copy lands before TMEM is released and the CTA leaves
  if (warp >= G::kMma && warp < G::kConv) {
    if (elect_one()) umma_commit(mma_fin);
    __syncwarp();
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(mma_fin, 0)) && lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
  } else if ((warp == G::kProducer || warp == G::kProducer + 1) && lane == 0) {
    for (int j = max(0, g_issued - RS); j < g_issued; ++j)
      if (!mbar_wait_bounded(rfull + j % RS, (j / RS) & 1)) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == G::kMma) {
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int QDT, int KVDT, int HEAD, int BS>
cudaError_t launch_t(const DiffParams& p, int num_items, int max_ctas, const CUtensorMap* tk, const CUtensorMap* tv,
                     cudaStream_t stream) {
  using G = DiffTc<HEAD, BS, is_fp8<KVDT>()>;
  constexpr auto kern = diff_prefill_kernel<QDT, KVDT, HEAD, BS>;
  const cudaError_t e = set_smem<kern>(G::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)num_items * p.a.num_kv_heads * ((p.a.group + 7) / 8);
  const int grid = static_cast<int>(std::min<long long>(tiles, std::max(1, max_ctas)));
  DiffPrefillArgs args;
  args.p = p;
  args.tk = *tk;
  args.tv = *tv;
  kern<<<grid, G::kThreads, G::kSmem, stream>>>(args);
  return cudaGetLastError();
}

template <int QDT, int KVDT, int HEAD>
cudaError_t launch_block(const DiffParams& p, int num_items, int max_ctas, const CUtensorMap* tk,
                         const CUtensorMap* tv, cudaStream_t s) {
  switch (p.a.block_size) {
    case 16: return launch_t<QDT, KVDT, HEAD, 16>(p, num_items, max_ctas, tk, tv, s);
    case 32: return launch_t<QDT, KVDT, HEAD, 32>(p, num_items, max_ctas, tk, tv, s);
    case 64: return launch_t<QDT, KVDT, HEAD, 64>(p, num_items, max_ctas, tk, tv, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int QDT>
cudaError_t launch_query(const DiffParams& p, int kv_dtype, int num_items, int max_ctas, const CUtensorMap* tk,
                         const CUtensorMap* tv, cudaStream_t s) {
  const int d = p.a.head_size;
  if (kv_dtype == QDT && d == 128) return launch_block<QDT, QDT, 128>(p, num_items, max_ctas, tk, tv, s);
  if (kv_dtype == QDT && d == 64) return launch_block<QDT, QDT, 64>(p, num_items, max_ctas, tk, tv, s);
  if (kv_dtype == PA_FP8_E4M3 && d == 128)
    return launch_block<QDT, PA_FP8_E4M3, 128>(p, num_items, max_ctas, tk, tv, s);
  if (kv_dtype == PA_FP8_E5M2 && d == 128)
    return launch_block<QDT, PA_FP8_E5M2, 128>(p, num_items, max_ctas, tk, tv, s);
  return cudaErrorInvalidValue;
}

}  // namespace

// Query tokens of a work item: the row tiles of one CTA.
int diff_prefill_tile_tokens(int group, int head_size) {
  int gp = 1;
  while (gp < group && gp < 8) gp <<= 1;
  return kRows / gp * (head_size == 128 ? 1 : 2);
}

bool diff_prefill_supported(int q_dtype, int kv_dtype, int head_size, int block_size) {
  if (q_dtype != PA_BF16 && q_dtype != PA_F16) return false;
  if (block_size != 16 && block_size != 32 && block_size != 64) return false;
  if (kv_dtype == q_dtype) return head_size == 64 || head_size == 128;
  return (kv_dtype == PA_FP8_E4M3 || kv_dtype == PA_FP8_E5M2) && head_size == 128;
}

cudaError_t launch_diff_prefill(const DiffParams& p, int q_dtype, int kv_dtype, int num_items, int max_ctas,
                                const CUtensorMap* tmap_k, const CUtensorMap* tmap_v, cudaStream_t stream) {
  if (num_items <= 0) return cudaSuccess;
  if (q_dtype == PA_BF16) return launch_query<PA_BF16>(p, kv_dtype, num_items, max_ctas, tmap_k, tmap_v, stream);
  if (q_dtype == PA_F16) return launch_query<PA_F16>(p, kv_dtype, num_items, max_ctas, tmap_k, tmap_v, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
