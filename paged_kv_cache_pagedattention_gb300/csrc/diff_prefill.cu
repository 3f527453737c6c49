// Differential attention of multi-token rows on the 5th-generation tensor cores.
//
// A persistent grid, one CTA per SM; a CTA claims tiles: a work item of the varlen plan (request,
// first query row, partition of the keys) for one (KV group, group of <= 8 heads).  A tile's rows
// are (token, head) pairs, token-major (row = token * GP + head, GP = the head group padded to a
// power of two), 128 to a row tile; row r lives in TMEM lane r.  The value row is twice as wide as
// a key, so a map's accumulators take 2 head_size columns: one row tile with head_size 128, two
// with 64.  Keys stream in chunks of 64 tokens (whole paged blocks), first under map 1, then under
// map 2, as one run of chunks.  Per chunk i, map j:
//   S(i)  = Q_j K_j(i)^T    M = 128 rows, N = 64 keys, K = head_size         -> TMEM
//   P(i)  = softmax numerators of S(i), 16-bit, over S(i)                    -> TMEM
//   O    += P(i) [V_1 V_2](i)   M = 128, N = 2 head_size, K = 64 keys        -> TMEM
// At the end of map 1 its rows A_1 = O / l go to their place in the workspace (fp32); at the end of
// map 2 the same threads take A_1 - lambda A_2, its norm, and write the result.  Rows whose keys lie
// in several partitions leave both maps' partial states instead.
// Warps: eight for the softmax, TMA producers (one for each 128-byte piece of the keys, whose copies
// are small where blocks are: one thread takes some 100 cycles a copy; one for the values), one
// issuer of MMAs a row tile; for FP8 caches one producer and six that widen codes to f16.
//
// The products of a chunk take 768 cycles, a softmax warp some 1,100 from S(i) to P(i).  With one row
// tile, two warps of each scheduler therefore take its chunks in turn (three S buffers), and hand the
// running maximum of a row from one to the other through shared memory; with two row tiles each has
// its own four warps (two S buffers each), and the softmax is what bounds it.  With one row tile the
// queries lie in tensor memory: from shared memory a product of S takes 49 cycles instead of 33 (its
// rows are read 64 columns at a time), and what the ring's copies write there comes on top (1,293
// cycles a chunk, 906 now in blocks of 16 tokens, 835 of 64).
//
// Measured (GB300, 32/8 heads of 128 bf16): 8,192 tokens 605 to 625 us in a graph, 638 to 647 call by call,
// 1,275 to 1,365 TFLOP/s, at the card's power limit (1,370 W, 1,957 MHz); of a tile's time 17 to 24% are the
// two ends of its maps, where the tensor core waits: 128 KB of sums through 32 bytes a cycle.  2 x 1,024
// tokens on 2K and 16K: 1,255 TFLOP/s, on an e4m3 cache 840 (tensor pipe 31%, issue slots 41%; a chunk's
// values are widened for each map), with head_size 64 795 (tensor pipe 38%, issue slots 45%, exponentials
// 25%: no unit's limit, so likely the softmax warps' chain of a chunk, which nothing overlaps).
//
// P is rounded to 16 bits, as in every tile of this kind: an output is then off by 2.6 10^-3 of its
// size where its own bf16 rounding is 1.7 10^-3 (f16: 3.2 10^-4 and 2.1 10^-4).  A second product with
// what P leaves out, as single-token rows have it, would take a chunk from 768 to 1,280 cycles.
#include <algorithm>

#include "diff.cuh"
#include "launch.cuh"
#include "tcgen05.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;      // rows of a row tile = TMEM lanes
constexpr int kChunk = 64;      // keys of a chunk
constexpr int kSoftWarps = 8;   // two warpgroups of softmax warps
constexpr int kValidRing = 16;

template <int HEAD, int BS, bool F8>
struct DiffTc {
  static constexpr int kTiles = HEAD == 128 ? 1 : 2;
  static constexpr bool kTurns = kTiles == 1;                // the two warpgroups take chunks in turn
  static constexpr int kSBufs = kTurns ? 3 : 2;              // S / P buffers of a row tile, 64 TMEM columns each
  static constexpr int kQCol = kSBufs * 64;                  // one row tile: the map's queries, 64 columns
  static constexpr int kOCol = kQCol + (kTurns ? 64 : 0);
  static constexpr int kWide = 2 * HEAD;
  static constexpr int kTileCols = kOCol + kWide;
  static constexpr int kCols = kTurns ? kWide / 2 : kWide;   // columns of O a thread finishes
  static constexpr int kPieces = HEAD / 64;                  // 128-byte pieces of a 16-bit key
  static constexpr int kBlocks = kChunk / BS;
  static constexpr int kPiece = kChunk * 128;
  static constexpr int kKBytes = kPieces * kPiece;           // keys of a chunk
  static constexpr int kVBytes = 2 * kKBytes;                // values of a chunk
  static constexpr int kKStages = F8 ? 3 : HEAD == 128 ? 4 : 5;
  static constexpr int kVStages = F8 ? 3 : HEAD == 128 ? 4 : 5;
  static constexpr int kQPiece = kRows * 128;
  static constexpr int kQTile = kPieces * kQPiece;           // of one map
  static constexpr int kKOff = kTurns ? 0 : kTiles * 2 * kQTile;
  static constexpr int kVOff = kKOff + kKStages * kKBytes;
  // FP8: codes land in staging rings, K [block][token][head_size bytes], V [block][half][token][..]
  static constexpr int kStg = F8 ? 2 : 0;
  static constexpr int kStgBlock = BS * HEAD;
  static constexpr int kStgTensor = kBlocks * kStgBlock;
  static constexpr int kStgKOff = kVOff + kVStages * kVBytes;
  static constexpr int kStgVOff = kStgKOff + kStg * kStgTensor;
  static constexpr int kTurnOff = kStgVOff + kStg * 2 * kStgTensor;  // 2 KB a softmax warp
  static constexpr int kBarOff = kTurnOff + kSoftWarps * 2048;
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 3 * kSBufs * kTiles + kTiles + 3 + 1 + 4 * kStg;
  static constexpr int kSmem = 1024 + kBarOff + 8 * kNumBars + 16;
  static constexpr int kProducers = F8 ? 1 : kPieces + 1;    // FP8: 16 warps leave 128 registers a thread
  static constexpr int kProducer = kSoftWarps, kMma = kProducer + kProducers, kConvK = kMma + kTiles, kConvV = kConvK + 2;
  static constexpr int kThreads = (F8 ? kConvV + 4 : kConvK) * 32;
  static_assert(kBlocks * BS == kChunk, "block size must divide the chunk");
  static_assert(kTiles * kTileCols == 512, "TMEM columns");
  static_assert(kSmem + 7 * 1024 <= 227 * 1024, "shared memory, with the static arrays");
  static_assert(!F8 || HEAD == 128, "FP8 rows are one 128-byte piece");
  static_assert(kSBufs + kKStages + kStg < kValidRing, "a chunk's word outlives its stages");
};

// A block's value tiles of both halves are one copy (the copies' number bounds small blocks: with two
// of them a block of 16 tokens a chunk took 960 cycles, in blocks of 32 800), which lands as [128-byte
// piece][half][token]: so piece pc of a chunk's V is piece pc / 2 of half pc % 2, and that is the order
// of O's columns, 64 to a piece.
__device__ __forceinline__ int value_column(int head, int c) {
  return head == 128 ? ((c >> 6) & 1) * 128 + (c >> 7) * 64 + (c & 63) : c;
}

// Byte offset, inside a chunk's V, of key `key`'s row in piece `pc`.
template <int HEAD, int BS>
__device__ __forceinline__ uint32_t v_row_off(int key, int pc) {
  return (uint32_t)((key / BS) * (HEAD / 32) * BS * 128 + pc * BS * 128 + (key % BS) * 128);
}

// A row of 128 codes widened to f16: two pieces of 128 bytes, piece_stride apart.
template <int KVDT>
__device__ __forceinline__ void widen_row(const uint8_t* srow, uint8_t* drow, int piece_stride, int sw) {
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
}

// A warp's 32 rows between "a row a thread" and memory, where rows are far apart: turned through 2 KB
// of shared memory (16 bytes of a row's 64 at a time, swizzled by row pairs), so that memory is touched
// in whole sectors.  In memory order lane l touches rows 8 k + l / 4, whose addresses it takes once a
// map from the lanes that own them: nullptr where a row is not touched.
__device__ __forceinline__ int turn_at(int row, int q) { return row * 4 + (q ^ ((row >> 1) & 3)); }

template <typename T>
__device__ __forceinline__ void row_addresses(T* mine, bool live, T* (&at)[4]) {
  const int lane = threadIdx.x & 31;
  const unsigned long long x = reinterpret_cast<unsigned long long>(live ? mine : nullptr);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    at[k] = reinterpret_cast<T*>(__shfl_sync(0xffffffffu, x, 8 * k + (lane >> 2)));
}

// 64 bytes a row: 16 floats, or 32 elements of 16 bits.
__device__ __forceinline__ void turn_out(uint4* t, const uint4 (&mine)[4], uint4 (&x)[4]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q) t[turn_at(lane, q)] = mine[q];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = t[turn_at(8 * k + (lane >> 2), lane & 3)];
}

__device__ __forceinline__ void rows_to_memory(uint4* turn, float* const (&at)[4], int col, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 mine[4], x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* f = v + 16 * h + 4 * q;
      mine[q] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    turn_out(turn, mine, x);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at[k]) reinterpret_cast<uint4*>(at[k] + col + 16 * h)[lane & 3] = x[k];
  }
}

// The loads and the turning apart, so that the next columns' loads are on their way meanwhile.
__device__ __forceinline__ void load_rows(const float* const (&at)[4], int col, uint4 (&x)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    x[k] = at[k & 3] ? reinterpret_cast<const uint4*>(at[k & 3] + col + 16 * (k >> 2))[lane & 3] : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void add_rows(uint4* t, const uint4 (&x)[8], float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) t[turn_at(8 * k + (lane >> 2), lane & 3)] = x[4 * h + k];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 y = t[turn_at(lane, q)];
      float* f = v + 16 * h + 4 * q;
      f[0] += __uint_as_float(y.x);
      f[1] += __uint_as_float(y.y);
      f[2] += __uint_as_float(y.z);
      f[3] += __uint_as_float(y.w);
    }
  }
}

template <int QDT>
__device__ __forceinline__ void rows_to_output(uint4* turn, typename Elem<QDT>::T* const (&at)[4], int col,
                                               const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  uint4 mine[4], x[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    mine[q] = make_uint4(pack2<QDT>(v[8 * q], v[8 * q + 1]), pack2<QDT>(v[8 * q + 2], v[8 * q + 3]),
                         pack2<QDT>(v[8 * q + 4], v[8 * q + 5]), pack2<QDT>(v[8 * q + 6], v[8 * q + 7]));
  turn_out(turn, mine, x);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (at[k]) reinterpret_cast<uint4*>(at[k] + col)[lane & 3] = x[k];
}

// A query row as 16-bit words: as it is, or for FP8 caches times 2^shift, so that f16 holds it.
template <int QDT, bool kCvt, int HEAD>
__device__ __forceinline__ int load_query_row(const uint4* src, uint32_t (&w)[HEAD / 2]) {
#pragma unroll
  for (int c = 0; c < HEAD / 8; ++c) {
    const uint4 v = src ? src[c] : make_uint4(0, 0, 0, 0);
    w[4 * c] = v.x;
    w[4 * c + 1] = v.y;
    w[4 * c + 2] = v.z;
    w[4 * c + 3] = v.w;
  }
  if constexpr (!kCvt) return 0;
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < HEAD / 2; ++i) {
    const float2 f = unpack2<QDT>(w[i]);
    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  int ex = 0;
  frexpf(top, &ex);
  const int shift = max(-100, min(100, 15 - ex));
#pragma unroll
  for (int i = 0; i < HEAD / 2; ++i) {
    const float2 f = unpack2<QDT>(w[i]);
    w[i] = pack2<PA_F16>(ldexpf(f.x, shift), ldexpf(f.y, shift));
  }
  return shift;
}

// A row's maximum handed from one warpgroup to the other: posted behind chunk `count` - 1, awaited
// (all lanes of the warp, with a limit) until that chunk's is there.
__device__ __forceinline__ void post(unsigned long long* at, int count, float m) {
  asm volatile("st.volatile.shared.b64 [%0], %1;" ::"r"(smem_u32(at)),
               "l"((unsigned long long)count << 32 | __float_as_uint(m))
               : "memory");
}

__device__ __forceinline__ bool await_post(unsigned long long* at, int count, float& m) {
  uint64_t since = 0;
  for (int spins = 0;; ++spins) {
    unsigned long long w;
    asm volatile("ld.volatile.shared.b64 %0, [%1];" : "=l"(w) : "r"(smem_u32(at)) : "memory");
    m = __uint_as_float(static_cast<unsigned>(w));
    if (__all_sync(0xffffffffu, static_cast<int>(w >> 32) == count || count == 0)) return true;
    if (spins >= 64 && spins % 64 == 0) {
      const uint64_t now = global_timer_ns();
      if (since == 0) since = now;
      if (__any_sync(0xffffffffu, now - since > 2000000000ull)) return false;
    }
  }
}

// Whether three barriers have passed their phases, without waiting.
__device__ __forceinline__ bool mbar_test3(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred x, y, z;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 x, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 y, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 z, [%5], %6;\n\t"
      "and.pred x, x, y;\n\tand.pred x, x, z;\n\t"
      "selp.u32 %0, 1, 0, x;\n\t}"
      : "=r"(all)
      : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb), "r"(smem_u32(c)), "r"(pc)
      : "memory");
  return all != 0;
}

// All 256 softmax threads.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// One request without a plan: whether its starts or lengths are out of range (flagged by one thread).
__device__ __forceinline__ bool alone_rejected(const AttnParams& p, bool flags) {
  const int q0 = p.query_start_loc[0], q_len = p.query_start_loc[1] - q0, seq_len = p.seq_lens[0];
  const bool query = q0 != 0 || q_len != p.num_rows || q_len > p.max_query_len || q_len > seq_len;
  const bool length = seq_len > p.max_seq_len || (long long)seq_len > (long long)p.max_blocks_per_seq * p.block_size;
  if (flags && (query || length)) flag_error(p.err, query ? PA_ERRFLAG_QUERY : PA_ERRFLAG_SEQ_LEN);
  return query || length;
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
  constexpr int KST = G::kKStages, VST = G::kVStages, SG = G::kStg;
  constexpr int NB = G::kBlocks, NT = G::kTiles, SB = G::kSBufs;
  constexpr bool kTurns = G::kTurns;
  const AttnParams& p = args.p.a;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                       // [row tile][map][piece][row][128 bytes]
  uint8_t* sK = smem + G::kKOff;            // [stage][piece][key][128 bytes]
  uint8_t* sV = smem + G::kVOff;            // [stage][block][piece of both halves][token][128 bytes]
  uint8_t* sStgK = smem + G::kStgKOff;
  uint8_t* sStgV = smem + G::kStgVOff;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + G::kBarOff);
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  // Row tile t, buffer b: S(i) is in TMEM (and its chunk's s_valid known), P(i) is, PV(i) is done
  uint64_t* s_full = v_empty + VST;
  uint64_t* p_full = s_full + NT * SB;
  uint64_t* o_done = p_full + NT * SB;
  uint64_t* o_free = o_done + NT * SB;      // a map's O has been read
  uint64_t* v_zeroed = o_free + NT;         // map j's last values have their end zeroed (two row tiles)
  uint64_t* q_full = v_zeroed + 2;          // map 2's queries are in TMEM (one row tile)
  uint64_t* mma_fin = q_full + 1;
  uint64_t* stgk_full = mma_fin + 1;
  uint64_t* stgk_empty = stgk_full + SG;
  uint64_t* stgv_full = stgk_empty + SG;
  uint64_t* stgv_empty = stgv_full + SG;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stgv_empty + SG);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int s_next, s_abort;
  __shared__ int s_valid[kValidRing];       // bit b: block b of the chunk can be read
  __shared__ int s_fail[2];                 // a softmax warp gave up in map j
  __shared__ float s_l[2][2][kRows], s_sq[2][kRows];
  __shared__ float4 s_norm[G::kWide / 4];
  // a row's maximum behind a chunk, with the chunk's number behind it in the upper half: one word, so that
  // it is read as soon as it is there
  __shared__ unsigned long long s_post[2][kRows];
  __shared__ int8_t s_shift[2][NT * kRows];  // FP8 caches: map j's row times 2^shift fits f16

  if (tid == 0) {
    tma_prefetch_desc(&args.tk);
    tma_prefetch_desc(&args.tv);
    for (int i = 0; i < KST; ++i) {
      mbar_init(k_full + i, kCvt ? 64 : G::kPieces);
      mbar_init(k_empty + i, NT);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(v_full + i, kCvt ? 128 : 1);
      mbar_init(v_empty + i, NT);
    }
    for (int i = 0; i < SG; ++i) {
      mbar_init(stgk_full + i, 1);
      mbar_init(stgk_empty + i, 64);
      mbar_init(stgv_full + i, 1);
      mbar_init(stgv_empty + i, 128);
    }
    for (int i = 0; i < NT * SB; ++i) {
      mbar_init(s_full + i, 2);
      mbar_init(p_full + i, kRows);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < NT; ++i) mbar_init(o_free + i, kTurns ? 2 * kRows : kRows);
    mbar_init(v_zeroed, kRows);
    mbar_init(v_zeroed + 1, kRows);
    mbar_init(q_full, kRows);
    mbar_init(mma_fin, NT);
    fence_mbar_init();
    s_abort = s_fail[0] = s_fail[1] = 0;
  }
  if (tid < 2 * kRows) s_post[tid / kRows][tid % kRows] = 0;
  if (warp == G::kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  previous_done();
  if (args.p.norm_weight)
    for (int i = tid; i < G::kWide; i += G::kThreads) reinterpret_cast<float*>(s_norm)[i] = args.p.norm_weight[i];
  const int num_groups = (p.group + 7) / 8;
  const int ny = p.num_kv_heads / 2 * num_groups;
  int gp = 1;
  while (gp < min(p.group, 8)) gp <<= 1;
  const int tile_tokens = kRows / gp;
  // One request of few tiles has no plan: each CTA takes the item of its own number.
  const bool alone = p.work == nullptr;
  const bool rejected = alone ? alone_rejected(p, blockIdx.x == 0 && tid == 0) : plan_rejected(p);
  int nwork = 0, nfull = 0, alone_parts = 1;
  if (!rejected) {
    if (alone) {
      const int q_len = p.num_rows, origin = window_origin(p, p.seq_lens[0], q_len);
      alone_parts = (p.seq_lens[0] - origin + p.part_pf - 1) / p.part_pf;
      nwork = (q_len + NT * tile_tokens - 1) / (NT * tile_tokens) * alone_parts;
    } else {
      nwork = *p.work_count;
      nfull = *p.work_full;
    }
  }
  const int total = nwork * ny, total_full = nfull * ny;
  if (tid == 0) s_next = alone ? blockIdx.x : rejected ? 0 : atomicAdd(p.work_claim, 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int L = s_next;
  int gch = 0;       // ring chunks of earlier tiles: a chunk's place in the K and V rings
  int tch[NT] = {};  // a row tile's chunks of earlier tiles
  int maps_done = 0; // maps of earlier tiles: o_free's phases
  int tails = 0;     // earlier tiles with a tail chunk: v_zeroed's
  int turns = 0;     // earlier tiles with chunks: q_full's
  int k_issued = 0, v_issued = 0;
  while (L < total) {
    const int lc = L < total_full ? L : L - total_full;
    const int nc = L < total_full ? nfull : nwork - nfull;
    // The list's last tiles run from a request's first rows to its last, whose keys are the most: they
    // are claimed from the end on, all KV groups of a tile together, so that the short ones fill the
    // tail.  Whole partitions are alike, and stay in their order.
    const int at = lc / ny, y = lc % ny, x = L < total_full ? at : nfull + nc - 1 - at;
    const int4 item = alone ? make_int4(0, x / alone_parts * NT * tile_tokens, x % alone_parts, 0) : p.work[x];
    const int r = item.x, row0 = item.y, z = item.z;
    const int g = y / num_groups, hg = y % num_groups, kvh = 2 * g;
    const int h0 = g * p.group + hg * 8;
    const int nh = min(8, p.group - hg * 8);
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
    if (alone && p.causal && k0 >= pos0 + ntok) {  // behind the last key that this tile attends
      L += gridDim.x;
      continue;
    }
    const int klo = p.window > 0 ? max(k0, max(0, pos0 - p.window + 1) / BS * BS) : k0;
    auto tile_chunks = [&](int t) {
      const int nt = min(ntok, (t + 1) * tile_tokens) - t * tile_tokens;
      if (nt <= 0) return 0;
      const int k1t = min(k0 + part, p.causal ? pos0 + t * tile_tokens + nt : seq_len);
      return k1t > klo ? (k1t - klo + kChunk - 1) / kChunk : 0;
    };
    int nch_t[NT];  // a row tile's chunks under one map
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

    // Softmax warpgroup w, thread = row.  One row tile: w loads map w's queries; two: w's own rows, both maps
    const int wg = warp >> 2, row = tid % kRows;
    const int tile_row = kTurns ? row : wg * kRows + row;
    const int row_tok = tile_row / gp, row_head = tile_row % gp;
    const bool row_valid = warp < kSoftWarps && row_tok < ntok && row_head < nh;
    const int row_pos = pos0 + row_tok;
    // map j's queries of this thread's row, to TMEM (one row tile) or to shared memory
    const int last_ci = tch[0] + nch_t[0] - 1;  // map 1's last chunk
    auto load_queries = [&](int mp) {
      const uint4* src = row_valid ? reinterpret_cast<const uint4*>(
                                         static_cast<const typename QE::T*>(p.q) +
                                         ((long long)(row0 + row_tok) * p.num_q_heads + 2 * (h0 + row_head) + mp) * HEAD)
                                   : nullptr;
      uint32_t w[HEAD / 2];
      const int shift = load_query_row<QDT, kCvt, HEAD>(src, w);
      if constexpr (kCvt) s_shift[mp][tile_row] = static_cast<int8_t>(shift);
      if constexpr (kTurns) {
        // before map 2's are stored, map 1's products are done with theirs
        if (mp == 1 && !mbar_wait_bounded(s_full + last_ci % SB, (last_ci / SB) & 1)) return false;
        tc_fence_after();
        const uint32_t at = tmem + G::kQCol + ((uint32_t)((warp & 3) * 32) << 16);
        tmem_st32(at, w);
        tmem_st32(at + 32, w + 32);
        tmem_wait_st();
      } else {
        uint8_t* dst = sQ + (wg * 2 + mp) * G::kQTile;
#pragma unroll
        for (int c = 0; c < HEAD / 8; ++c)
          *reinterpret_cast<uint4*>(dst + (c >> 3) * G::kQPiece + swz128(row, c & 7)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      }
      return true;
    };
    if (kTurns ? warp < 4 : warp < kSoftWarps) {
      load_queries(0);
      if constexpr (!kTurns) {
        load_queries(1);
        fence_proxy_async();
      }
    }
    tc_fence_before();
    __syncthreads();  // the queries are in place; every role of the previous tile is done
    tc_fence_after();
    const int32_t* table = p.block_tables + (long long)r * p.max_blocks_per_seq;

    if (warp >= G::kProducer && warp < G::kMma) {
      // ------------------------------------------------------------ TMA producers
      const int piece = warp - G::kProducer;  // of the keys
      const bool does_v = kCvt || warp == G::kMma - 1, does_k = kCvt || !does_v;
      const int kb_end = (k1 + BS - 1) / BS;
      auto load_window = [&](int w) {
        const int kb = kb_first + 32 * w + lane;
        return kb < kb_end ? table[kb] : -1;
      };
      bool ok = true;
      // stage gi of a ring is free: its last reader is done
      auto free_stage = [&](uint64_t* empty, int stages, int gi) {
        return gi < stages || __all_sync(0xffffffffu, mbar_wait_bounded(empty + gi % stages, ((gi / stages) - 1) & 1));
      };
      for (int mp = 0; ok && mp < 2; ++mp) {
        int cur_w = 0;
        int win = load_window(0);
        int win_next = load_window(1);
        for (int i = 0; i < nch; ++i) {
          const int gi = gch + mp * nch + i;
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
            if (in_range && !ok_b && lane == 0 && piece == 0) flag_error(p.err, PA_ERRFLAG_BLOCK_TABLE);
            phys[b] = in_range && ok_b ? e : p.num_blocks;
            valid |= (ok_b || !in_range) << b;
          }
          if (does_k) {
            constexpr int RS = kCvt ? SG : KST;
            uint64_t* full = (kCvt ? stgk_full : k_full) + gi % RS;
            if (!(ok = free_stage(kCvt ? stgk_empty : k_empty, RS, gi))) break;
            if (elect_one()) {
              if (piece == 0) s_valid[gi % kValidRing] = valid;
              mbar_arrive_expect_tx(full, kCvt ? G::kStgTensor : G::kPiece);
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                if constexpr (kCvt) {
                  tma_load_4d(sStgK + gi % RS * G::kStgTensor + b * G::kStgBlock, &args.tk, 0, (kvh + mp) * BS, 0, phys[b],
                              full);
                } else {
                  tma_load_4d(sK + gi % RS * G::kKBytes + piece * G::kPiece + b * BS * 128, &args.tk, 0, (kvh + mp) * BS,
                              piece, phys[b], full);
                }
              }
            }
            __syncwarp();
            k_issued = gi + 1;
          }
          if (does_v) {
            constexpr int RS = kCvt ? SG : VST;
            uint64_t* full = (kCvt ? stgv_full : v_full) + gi % RS;
            if (!(ok = free_stage(kCvt ? stgv_empty : v_empty, RS, gi))) break;
            if (elect_one()) {
              mbar_arrive_expect_tx(full, kCvt ? 2 * G::kStgTensor : G::kVBytes);
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                uint8_t* d = kCvt ? sStgV + gi % RS * 2 * G::kStgTensor + b * 2 * G::kStgBlock
                                  : sV + gi % RS * G::kVBytes + v_row_off<HEAD, BS>(b * BS, 0);
                tma_load_4d(d, &args.tv, 0, kvh * BS, 0, phys[b], full);
              }
            }
            __syncwarp();
            v_issued = gi + 1;
          }
        }
      }
      if (!ok) {
        if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
        s_abort = 1;
      }
    } else if (kCvt && warp >= G::kConvK) {
      // ------------------------------------------------------------ FP8 converters: a row a thread
      if constexpr (kCvt) {
        const bool is_v = warp >= G::kConvV;
        const int ct = tid - (is_v ? G::kConvV : G::kConvK) * 32;
        const int half = ct / kChunk, key = ct % kChunk, blk = key / BS, tok = key % BS;
        uint64_t* sf = is_v ? stgv_full : stgk_full;
        uint64_t* se = is_v ? stgv_empty : stgk_empty;
        uint64_t* df = is_v ? v_full : k_full;
        uint64_t* de = is_v ? v_empty : k_empty;
        const int DST = is_v ? VST : KST;
        for (int i = 0; i < 2 * nch; ++i) {
          const int gi = gch + i, s = gi % DST, ss = gi % SG;
          bool ok = mbar_wait_bounded(sf + ss, (gi / SG) & 1);
          if (gi >= DST) ok = ok && mbar_wait_bounded(de + s, ((gi / DST) - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
            s_abort = 1;
            break;
          }
          if (is_v)
            widen_row<KVDT>(sStgV + ss * 2 * G::kStgTensor + (blk * 2 + half) * G::kStgBlock + tok * 128,
                            sV + s * G::kVBytes + v_row_off<HEAD, BS>(key, half), 2 * BS * 128, key & 7);
          else
            widen_row<KVDT>(sStgK + ss * G::kStgTensor + blk * G::kStgBlock + tok * 128, sK + s * G::kKBytes + key * 128,
                            G::kPiece, key & 7);
          fence_proxy_async();
          mbar_arrive(se + ss);
          mbar_arrive(df + s);
        }
      }
    } else if (warp >= G::kMma && warp < G::kConvK) {
      // ------------------------------------------------------------ MMA issuers, one thread a row tile
      // As soon as P(i) is written PV(i), then S(i + SB) into the buffer that PV(i) frees: a thread's
      // MMAs run in the order of their issue.
      const int t = NT == 1 ? 0 : warp - G::kMma;
      const int my_nch = t == 0 ? nch_t[0] : nch_t[NT - 1];
      const int tc = t == 0 ? tch[0] : tch[NT - 1];
      const uint32_t fmt = ODT == PA_BF16 ? 1u : 0u;
      const uint32_t id_s = umma_idesc(kRows, kChunk, fmt, 0);
      const uint32_t id_o = umma_idesc(kRows, G::kWide, fmt, 1);
      const uint64_t kd0 = umma_desc(smem_u32(sK), 16, 1024);
      const uint64_t vd0 = umma_desc(smem_u32(sV), BS * 128, 1024);
      const uint32_t tT = tmem + t * G::kTileCols;
      uint64_t* my_s_full = s_full + t * SB;
      uint64_t* my_p_full = p_full + t * SB;
      if (elect_one()) {
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = mbar_wait_bounded(bar, parity); };
        // chunks of a ring that this row tile does not read are released once they have landed
        auto skip = [&](uint64_t* full, uint64_t* empty, int stages, int gi) {
          if (wait(full + gi % stages, (gi / stages) & 1)) mbar_arrive(empty + gi % stages);
        };
        for (int mp = 0; ok && mp < 2; ++mp) {
          const int g0 = gch + mp * nch, c0 = tc + mp * my_nch;
          // chunk i's S behind its keys
          auto wait_k = [&](int i) { return wait(k_full + (g0 + i) % KST, ((g0 + i) / KST) & 1); };
          auto issue_s = [&](int i) {
            const int gi = g0 + i, buf = (c0 + i) % SB;
            const uint64_t kd = kd0 + (uint64_t)((gi % KST) * G::kKBytes >> 4);
            const uint64_t qd = umma_desc(smem_u32(sQ) + (t * 2 + mp) * G::kQTile, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < HEAD / 16; ++ks) {
              const uint32_t ko = ((ks >> 2) * G::kPiece + (ks & 3) * 32) >> 4;
              if constexpr (kTurns)
                umma_tmem_a(tT + buf * 64, tmem + G::kQCol + ks * 8, kd + ko, id_s, ks > 0 ? 1u : 0u);
              else
                umma(tT + buf * 64, qd + (((ks >> 2) * G::kQPiece + (ks & 3) * 32) >> 4), kd + ko, id_s, ks > 0 ? 1u : 0u);
            }
            umma_commit(my_s_full + buf);
            umma_commit(k_empty + gi % KST);
            mbar_arrive(my_s_full + buf);  // passes on what k_full brought: the chunk's s_valid
          };
          if (kTurns && mp == 1 && my_nch > 0 && !wait(q_full, turns & 1)) break;
          for (int i = 0; i < SB && i < my_nch && wait_k(i); ++i) {
            tc_fence_after();
            issue_s(i);
          }
          // The tensor core's queue is short: a wait hides behind the long products of PV(i), not behind
          // the short ones of S.  So the next chunk's waits come between the two; the one for P(i + 1)
          // too where S runs far enough ahead of it (one row tile).
          auto ready = [&](int i) {
            const int gi = g0 + i;
            // the last chunk's V is read only after the row tile that zeroes its end has done so
            if (NT > 1 && tail_chunk && i == nch - 1 && t != zero_tile && !wait(v_zeroed + mp, tails & 1)) return false;
            return wait(v_full + gi % VST, (gi / VST) & 1);
          };
          auto wait_p = [&](int i) { return wait(my_p_full + (c0 + i) % SB, ((c0 + i) / SB) & 1); };
          // a map's first product overwrites O, which the map before it must have been read from
          if (ok && my_nch > 0 && maps_done + mp > 0) wait(o_free + t, (maps_done + mp - 1) & 1);
          ok = ok && (my_nch == 0 || (ready(0) && wait_p(0)));
          for (int i = 0; ok && i < my_nch; ++i) {
            const int gi = g0 + i, buf = (c0 + i) % SB;
            tc_fence_after();
            const uint64_t vd = vd0 + (uint64_t)((gi % VST) * G::kVBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < kChunk / 16; ++ks)
              umma_tmem_a(tT + G::kOCol, tT + buf * 64 + ks * 8, vd + (uint64_t)(v_row_off<HEAD, BS>(16 * ks, 0) >> 4),
                          id_o, (i > 0 || ks > 0) ? 1u : 0u);
            umma_commit(o_done + t * SB + buf);
            umma_commit(v_empty + gi % VST);
            const bool more = i + 1 < my_nch;
            if constexpr (kTurns) {
              // all three looked at together: one trip to shared memory where they are there
              if (i + SB < my_nch) {
                const int gv = gi + 1, gk = gi + SB, cp = c0 + i + 1;
                if (!mbar_test3(v_full + gv % VST, (gv / VST) & 1, k_full + gk % KST, (gk / KST) & 1,
                                my_p_full + cp % SB, (cp / SB) & 1) &&
                    !(ready(i + 1) && wait_k(i + SB) && wait_p(i + 1)))
                  break;
              } else if (more && !(ready(i + 1) && wait_p(i + 1))) {
                break;
              }
            } else {
              if (more && !ready(i + 1)) break;
              if (i + SB < my_nch && !wait_k(i + SB)) break;
            }
            tc_fence_after();
            if (i + SB < my_nch) issue_s(i + SB);
            if (!kTurns && more && !wait_p(i + 1)) break;
          }
          for (int i = my_nch; NT > 1 && ok && i < nch; ++i) {
            skip(k_full, k_empty, KST, g0 + i);
            if (ok) skip(v_full, v_empty, VST, g0 + i);
          }
        }
        if (!ok) {
          flag_error(p.err, PA_ERRFLAG_TIMEOUT);
          s_abort = 1;
        }
      }
      __syncwarp();
    } else if (warp < kSoftWarps) {
      // ------------------------------------------------------------ softmax: a row a thread
      const int t = kTurns ? 0 : wg;
      const int my_nch = t == 0 ? nch_t[0] : nch_t[NT - 1];
      const int tc = t == 0 ? tch[0] : tch[NT - 1];
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tT = tmem + t * G::kTileCols;
      const uint32_t tO = tT + G::kOCol + (kTurns ? wg * G::kCols : 0);  // this thread's columns of O
      uint64_t* my_s_full = s_full + t * SB;
      uint64_t* my_p_full = p_full + t * SB;
      uint64_t* my_o_done = o_done + t * SB;
      const int row_limit = p.causal ? min(k1, row_pos + 1) : k1;
      const int row_lo = p.window > 0 ? max(0, row_pos - p.window + 1) : 0;
      const int kv_len = p.causal ? row_pos + 1 : seq_len;
      const int parts_row = (kv_len - origin + part - 1) / part;
      const bool write = row_valid && z < parts_row;
      const bool direct = parts_row == 1;
      const int head = h0 + row_head;
      const long long pi = (alone ? (long long)(t0 + row_tok) * p.max_partitions
                                  : (long long)p.part_off[r] + (long long)(t0 + row_tok) * parts_req) + z;
      const int col0 = kTurns ? wg * G::kCols : 0;
      uint4* turn = reinterpret_cast<uint4*>(smem + G::kTurnOff + warp * 2048);
      const float lam = write && direct ? diff_lambda(args.p, qs + t0 + row_tok, head) : 0.f;
      bool fail = false;
#pragma unroll 1
      for (int mp = 0; !fail && mp < 2; ++mp) {
        const float unit = kCvt ? p.scale * kLog2e * p.k_scale[(kvh + mp) * p.scale_stride] : p.scale * kLog2e;
        float m = -INFINITY, l = 0.f;  // m: the row's maximum when this thread last saw it
#pragma unroll 1
        for (int i = 0; i < my_nch; ++i) {
          const int ci = tc + mp * my_nch + i, buf = ci % SB;
          if (kTurns && (ci & 1) != wg) continue;
          const int gi = gch + mp * nch + i;
          const int base = klo + i * kChunk;
          const uint32_t tS = tT + buf * 64;
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(my_s_full + buf, (ci / SB) & 1))) {
            fail = true;
            break;
          }
          tc_fence_after();
          uint32_t sr[kChunk];
          tmem_ld32(tS + lane_base, sr);
          tmem_ld32(tS + 32 + lane_base, sr + 32);
          const int valid = s_valid[gi % kValidRing];
          const float c = kCvt ? ldexpf(unit, -s_shift[mp][tile_row]) : unit;
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
          float m_prev = m;  // the row's maximum before this chunk
          if constexpr (kTurns) {
            // the other warpgroup posted it with the chunk before
            if (!await_post(&s_post[wg ^ 1][row], ci, m_prev)) {
              fail = true;
              break;
            }
            if (i == 0) m_prev = -INFINITY;
          }
          const bool need = mx > m_prev + kRescaleSlack;
          const float nm = need ? fmaxf(m_prev, mx) : m_prev;
          if constexpr (kTurns) {
            post(&s_post[wg][row], ci + 1, nm);
          }
          if (nm != m) {
            l *= ex2_approx(m - nm);  // 0 while this thread's sum is
            m = nm;
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
          tmem_st32(tS + lane_base, pk);  // P(i) over the first half of S(i)'s columns
          // O is rescaled only once PV(i - 1) has completed
          if (__any_sync(0xffffffffu, need) && i > 0) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(my_o_done + (ci - 1) % SB, ((ci - 1) / SB) & 1))) {
              fail = true;
              break;
            }
            tc_fence_after();
            const float al = need ? ex2_approx(m_prev - nm) : 1.f;
#pragma unroll 1
            for (int cb = 0; cb < G::kWide; cb += 32) {
              uint32_t o[32];
              tmem_ld32(tT + G::kOCol + cb + lane_base, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
              tmem_st32(tT + G::kOCol + cb + lane_base, o);
            }
          }
          // V rows past the sequence may hold any bits: zeroed, to keep 0 * V finite
          if (tail_chunk && t == zero_tile && i == nch - 1) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(v_full + gi % VST, (gi / VST) & 1))) {
              fail = true;
              break;
            }
            const int vrem = kv_loaded_end - base;
            for (int q = row; q < 2 * G::kPieces * kChunk; q += kRows) {
              const int key = q % kChunk;
              if (key < vrem) continue;
              uint4* d = reinterpret_cast<uint4*>(sV + (gi % VST) * G::kVBytes + v_row_off<HEAD, BS>(key, q / kChunk));
#pragma unroll
              for (int e = 0; e < 8; ++e) d[e] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            if (NT > 1) mbar_arrive(v_zeroed + mp);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(my_p_full + buf);
        }
        const int cl = tc + (mp + 1) * my_nch - 1;  // the map's last chunk
        // map 2's queries: by the warpgroup that is done with map 1's chunks first
        if (kTurns && !fail && mp == 0 && my_nch > 0 && (cl & 1) != wg) {
          fail = !__all_sync(0xffffffffu, load_queries(1));
          tc_fence_before();
          if (!fail) mbar_arrive(q_full);
        }
        // ---- the map's end.  Where the rows go, and map 1's result for those that end here, are fetched
        // while the last products run: fp32 rows go to the workspace, map 1's of rows that end here come
        // from there
        const long long at = pi * p.num_q_heads + 2 * head + mp;
        float* ws = p.ws_acc + at * G::kWide;
        typename QE::T* out = static_cast<typename QE::T*>(p.out) +
                              ((long long)(qs + t0 + row_tok) * (p.num_q_heads / 2) + head) * G::kWide;
        const bool norm = mp == 1 && args.p.norm_weight != nullptr;
        float* to[4];
        const float* from[4];
        typename QE::T* out_at[4];
        const bool any_to = __any_sync(0xffffffffu, write && (mp == 0 || !direct));
        const bool any_from = mp == 1 && __any_sync(0xffffffffu, write && direct);
        row_addresses(ws, write && (mp == 0 || !direct), to);
        row_addresses(static_cast<const float*>(ws - G::kWide), mp == 1 && write && direct, from);
        row_addresses(out, write && direct, out_at);
        uint4 next[8];
        if (any_from) load_rows(from, value_column(HEAD, col0), next);
        // O is complete, the row's maximum and sum are joined
        if (!fail && my_nch > 0) {
          fail = !__all_sync(0xffffffffu, mbar_wait_bounded(my_o_done + cl % SB, (cl / SB) & 1));
          tc_fence_after();
        }
        if constexpr (kTurns) {
          if (!fail && my_nch > 0) {
            float last = m;
            fail = !await_post(&s_post[cl & 1][row], cl + 1, last);
            if (last != m) {
              l *= ex2_approx(m - last);
              m = last;
            }
          }
          s_l[mp][wg][row] = l;
          if (fail) s_fail[mp] = 1;
          softmax_sync();
          fail = s_fail[mp] != 0;  // all or none go on: there is another such meeting below
          l = s_l[mp][0][row] + s_l[mp][1][row];
        }
        if (fail) break;
        float weight = diff_weight(l);
        if (mp == 1) weight *= -lam;
        float sq = 0.f;
#pragma unroll 1
        for (int cb = 0; cb < G::kCols; cb += 32) {
          const int col = value_column(HEAD, col0 + cb);
          const float vs = kCvt ? p.v_scale[(kvh + col / HEAD) * p.scale_stride] : 1.f;
          const float f = direct ? vs * weight : vs;
          uint32_t o[32];
          if (my_nch > 0) {
            tmem_ld32(tO + cb + lane_base, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
          }
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]) * f;
          if (any_from) {
            add_rows(turn, next, v);
            if (cb + 32 < G::kCols) load_rows(from, value_column(HEAD, col0 + cb + 32), next);
          }
          if (norm && any_from) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              sq = fmaf(v[j], v[j], sq);
              o[j] = __float_as_uint(v[j]);
            }
            tmem_st32(tO + cb + lane_base, o);  // kept for the second look
          }
          if (any_to) rows_to_memory(turn, to, col, v);
          if (any_from && !norm) rows_to_output<QDT>(turn, out_at, col, v);
        }
        if (write && !direct && (!kTurns || wg == 0)) p.ws_ml[at] = make_float2(m, l);
        if (norm) {
          if constexpr (kTurns) {
            s_sq[wg][row] = sq;
            softmax_sync();
            sq = s_sq[0][row] + s_sq[1][row];
          }
          const float rn = rsqrtf(sq / G::kWide + args.p.norm_eps);
          tmem_wait_st();
#pragma unroll 1
          for (int cb = 0; any_from && cb < G::kCols; cb += 32) {
            const int col = value_column(HEAD, col0 + cb);
            uint32_t o[32];
            tmem_ld32(tO + cb + lane_base, o);
            tmem_wait_ld();
            float v[32];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 w = s_norm[col / 4 + q];
              v[4 * q] = __uint_as_float(o[4 * q]) * (rn * w.x);
              v[4 * q + 1] = __uint_as_float(o[4 * q + 1]) * (rn * w.y);
              v[4 * q + 2] = __uint_as_float(o[4 * q + 2]) * (rn * w.z);
              v[4 * q + 3] = __uint_as_float(o[4 * q + 3]) * (rn * w.w);
            }
            rows_to_output<QDT>(turn, out_at, col, v);
          }
        }
        tc_fence_before();
        mbar_arrive(o_free + t);
      }
      if (fail) {
        if (lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
        s_abort = 1;
      }
    }

    gch += 2 * nch;
    maps_done += 2;
    tails += tail_chunk;
    turns += nch > 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) tch[t] += 2 * nch_t[t];
    if (tid == 0 && !alone) s_next = atomicAdd(p.work_claim, 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    L = alone ? L + gridDim.x : s_next;
    if (s_abort) break;
  }

  next_may_start();
  // ---- every MMA completes and every copy lands before TMEM is released and the CTA leaves
  if (warp >= G::kMma && warp < G::kConvK) {
    if (elect_one()) umma_commit(mma_fin);
    __syncwarp();
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(mma_fin, 0)) && lane == 0) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
  } else if (warp >= G::kProducer && warp < G::kMma && lane == 0) {
    constexpr int KR = kCvt ? SG : KST, VR = kCvt ? SG : VST;
    bool ok = true;
    for (int j = max(0, k_issued - KR); j < k_issued; ++j)
      ok = mbar_wait_bounded((kCvt ? stgk_full : k_full) + j % KR, (j / KR) & 1) && ok;
    for (int j = max(0, v_issued - VR); j < v_issued; ++j)
      ok = mbar_wait_bounded((kCvt ? stgv_full : v_full) + j % VR, (j / VR) & 1) && ok;
    if (!ok) flag_error(p.err, PA_ERRFLAG_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == G::kMma) {
    tc_fence_after();
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
  const long long tiles = (long long)num_items * (p.a.num_kv_heads / 2) * ((p.a.group + 7) / 8);
  const int grid = static_cast<int>(std::min<long long>(tiles, std::max(1, max_ctas)));
  DiffPrefillArgs args;
  args.p = p;
  args.tk = *tk;
  args.tv = *tv;
  return launch_early<DiffPrefillArgs>(kern, dim3(grid), G::kThreads, G::kSmem, 1, args, stream);
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
