// Rotary positions written with the cache: the new tokens' q and k rows are rotated by
// their positions' angles, q into a buffer of its own, k (with v) into the token's slot.
//
//   angle of pair i at position p: p * f_i, f_i = inv_freq[i]; c, s = attn_factor * (cos, sin)
//   (x, y) -> (x c - y s, y c + x s), pairs (i, i + R/2) or (2i, 2i + 1), i < R/2
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: f_i / 2 pi is rounded
// once (fp64, 53 bits), and p times it modulo 2^64 drops whole turns exactly, so far
// positions lose nothing to a range reduction (fp32 angles at position 262,144 would be
// off by up to 2^-7 rad).  The rotation runs in fp32 and is rounded or quantised once.
#include "launch.cuh"
#include "pa_common.cuh"
#include "quantize.cuh"

namespace pa {

namespace {

// f / 2 pi modulo one turn, as a 64-bit fraction.
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  const double t = static_cast<double>(f) * 0.15915494309189533577;
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of pos * turn, times m.  The nearest quarter turn comes off as an integer;
// what is left is at most an eighth of a turn, exact to 2^-32 before it is converted.
__device__ __forceinline__ float2 rotation(int pos, unsigned long long turn, float m) {
  const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(pos)) * turn;
  const unsigned hi = static_cast<unsigned>(phase >> 32);
  const unsigned quarter = (hi + 0x20000000u) >> 30;
  const int rest = static_cast<int>(hi - (quarter << 30));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c * m, s * m);
}

// Element j of a row after rotation, its partner read from the row.
template <int SRC>
__device__ __forceinline__ float rotated_at(const RotaryParams& p, const typename Elem<SRC>::T* row, int j, int pos) {
  const float x = Elem<SRC>::load(row + j);
  if (j >= p.rotary_dim) return x;
  const int half = p.rotary_dim / 2;
  int i, partner;
  bool first;
  if (p.interleaved) {
    i = j >> 1;
    first = (j & 1) == 0;
    partner = j ^ 1;
  } else {
    first = j < half;
    i = first ? j : j - half;
    partner = first ? j + half : j - half;
  }
  const float2 cs = rotation(pos, turn_fraction(p.inv_freq[i]), p.attn_factor);
  const float y = Elem<SRC>::load(row + partner);
  return first ? x * cs.x - y * cs.y : x * cs.x + y * cs.y;
}

// Any even rotary size, stride and element alignment: a thread handles four pairs (or
// eight elements behind the rotated ones) of a q row, or one group of a k or v row that
// makes 16 bytes of cache (8 bytes of code and a block scale in NVFP4).  q is handled by
// whole pairs, so it may be rotated in place.
template <int SRC, int CDT>
__global__ void __launch_bounds__(256) rotary_generic_kernel(const RotaryParams p) {
  using SE = Elem<SRC>;
  using T = typename SE::T;
  constexpr bool kCopy = SRC == CDT;
  constexpr int kGroup = kCopy ? 16 / SE::bytes : 16;
  const int d = p.head_size, half = p.rotary_dim / 2;
  const int pair_units = (half + 3) / 4, rest_units = (d - p.rotary_dim + 7) / 8;
  const int q_row = pair_units + rest_units;
  const long long q_units = (long long)p.num_q_heads * q_row;
  const int groups = d / kGroup;
  const long long kv_units = (long long)p.num_kv_heads * groups;
  const long long per_token = q_units + 2 * kv_units;
  const long long total = per_token * p.num_tokens;
  const long long limit = (long long)p.num_blocks * p.block_size;
  previous_done();
  for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < total;
       u += (long long)gridDim.x * blockDim.x) {
    const long long t = u / per_token;
    long long rem = u - t * per_token;
    const long long slot = p.slot_mapping[t];
    if (slot < 0) continue;
    if (slot >= limit) {
      flag_error(p.err, PA_ERRFLAG_SLOT);
      continue;
    }
    const int pos = p.positions[t];
    if (rem < q_units) {
      const int h = static_cast<int>(rem / q_row), c = static_cast<int>(rem % q_row);
      const T* src = static_cast<const T*>(p.q) + t * p.q_stride + (long long)h * d;
      T* dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + (long long)h * d;
      if (c < pair_units) {
        for (int i = 4 * c; i < min(half, 4 * c + 4); ++i) {
          const int a = p.interleaved ? 2 * i : i, b = p.interleaved ? 2 * i + 1 : i + half;
          const float2 cs = rotation(pos, turn_fraction(p.inv_freq[i]), p.attn_factor);
          const float x = SE::load(src + a), y = SE::load(src + b);
          dst[a] = SE::from_float(x * cs.x - y * cs.y);
          dst[b] = SE::from_float(y * cs.x + x * cs.y);
        }
      } else {
        const int j0 = p.rotary_dim + 8 * (c - pair_units);
        for (int j = j0; j < min(d, j0 + 8); ++j) dst[j] = src[j];
      }
      continue;
    }
    rem -= q_units;
    const bool is_v = rem >= kv_units;
    if (is_v) rem -= kv_units;
    const int h = static_cast<int>(rem / groups), j0 = static_cast<int>(rem % groups) * kGroup;
    const T* src = is_v ? static_cast<const T*>(p.value) + t * p.value_stride + (long long)h * d
                        : static_cast<const T*>(p.key) + t * p.key_stride + (long long)h * d;
    void* cache = is_v ? p.v_cache : p.k_cache;
    const long long blk = slot / p.block_size;
    const int off = static_cast<int>(slot % p.block_size);
    const long long tile = blk * p.num_kv_heads + h;
    if constexpr (kCopy) {
      T* dst = static_cast<T*>(cache) + (tile * p.block_size + off) * d + j0;
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        dst[i] = is_v || j0 + i >= p.rotary_dim ? src[j0 + i] : SE::from_float(rotated_at<SRC>(p, src, j0 + i, pos));
    } else {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = is_v ? SE::load(src + j0 + i) : rotated_at<SRC>(p, src, j0 + i, pos);
      const float scale = (is_v ? p.v_scale : p.k_scale)[h * p.scale_stride];
      if constexpr (CDT == PA_NVFP4) {
        uint2 codes;
        uint8_t block_scale;
        quant_nvfp4(x, scale, codes, block_scale);
        uint8_t* dst = static_cast<uint8_t*>(cache) + tile * nvfp4_tile_bytes(p.block_size, d);
        *reinterpret_cast<uint2*>(dst + (long long)off * (d / 2) + j0 / 2) = codes;
        dst[(long long)p.block_size * (d / 2) + (long long)off * (d / 16) + j0 / 16] = block_scale;
      } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4] |= static_cast<uint32_t>(quant_fp8<CDT>(x[i], scale)) << (8 * (i % 4));
        uint8_t* dst = static_cast<uint8_t*>(cache) + (tile * p.block_size + off) * d + j0;
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// ---------------------------------------------------------------- whole 16-byte pieces

template <int DT>
struct Piece {  // 16 bytes of elements as fp32
  static constexpr int n = 16 / Elem<DT>::bytes;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == PA_F32) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2<DT>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == PA_F32) w[i] = __float_as_uint(x[i]);
      else w[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Elements of a k or v row that one thread stores: one piece, 8 FP8 codes, or a group of 16
// NVFP4 codes.  (A division an element makes the codes dear: with 16 FP8 codes a thread, 96 of
// 256 threads had twice the work.)
template <int SRC, int CDT>
constexpr int kv_unit() { return SRC == CDT ? Piece<SRC>::n : CDT == PA_NVFP4 ? 16 : 8; }

// Store kv_unit elements x of row (tile, off) at element j of a cache.
template <int SRC, int CDT>
__device__ __forceinline__ void store_unit(const RotaryParams& p, void* cache, long long tile, int off, int j,
                                           const float (&x)[kv_unit<SRC, CDT>()], float scale) {
  const int d = p.head_size;
  if constexpr (SRC == CDT) {
    typename Elem<SRC>::T* dst = static_cast<typename Elem<SRC>::T*>(cache) + (tile * p.block_size + off) * d + j;
    *reinterpret_cast<uint4*>(dst) = Piece<SRC>::pack(x);
  } else if constexpr (CDT == PA_NVFP4) {
    uint2 codes;
    uint8_t block_scale;
    quant_nvfp4(x, scale, codes, block_scale);
    uint8_t* dst = static_cast<uint8_t*>(cache) + tile * nvfp4_tile_bytes(p.block_size, d);
    *reinterpret_cast<uint2*>(dst + (long long)off * (d / 2) + j / 2) = codes;
    dst[(long long)p.block_size * (d / 2) + (long long)off * (d / 16) + j / 16] = block_scale;
  } else {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      w[i / 4] |= static_cast<uint32_t>(quant_fp8x2<CDT>(x[i], x[i + 1], scale)) << (8 * (i % 4));
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + (tile * p.block_size + off) * d + j) =
        make_uint2(w[0], w[1]);
  }
}

// N elements of a row in whole pieces: loaded, and as fp32.
template <int SRC, int N>
struct Unit {
  static constexpr int kPieces = N / Piece<SRC>::n;
  uint4 raw[kPieces];
  __device__ __forceinline__ void load(const typename Elem<SRC>::T* src) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) raw[i] = reinterpret_cast<const uint4*>(src)[i];
  }
  __device__ __forceinline__ void values(float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) Piece<SRC>::unpack(raw[i], x + i * Piece<SRC>::n);
  }
};

__device__ __forceinline__ void rotate(float& x, float& y, float2 cs) {
  const float a = x, b = y;
  x = a * cs.x - b * cs.y;
  y = b * cs.x + a * cs.y;
}

// The rotations of a token lie in shared memory by the pair's place in its piece, then by
// the piece: threads of a warp take neighbouring pieces, so they read neighbouring words.
template <int kPairs>
__device__ __forceinline__ float2 rotation_of(const float2* table, int pieces, int pair) {
  return table[pair % kPairs * pieces + pair / kPairs];
}

// One block a token.  Its R / 2 rotations are formed once, for all heads, in shared memory;
// then every thread moves units of rows: a piece of q (two, one of each half, for pairs
// (i, i + R / 2)) or kv_unit elements of k or v.  A thread's first unit of each kind is
// loaded before anything else, so its way from memory and the rotations' overlap.
//
// Bound by memory once there are some thousand tokens, by its chain of latencies (slot,
// position and rows, then the rotations) below; what counts is how many tokens are on their
// way, so registers are held to 32 for eight blocks an SM (8,192 tokens of 64/8 heads, pairs
// side by side: 52 us, 6.4 TB/s, against 61 us with five blocks and no spills; FP8 cache
// 54 against 66 us).  256 threads, captured calls on changing inputs: with 128, 2,176 tokens of
// 32/8 heads take 12.3 us instead of 13.2, but 256 onto an e4m3 cache 4.8 instead of 3.8; with
// 512, 19.7 and 3.4, and the long case 91.  Onto an NVFP4 cache the groups of 16 go to a few
// warps of a block, which the others await (2,176 tokens 28 us, 8,192 of 64/8 heads 103, whose
// bytes take 7 and 46; 43% of the issue slots, the barrier the largest stall).
template <int SRC, int CDT, bool kInterleaved>
__global__ void __launch_bounds__(256, CDT == PA_NVFP4 ? 4 : 8) rotary_piece_kernel(const RotaryParams p) {
  using T = typename Elem<SRC>::T;
  constexpr int kQ = Piece<SRC>::n, kKv = kv_unit<SRC, CDT>();
  constexpr int kPairs = kInterleaved ? kQ / 2 : kQ;  // pairs whose rotations a q piece needs
  extern __shared__ float2 table[];
  const long long t = blockIdx.x;
  const int d = p.head_size, rot = p.rotary_dim, half = rot / 2;
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  T* q_out = static_cast<T*>(p.q_out) + t * p.q_out_stride;
  const T* key = static_cast<const T*>(p.key) + t * p.key_stride;
  const T* value = static_cast<const T*>(p.value) + t * p.value_stride;
  const int pieces = half / kPairs, k_pieces = kInterleaved ? rot / kKv : half / kKv;
  const int k_rest = (d - rot) / kKv, plain = k_rest + d / kKv;  // k behind the rotated elements, and v
  const int q_units = p.num_q_heads * pieces, k_units = p.num_kv_heads * k_pieces, plain_units = p.num_kv_heads * plain;

  // first elements of the units
  auto q_at = [&](int u) { return u / pieces * d + u % pieces * kQ; };
  auto k_at = [&](int u) { return u / k_pieces * d + u % k_pieces * kKv; };
  Unit<SRC, kQ> qx, qy;
  auto load_q = [&](int u) {
    if (u >= q_units) return;
    qx.load(q + q_at(u));
    if constexpr (!kInterleaved) qy.load(q + q_at(u) + half);
  };
  Unit<SRC, kKv> kx, ky, vx;
  auto load_k = [&](int u) {
    if (u >= k_units) return;
    kx.load(key + k_at(u));
    if constexpr (!kInterleaved) ky.load(key + k_at(u) + half);
  };
  auto load_plain = [&](int u) {
    if (u >= plain_units) return;
    const int h = u / plain, c = u % plain;
    vx.load(c < k_rest ? key + h * d + rot + c * kKv : value + h * d + (c - k_rest) * kKv);
  };
  // the units are dealt round, so that the threads without a second q unit take k and v
  const int k_first = (threadIdx.x + 256 - q_units % 256) % 256;
  const int plain_first = (threadIdx.x + 512 - (q_units + k_units) % 256) % 256;
  previous_done();
  load_q(threadIdx.x);
  load_k(k_first);
  load_plain(plain_first);

  const long long slot = p.slot_mapping[t];
  const int pos = p.positions[t];
  for (int i = threadIdx.x; i < half; i += 256)
    table[i % kPairs * pieces + i / kPairs] = rotation(pos, turn_fraction(p.inv_freq[i]), p.attn_factor);
  if (slot < 0 || slot >= (long long)p.num_blocks * p.block_size) {
    if (slot >= 0 && threadIdx.x == 0) flag_error(p.err, PA_ERRFLAG_SLOT);
    return;
  }
  const long long tile0 = slot / p.block_size * p.num_kv_heads;
  const int off = static_cast<int>(slot % p.block_size);
  for (int u = plain_first; u < plain_units; u += 256) {
    if (u != plain_first) load_plain(u);
    const int h = u / plain, c = u % plain;
    const bool is_v = c >= k_rest;
    const int j = is_v ? (c - k_rest) * kKv : rot + c * kKv;
    void* cache = is_v ? p.v_cache : p.k_cache;
    if constexpr (SRC == CDT) {
      T* dst = static_cast<T*>(cache) + ((tile0 + h) * p.block_size + off) * d + j;
      *reinterpret_cast<uint4*>(dst) = vx.raw[0];
    } else {
      float x[kKv];
      vx.values(x);
      store_unit<SRC, CDT>(p, cache, tile0 + h, off, j, x, (is_v ? p.v_scale : p.k_scale)[h * p.scale_stride]);
    }
  }
  if (rot < d && q != q_out) {
    const int rest = (d - rot) / kQ, rest_units = p.num_q_heads * rest;
    for (int u = threadIdx.x; u < rest_units; u += 2 * 256) {
      const int u2 = u + 256;
      const int j = u / rest * d + rot + u % rest * kQ, j2 = u2 / rest * d + rot + u2 % rest * kQ;
      const uint4 a = *reinterpret_cast<const uint4*>(q + j);
      uint4 b;
      if (u2 < rest_units) b = *reinterpret_cast<const uint4*>(q + j2);
      *reinterpret_cast<uint4*>(q_out + j) = a;
      if (u2 < rest_units) *reinterpret_cast<uint4*>(q_out + j2) = b;
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < q_units; u += 256) {
    const int c = u % pieces;
    float x[kQ], y[kQ];
    if (!kInterleaved && u != static_cast<int>(threadIdx.x)) load_q(u);
    qx.values(x);
    if constexpr (kInterleaved) load_q(u + 256);
    else qy.values(y);
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < kQ; i += 2) rotate(x[i], x[i + 1], rotation_of<kPairs>(table, pieces, c * kPairs + i / 2));
    } else {
#pragma unroll
      for (int i = 0; i < kQ; ++i) rotate(x[i], y[i], rotation_of<kPairs>(table, pieces, c * kPairs + i));
      *reinterpret_cast<uint4*>(q_out + q_at(u) + half) = Piece<SRC>::pack(y);
    }
    *reinterpret_cast<uint4*>(q_out + q_at(u)) = Piece<SRC>::pack(x);
  }
  for (int u = k_first; u < k_units; u += 256) {
    const int h = u / k_pieces, j = u % k_pieces * kKv;
    const float scale = SRC == CDT ? 1.f : p.k_scale[h * p.scale_stride];
    float x[kKv], y[kKv];
    if (u != k_first) load_k(u);
    kx.values(x);
    if constexpr (!kInterleaved) ky.values(y);
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < kKv; i += 2) rotate(x[i], x[i + 1], rotation_of<kPairs>(table, pieces, (j + i) / 2));
    } else {
#pragma unroll
      for (int i = 0; i < kKv; ++i) rotate(x[i], y[i], rotation_of<kPairs>(table, pieces, j + i));
      store_unit<SRC, CDT>(p, p.k_cache, tile0 + h, off, j + half, y, scale);
    }
    store_unit<SRC, CDT>(p, p.k_cache, tile0 + h, off, j, x, scale);
  }
}

// ---------------------------------------------------------------- choice and launch

bool aligned16(const void* ptr, long long stride, int num_tokens, int bytes) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (num_tokens == 1 || stride * bytes % 16 == 0);
}

template <int SRC, int CDT>
cudaError_t launch(const RotaryParams& p, cudaStream_t stream) {
  constexpr int kBytes = Elem<SRC>::bytes, kKv = kv_unit<SRC, CDT>();
  const int half = p.rotary_dim / 2;
  // Pieces where every row allows them: on 2,176 tokens of 32/8 heads of 128 bf16 the pieces
  // take 13 us and the generic kernel, which forms a rotation for every head, 82 us.  Rows that
  // are no pieces: 2,176 tokens of 64/8 heads of 96, 24 elements turned, take 99 us (96 turned,
  // in pieces: 15), of 32/32 heads of 80, 20 turned, 104.
  const bool pieces = (p.interleaved ? p.rotary_dim : half) % kKv == 0 &&
                      aligned16(p.key, p.key_stride, p.num_tokens, kBytes) &&
                      aligned16(p.value, p.value_stride, p.num_tokens, kBytes) &&
                      (p.num_q_heads == 0 || (aligned16(p.q, p.q_stride, p.num_tokens, kBytes) &&
                                              aligned16(p.q_out, p.q_out_stride, p.num_tokens, kBytes))) &&
                      half * sizeof(float2) <= 48 * 1024;
  if (pieces) {
    const size_t smem = half * sizeof(float2);
    return launch_early(p.interleaved ? rotary_piece_kernel<SRC, CDT, true> : rotary_piece_kernel<SRC, CDT, false>,
                        dim3(p.num_tokens), 256, smem, 1, p, stream);
  }
  const long long per_token = (long long)p.num_q_heads * ((half + 3) / 4 + (p.head_size - p.rotary_dim + 7) / 8) +
                              2ll * (p.head_size / (SRC == CDT ? kKv : 16)) * p.num_kv_heads;
  const long long blocks = (per_token * p.num_tokens + 255) / 256;
  return launch_early(rotary_generic_kernel<SRC, CDT>, dim3(static_cast<unsigned>(blocks < 152 * 64 ? blocks : 152 * 64)),
                      256, 0, 1, p, stream);
}

template <int SRC>
cudaError_t launch_source(const RotaryParams& p, int cache_dtype, cudaStream_t stream) {
  switch (cache_dtype) {
    case PA_FP8_E4M3: return launch<SRC, PA_FP8_E4M3>(p, stream);
    case PA_FP8_E5M2: return launch<SRC, PA_FP8_E5M2>(p, stream);
    case PA_NVFP4: return launch<SRC, PA_NVFP4>(p, stream);
    default: return launch<SRC, SRC>(p, stream);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int src_dtype, int cache_dtype, cudaStream_t stream) {
  switch (src_dtype) {
    case PA_F32: return launch_source<PA_F32>(p, cache_dtype, stream);
    case PA_F16: return launch_source<PA_F16>(p, cache_dtype, stream);
    case PA_BF16: return launch_source<PA_BF16>(p, cache_dtype, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
