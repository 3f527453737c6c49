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

template <int SRC, int CDT>
cudaError_t launch_generic(const RotaryParams& p, cudaStream_t stream) {
  const long long groups = p.head_size / (SRC == CDT ? 16 / Elem<SRC>::bytes : 16);
  const long long per_token = (long long)p.num_q_heads * ((p.rotary_dim / 2 + 3) / 4 + (p.head_size - p.rotary_dim + 7) / 8) +
                              2 * groups * p.num_kv_heads;
  const long long blocks = (per_token * p.num_tokens + 255) / 256;
  rotary_generic_kernel<SRC, CDT><<<static_cast<int>(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int SRC>
cudaError_t launch_source(const RotaryParams& p, int cache_dtype, cudaStream_t stream) {
  switch (cache_dtype) {
    case PA_FP8_E4M3: return launch_generic<SRC, PA_FP8_E4M3>(p, stream);
    case PA_FP8_E5M2: return launch_generic<SRC, PA_FP8_E5M2>(p, stream);
    case PA_NVFP4: return launch_generic<SRC, PA_NVFP4>(p, stream);
    default: return launch_generic<SRC, SRC>(p, stream);
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
