// Single elements of cached token rows in every cache format, and the joining of two softmax
// states: what the attention kernels without matrix instructions share.
#pragma once

#include "pa_common.cuh"

namespace pa {

// A token row of a cache tile (= physical block x Hkv + KV head): the address of its
// first element (NVFP4: of its code row) and, for NVFP4, of its block-scale row.
struct KvRow {
  const uint8_t* row;
  const uint8_t* scales;
};

template <int KVDT>
__device__ __forceinline__ KvRow kv_row(const void* cache, long long tile, int bs, int d, int off) {
  const uint8_t* base = static_cast<const uint8_t*>(cache);
  if constexpr (is_nvfp4<KVDT>()) {
    const uint8_t* t = base + tile * nvfp4_tile_bytes(bs, d);
    return {t + off * (d / 2), t + bs * (d / 2) + off * (d / 16)};
  } else {
    return {base + ((tile * bs + off) * d) * Elem<KVDT>::bytes, nullptr};
  }
}

// Stored value (without the fp32 scale) of element dd of a token row.
template <int KVDT>
__device__ __forceinline__ float kv_elem(const KvRow& r, int dd) {
  if constexpr (is_nvfp4<KVDT>()) {
    const uint32_t byte = r.row[dd >> 1];
    const __half2_raw c = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
    __half_raw v;
    v.x = (dd & 1) ? c.y : c.x;
    const __half_raw b = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(r.scales[dd >> 4]), __NV_E4M3);
    return __half2float(__half(v)) * __half2float(__half(b));
  } else {
    using KE = Elem<KVDT>;
    return KE::load(reinterpret_cast<const typename KE::T*>(r.row) + dd);
  }
}

// The running maximum and sum (m, l) of one softmax joined with another's (m2, l2).
__device__ __forceinline__ void combine_ml(float& m, float& l, float m2, float l2) {
  if (l2 <= 0.f) return;
  if (l <= 0.f) {
    m = m2;
    l = l2;
    return;
  }
  const float nm = fmaxf(m, m2);
  l = l * exp2f(m - nm) + l2 * exp2f(m2 - nm);
  m = nm;
}

}  // namespace pa
