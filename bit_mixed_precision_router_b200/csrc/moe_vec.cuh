// Element types of the row operators (bf16, fp16, fp32) and their loads and stores as fp32
// vectors of V elements: V * sizeof(T) is 16 bytes (one 128-bit access) or V = 1.
#pragma once

#include "moe_common.cuh"

namespace moe {

MOE_DEVICE float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
MOE_DEVICE float to_float(__half v) { return __half2float(v); }
MOE_DEVICE float to_float(float v) { return v; }
template <typename T>
MOE_DEVICE T from_float(float f);
template <>
MOE_DEVICE __nv_bfloat16 from_float<__nv_bfloat16>(float f) {
  return __float2bfloat16_rn(f);
}
template <>
MOE_DEVICE __half from_float<__half>(float f) {
  return __float2half_rn(f);
}
template <>
MOE_DEVICE float from_float<float>(float f) {
  return f;
}

MOE_DEVICE void unpack2(uint32_t w, float& lo, float& hi, __nv_bfloat16) {
  lo = bf16_lo(w);
  hi = bf16_hi(w);
}
MOE_DEVICE void unpack2(uint32_t w, float& lo, float& hi, __half) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = v.x;
  hi = v.y;
}

// V elements as they lie in memory (kept packed while a load is in flight).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
  MOE_DEVICE void unpack(float (&f)[V]) const {
    if constexpr (V == 8) {  // two 16-bit elements per register
      const uint4 u = *reinterpret_cast<const uint4*>(e);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack2(w[i], f[2 * i], f[2 * i + 1], T());
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = to_float(e[i]);
    }
  }
  MOE_DEVICE static Pack of(const float (&f)[V]) {
    Pack p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = from_float<T>(f[i]);
    return p;
  }
  MOE_DEVICE static Pack zero() {
    Pack p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = from_float<T>(0.0f);
    return p;
  }
};

// Vector v of a row (plain load: the row may be written by the same call, e.g. an output
// that aliases its input).
template <typename T, int V>
MOE_DEVICE Pack<T, V> load_vec(const T* row, int v) {
  return *reinterpret_cast<const Pack<T, V>*>(row + size_t(v) * V);
}
// The same through the read-only path, for data that no one writes during the call; the line
// is not kept in L1 (each row is read once).
template <typename T, int V>
MOE_DEVICE Pack<T, V> load_vec_once(const T* row, int v) {
  Pack<T, V> p;
  if constexpr (sizeof(p) == 16) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(row + size_t(v) * V));
    p = *reinterpret_cast<const Pack<T, V>*>(&u);
  } else {
    p = *reinterpret_cast<const Pack<T, V>*>(row + size_t(v) * V);
  }
  return p;
}
template <typename T, int V>
MOE_DEVICE void store_vec(T* row, int v, const Pack<T, V>& p) {
  *reinterpret_cast<Pack<T, V>*>(row + size_t(v) * V) = p;
}

MOE_DEVICE float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sums of N values over the CTA (blockDim.x a multiple of 32), in one fixed order.  `red`:
// 32 * N floats of shared memory that no earlier sum of the same iteration used.
template <int N>
MOE_DEVICE void block_sum(float (&v)[N], float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (nw == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < nw ? red[i * 32 + lane] : 0.0f);
}

template <typename T>
constexpr int vec_width() {
  return 16 / int(sizeof(T));
}
inline bool vec_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace moe
