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

// Two 16-bit elements of a register, and back (rounded to nearest even).
MOE_DEVICE void unpack2(uint32_t w, float& lo, float& hi, __nv_bfloat16) {
  lo = bf16_lo(w);
  hi = bf16_hi(w);
}
MOE_DEVICE void unpack2(uint32_t w, float& lo, float& hi, __half) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = v.x;
  hi = v.y;
}
MOE_DEVICE uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
MOE_DEVICE uint32_t pack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// V elements as they lie in memory (kept packed while a load is in flight): V * sizeof(T) is 16, or V = 1.
template <int BYTES>
struct RawOf;
template <>
struct RawOf<16> {
  using type = uint4;
};
template <>
struct RawOf<8> {
  using type = uint2;
};
template <>
struct RawOf<4> {
  using type = uint32_t;
};
template <>
struct RawOf<2> {
  using type = uint16_t;
};
template <typename T, int V>
struct Pack {
  using Raw = typename RawOf<V * int(sizeof(T))>::type;
  Raw raw;
  MOE_DEVICE void unpack(float (&f)[V]) const {
    if constexpr (V == 8) {
      unpack2(raw.x, f[0], f[1], T());
      unpack2(raw.y, f[2], f[3], T());
      unpack2(raw.z, f[4], f[5], T());
      unpack2(raw.w, f[6], f[7], T());
    } else if constexpr (V == 4) {
      f[0] = __uint_as_float(raw.x);
      f[1] = __uint_as_float(raw.y);
      f[2] = __uint_as_float(raw.z);
      f[3] = __uint_as_float(raw.w);
    } else {
      f[0] = to_float(*reinterpret_cast<const T*>(&raw));
    }
  }
  MOE_DEVICE static Pack of(const float (&f)[V]) {
    Pack p;
    if constexpr (V == 8) {
      p.raw = make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()), pack2(f[6], f[7], T()));
    } else if constexpr (V == 4) {
      p.raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      const T v = from_float<T>(f[0]);
      p.raw = *reinterpret_cast<const Raw*>(&v);
    }
    return p;
  }
  MOE_DEVICE static Pack zero() {
    Pack p;
    if constexpr (V > 1)
      p.raw = make_uint4(0, 0, 0, 0);
    else
      p.raw = 0;
    return p;
  }
};

// Vector v of a row (plain load: the row may be written by the same call, e.g. an output
// that aliases its input).
template <typename T, int V>
MOE_DEVICE Pack<T, V> load_vec(const T* row, int v) {
  Pack<T, V> p;
  p.raw = *reinterpret_cast<const typename Pack<T, V>::Raw*>(row + size_t(v) * V);
  return p;
}
// The same through the read-only path, for data that no one writes during the call; the line
// is not kept in L1 (each row is read once).
template <typename T, int V>
MOE_DEVICE Pack<T, V> load_vec_once(const T* row, int v) {
  Pack<T, V> p;
  if constexpr (V > 1)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(p.raw.x), "=r"(p.raw.y), "=r"(p.raw.z), "=r"(p.raw.w)
                 : "l"(row + size_t(v) * V));
  else
    p.raw = __ldg(reinterpret_cast<const typename Pack<T, V>::Raw*>(row + v));
  return p;
}
template <typename T, int V>
MOE_DEVICE void store_vec(T* row, int v, const Pack<T, V>& p) {
  *reinterpret_cast<typename Pack<T, V>::Raw*>(row + size_t(v) * V) = p.raw;
}

MOE_DEVICE float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The warp's sums of N values (N a power of two up to 32): lane l returns the sum of value l / (32 / N).  Each step of the
// butterfly halves the values a lane carries: N - 1 + log2(32 / N) exchanges instead of 5 N.
template <int N>
MOE_DEVICE float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int w = 16;
#pragma unroll
  for (int n = N; n > 1; n /= 2, w /= 2) {
    const bool upper = lane & w;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = upper ? v[i] : v[n / 2 + i], keep = upper ? v[n / 2 + i] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
    }
  }
#pragma unroll
  for (; w >= 1; w /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
  return v[0];
}

// Sums of N values (1, 2 or 4) over the CTA (blockDim.x a multiple of 32, at most 1024), in one fixed order, to every
// thread.  `red`: 32 * N floats of shared memory that no sum wrote since the barrier before last.
template <int N>
MOE_DEVICE void block_sum(float (&v)[N], float* red) {
  constexpr int L = 32 / N;  // lanes per value
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float s = warp_sums<N>(v);
  if (nw > 1) {
    if (lane % L == 0) red[(lane / L) * 32 + warp] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < N; ++w)
      if (lane % L + w * L < nw) s += red[(lane / L) * 32 + lane % L + w * L];
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = N > 1 ? __shfl_sync(0xffffffffu, s, i * L) : s;
}

template <typename T>
constexpr int vec_width() {
  return 16 / int(sizeof(T));
}
inline bool vec_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace moe
