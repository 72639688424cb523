// The norms around a block, fused with its gate, residual scale and residual add.  Per token row,
// with a = gate or sigmoid(gate) (1 without a gate):
//   y = the block's output row, or sum_j w_p rows[pair_to_row[p]] over the token's routed rows
//   n = y rsqrt(mean y^2 + eps) w_post        (n = y without w_post)
//   z = x + alpha a n,   h = z rsqrt(mean z^2 + eps) w_next
// One CTA holds one row in registers, so each input is read once and z, h written once; the row
// sums (two at most, dependent) are CTA reductions in fp32.  Bound by HBM.
// Backward, from z, y and the gate (the statistics are recomputed from the row, which is read
// anyway; nothing is saved by the forward pass), with r = rsqrt(mean z^2 + eps), q = rsqrt(mean y^2 + eps):
//   d = dz + r (w_next dh) - z r^3 <z, w_next dh> / H                       (the gradient of x)
//   dn = alpha a d;  dy = q (w_post dn) - y q^3 <y, w_post dn> / H;  dgate = alpha a' d n
//   dw_next = sum_t dh z r,  dw_post = sum_t dn y q
// A persistent grid: each CTA walks rows t = b, b + gridDim.x, ... with its columns fixed per
// thread, so the weight gradients accumulate in registers (fp32) and each CTA writes one partial row;
// a second kernel adds the partial rows in CTA order (no atomics: the result does not depend on timing).
#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {
namespace {

struct NormArgs {
  const void *x, *y, *w_post, *w_next, *gate_full;
  const float* gate_tok;
  const int32_t* p2r;
  const float* topk_w;
  int T, H, k, sigmoid;
  float alpha, eps;
  void *z, *h;
  // backward
  const void *dz, *dh;
  void *dx, *dy, *dgate_full;
  float *dgate_tok, *part;
};

MOE_DEVICE float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// The sigmoid and its derivative without the cancellation of a (1 - a): with e = exp(-|v|) <= 1,
// sigmoid(|v|) = 1 / (1 + e), sigmoid(-|v|) = e / (1 + e) and the derivative e / (1 + e)^2.
MOE_DEVICE void sigmoid_grad(const float v, float& a, float& da) {
  const float e = expf(-fabsf(v)), s = 1.0f / (1.0f + e);
  a = v >= 0.0f ? s : e * s;
  da = e * s * s;
}

// W: vectors of V elements per thread.
template <typename T, int V, int W>
__global__ void __launch_bounds__(1024) k_block_norm(NormArgs a) {
  __shared__ float red[2][32];
  const int t = blockIdx.x, nv = a.H / V;
  const size_t off = size_t(t) * a.H;
  const T* x = static_cast<const T*>(a.x) + off;
  float z[W][V];
  float inv_h = 1.0f / float(a.H);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nv) {
      load_vec<T, V>(x, v).unpack(z[i]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) z[i][e] = 0.0f;
    }
  }
  if (a.y) {
    float y[W][V];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int e = 0; e < V; ++e) y[i][e] = 0.0f;
      if (v >= nv) continue;
      if (!a.p2r) {
        load_vec_once<T, V>(static_cast<const T*>(a.y) + off, v).unpack(y[i]);
      } else {
#pragma unroll 8
        for (int j = 0; j < a.k; ++j) {
          const int row = a.p2r[size_t(t) * a.k + j];
          const float w = a.topk_w ? a.topk_w[size_t(t) * a.k + j] : 1.0f;
          if (row < 0) continue;
          float f[V];
          load_vec_once<T, V>(static_cast<const T*>(a.y) + size_t(row) * a.H, v).unpack(f);
#pragma unroll
          for (int e = 0; e < V; ++e) y[i][e] = fmaf(w, f[e], y[i][e]);
        }
      }
    }
    float scale = a.alpha;
    if (a.gate_tok) scale *= a.sigmoid ? sigmoid(a.gate_tok[t]) : a.gate_tok[t];
    if (a.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] = fmaf(y[i][e], y[i][e], s[0]);
      block_sum<1>(s, red[0]);
      scale *= rsqrtf(s[0] * inv_h + a.eps);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      float m[V];
#pragma unroll
      for (int e = 0; e < V; ++e) m[e] = scale;
      if (a.w_post) {
        float w[V];
        load_vec<T, V>(static_cast<const T*>(a.w_post), v).unpack(w);
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] *= w[e];
      }
      if (a.gate_full) {
        float g[V];
        load_vec_once<T, V>(static_cast<const T*>(a.gate_full) + off, v).unpack(g);
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] *= a.sigmoid ? sigmoid(g[e]) : g[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) z[i][e] = fmaf(m[e], y[i][e], z[i][e]);
      store_vec(static_cast<T*>(a.z) + off, v, Pack<T, V>::of(z[i]));
    }
  }
  if (!a.h) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] = fmaf(z[i][e], z[i][e], s[0]);
  block_sum<1>(s, red[1]);
  const float r = rsqrtf(s[0] * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    float w[V];
    load_vec<T, V>(static_cast<const T*>(a.w_next), v).unpack(w);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] *= z[i][e] * r;
    store_vec(static_cast<T*>(a.h) + off, v, Pack<T, V>::of(w));
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(1024) k_block_norm_bwd(NormArgs a) {
  __shared__ float red1[3 * 32], red2[32];
  const int nv = a.H / V;
  const float inv_h = 1.0f / float(a.H);
  float gp[W][V], gn[W][V];  // this CTA's sums for dw_post, dw_next
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) gp[i][e] = gn[i][e] = 0.0f;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t off = size_t(t) * a.H;
    Pack<T, V> z[W], y[W], dz[W], dh[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      z[i] = y[i] = dz[i] = dh[i] = Pack<T, V>::zero();
      if (v >= nv) continue;
      if (a.dh) {
        z[i] = load_vec<T, V>(static_cast<const T*>(a.x) + off, v);
        dh[i] = load_vec<T, V>(static_cast<const T*>(a.dh) + off, v);
      }
      if (a.dz) dz[i] = load_vec<T, V>(static_cast<const T*>(a.dz) + off, v);
      if (a.y) y[i] = load_vec<T, V>(static_cast<const T*>(a.y) + off, v);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};  // <z, z>, <z, w_next dh>, <y, y>
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      float zf[V], f[V], w[V];
      if (a.dh) {
        z[i].unpack(zf);
        dh[i].unpack(f);
        load_vec<T, V>(static_cast<const T*>(a.w_next), v).unpack(w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[0] = fmaf(zf[e], zf[e], s[0]);
          s[1] = fmaf(zf[e], w[e] * f[e], s[1]);
        }
      }
      if (a.w_post) {
        y[i].unpack(f);
#pragma unroll
        for (int e = 0; e < V; ++e) s[2] = fmaf(f[e], f[e], s[2]);
      }
    }
    block_sum<3>(s, red1);
    const float r = a.dh ? rsqrtf(s[0] * inv_h + a.eps) : 0.0f;
    const float q = a.w_post ? rsqrtf(s[2] * inv_h + a.eps) : 1.0f;
    const float zc = r * r * (s[1] * inv_h);  // d = dz + r (w dh - z zc)
    float at = 1.0f, dat = 1.0f;              // the token's gate and its derivative
    if (a.gate_tok) {
      at = a.gate_tok[t];
      if (a.sigmoid) sigmoid_grad(at, at, dat);
    }
    float d[W][V];
    float s2[1] = {0.0f};  // <y, w_post d> (with the elementwise gate: <y, w_post a d>)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      dz[i].unpack(d[i]);
      if (a.dh) {
        float zf[V], f[V], w[V];
        z[i].unpack(zf);
        dh[i].unpack(f);
        load_vec<T, V>(static_cast<const T*>(a.w_next), v).unpack(w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          gn[i][e] = fmaf(f[e], zf[e] * r, gn[i][e]);
          d[i][e] = fmaf(r, w[e] * f[e] - zf[e] * zc, d[i][e]);
        }
      }
      if (a.dx) store_vec(static_cast<T*>(a.dx) + off, v, Pack<T, V>::of(d[i]));
      if (!a.y) continue;
      float yf[V], w[V], g[V];
      y[i].unpack(yf);
      if (a.w_post) load_vec<T, V>(static_cast<const T*>(a.w_post), v).unpack(w);
      if (a.gate_full) load_vec<T, V>(static_cast<const T*>(a.gate_full) + off, v).unpack(g);
      if (a.gate_full) {
        float dg[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float n = a.w_post ? yf[e] * q * w[e] : yf[e];
          float c = g[e], dc = 1.0f;
          if (a.sigmoid) sigmoid_grad(g[e], c, dc);
          dg[e] = a.alpha * dc * d[i][e] * n;
          d[i][e] *= c;
        }
        if (a.dgate_full) store_vec(static_cast<T*>(a.dgate_full) + off, v, Pack<T, V>::of(dg));
      }
#pragma unroll
      for (int e = 0; e < V; ++e) s2[0] = fmaf(yf[e], (a.w_post ? w[e] : 1.0f) * d[i][e], s2[0]);
    }
    if (a.y) {
      const bool sum2 = a.w_post || a.gate_tok;
      if (sum2) block_sum<1>(s2, red2);
      if (a.dgate_tok && threadIdx.x == 0) a.dgate_tok[t] = a.alpha * dat * q * s2[0];
      const float c = a.alpha * at;
      const float yc = q * q * (s2[0] * inv_h);  // dy = c q (w_post d - y yc)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nv) continue;
        float o[V];
        if (a.w_post) {
          float yf[V], w[V];
          y[i].unpack(yf);
          load_vec<T, V>(static_cast<const T*>(a.w_post), v).unpack(w);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            gp[i][e] = fmaf(c * d[i][e], yf[e] * q, gp[i][e]);
            o[e] = c * q * (w[e] * d[i][e] - yf[e] * yc);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = c * d[i][e];
        }
        if (a.dy) store_vec(static_cast<T*>(a.dy) + off, v, Pack<T, V>::of(o));
      }
    }
    __syncthreads();  // the next row's sums reuse red1 and red2
  }
  // partial rows: [gridDim.x][2][H]
  float* part = a.part + size_t(blockIdx.x) * 2 * a.H;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (a.w_post) part[size_t(v) * V + e] = gp[i][e];
      if (a.dh) part[a.H + size_t(v) * V + e] = gn[i][e];
    }
  }
}

// out[c] = sum over g of part[g][which][c], 32 columns per CTA, 32 row groups joined in shared memory
__global__ void __launch_bounds__(1024) k_norm_weight_sum(const float* __restrict__ part, int G, int H,
                                                          float* __restrict__ dw_post, float* __restrict__ dw_next) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g0 = threadIdx.x >> 5;
  float* out = blockIdx.y == 0 ? dw_post : dw_next;
  if (!out) return;
  float v = 0.0f;
  if (c < H)
    for (int g = g0; g < G; g += 32) v += part[(size_t(g) * 2 + blockIdx.y) * H + c];
  s[g0][threadIdx.x & 31] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x & 31][g0]);
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + g0 < H) out[blockIdx.x * 32 + g0] = v;
}

// ---------------------------------------------------------------- launchers
constexpr int kBwdCtas = 148;  // one persistent CTA per SM: partial rows of the weight gradients

NormArgs args_of(const moe_block_norm_t& b, int T, int H) {
  NormArgs a = {};
  a.y = b.y;
  a.p2r = b.pair_to_row;
  a.topk_w = b.topk_w;
  a.k = int(b.k);
  a.w_post = b.w_post;
  a.w_next = b.w_next;
  if (b.gate_mode == MOE_GATE_TOKEN) a.gate_tok = static_cast<const float*>(b.gate);
  if (b.gate_mode == MOE_GATE_FULL) a.gate_full = b.gate;
  a.sigmoid = b.gate_sigmoid;
  a.alpha = b.alpha;
  a.eps = b.eps;
  a.T = T;
  a.H = H;
  return a;
}

int round32(int n) { return (n + 31) / 32 * 32; }

template <typename T, int V>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st) {
  const int nv = a.H / V;
  if (nv <= 1024)
    k_block_norm<T, V, 1><<<unsigned(a.T), round32(nv), 0, st>>>(a);
  else if (nv <= 4096)
    k_block_norm<T, V, 4><<<unsigned(a.T), round32((nv + 3) / 4), 0, st>>>(a);
  else if constexpr (V == 1)
    k_block_norm<T, V, 16><<<unsigned(a.T), round32((nv + 15) / 16), 0, st>>>(a);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t norm_bwd(const NormArgs& a, cudaStream_t st) {
  const int nv = a.H / V;
  const unsigned grid = unsigned(a.T < kBwdCtas ? a.T : kBwdCtas);
  if (nv <= 1024)
    k_block_norm_bwd<T, V, 1><<<grid, round32(nv), 0, st>>>(a);
  else if (nv <= 4096)
    k_block_norm_bwd<T, V, 4><<<grid, round32((nv + 3) / 4), 0, st>>>(a);
  else if constexpr (V == 1)
    k_block_norm_bwd<T, V, 16><<<grid, round32((nv + 15) / 16), 0, st>>>(a);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_of(const NormArgs& a, bool bwd, cudaStream_t st) {
  constexpr int V = vec_width<T>();
  bool wide = a.H % V == 0;
  const void* ps[] = {a.x, a.y, a.w_post, a.w_next, a.gate_full, a.z, a.h, a.dz, a.dh, a.dx, a.dy, a.dgate_full};
  for (const void* p : ps) wide = wide && vec_aligned(p);
  if (bwd) return wide ? norm_bwd<T, V>(a, st) : norm_bwd<T, 1>(a, st);
  return wide ? norm_fwd<T, V>(a, st) : norm_fwd<T, 1>(a, st);
}

cudaError_t norm_any(const NormArgs& a, moe_dtype_t dt, bool bwd, cudaStream_t st) {
  if (dt == MOE_BF16) return norm_of<__nv_bfloat16>(a, bwd, st);
  if (dt == MOE_F16) return norm_of<__half>(a, bwd, st);
  return norm_of<float>(a, bwd, st);
}

}  // namespace

cudaError_t launch_block_norm(const moe_block_norm_t& b, const void* x, int T, int H, moe_dtype_t dt, void* z, void* h,
                              cudaStream_t st) {
  NormArgs a = args_of(b, T, H);
  a.x = x;
  a.z = z;
  a.h = h;
  return norm_any(a, dt, false, st);
}

size_t block_norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  const int64_t g = T < kBwdCtas ? T : kBwdCtas;
  return size_t(g) * 2 * size_t(H) * sizeof(float);
}

cudaError_t launch_block_norm_bwd(const moe_block_norm_t& b, const void* z, const void* dz, const void* dh, int T, int H,
                                  moe_dtype_t dt, const moe_block_norm_grads_t& g, void* ws, cudaStream_t st) {
  NormArgs a = args_of(b, T, H);
  a.x = z;
  a.dz = dz;
  a.dh = dh;
  a.dx = g.dx;
  a.dy = g.dy;
  if (b.gate_mode == MOE_GATE_TOKEN) a.dgate_tok = static_cast<float*>(g.dgate);
  if (b.gate_mode == MOE_GATE_FULL) a.dgate_full = g.dgate;
  a.part = static_cast<float*>(ws);
  cudaError_t err = norm_any(a, dt, true, st);
  if (err != cudaSuccess || (!g.dw_post && !g.dw_next)) return err;
  k_norm_weight_sum<<<dim3(unsigned((H + 31) / 32), 2), 1024, 0, st>>>(a.part, T < kBwdCtas ? T : kBwdCtas, H, g.dw_post,
                                                                       g.dw_next);
  return cudaGetLastError();
}

}  // namespace moe
