// The norms around a block, fused with its gate, residual scale and residual add.  Per token row,
// with a = gate or sigmoid(gate) (1 without a gate):
//   y = the block's output row, or sum_j w_p rows[pair_to_row[p]] over the token's routed rows
//   n = y rsqrt(mean y^2 + eps) w_post        (n = y without w_post)
//   z = x + alpha a n,   h = z rsqrt(mean z^2 + eps) w_next
// One CTA holds one row in registers, so each input is read once and z, h written once; the row
// sums (two at most, dependent) are CTA reductions in fp32.  Bound by HBM (4096 x 7168 bf16: 46 us, 36 us at the copy's rate);
// with an elementwise gate by half by its sigmoids.
// Backward, from z, y and the gate (the statistics are recomputed from the row, which is read
// anyway; nothing is saved by the forward pass), with r = rsqrt(mean z^2 + eps), q = rsqrt(mean y^2 + eps):
//   d = dz + r (w_next dh) - z r^3 <z, w_next dh> / H                       (the gradient of x)
//   dn = alpha a d;  dy = q (w_post dn) - y q^3 <y, w_post dn> / H;  dgate = alpha a' d n
//   dw_next = sum_t dh z r,  dw_post = sum_t dn y q
// 4096 x 7168 bf16, gate per token: 76 us, 54 us at the copy's rate; with an elementwise gate 122 us, 72 at the copy's rate.
// A persistent grid: each CTA walks rows t = b, b + gridDim.x, ... with its columns fixed per
// thread, so the weight gradients accumulate in registers and each CTA writes one partial row; a second kernel adds the
// partial rows in CTA order (no atomics: the result does not depend on timing).  These sums are fp32, T / CTAs terms in a CTA
// and then the CTAs' (64 bits would take twice the registers, which bound the kernel): off by at most (T + 128) 2^-24 of the
// terms' magnitudes.
#include <atomic>
#include <climits>
#include <type_traits>

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

constexpr int kNormSlots = 8;  // routed rows in flight per thread

MOE_DEVICE float rcp_approx(float v) {  // within one unit of the last place; 0 for v > 2^126
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The sigmoid: with e = exp(-|v|) <= 1, sigmoid(|v|) = 1 / (1 + e) and sigmoid(-|v|) = e / (1 + e): nothing overflows, and it
// keeps its last places down to where fp32 ends.  The gates that are fp32 themselves, and all gradients (w_post's is fp32 whatever
// the gate is), take these two.
MOE_DEVICE float sigmoid_of(float v) {
  const float e = expf(-fabsf(v)), s = rcp_approx(1.0f + e);
  return v >= 0.0f ? s : e * s;
}
// The sigmoid and its derivative e / (1 + e)^2, without the cancellation of a (1 - a).
MOE_DEVICE void sigmoid_grad(const float v, float& a, float& da) {
  const float e = expf(-fabsf(v)), s = rcp_approx(1.0f + e);
  a = v >= 0.0f ? s : e * s;
  da = e * s * s;
}

// The sigmoid of an elementwise gate on its way into z, which has the gate's type.  For 16 bits ex2.approx.ftz does: 2^-22 relative
// by itself and 1.3 |v| 2^-24 by the rounded product v log2(e), together below 2^-17, where z's half step is 2^-8 (bf16) or
// 2^-11 (fp16); a sigmoid below 2^-126 becomes 0.  A third of the instructions: 2048 x 7168 bf16 29.1 us, with expf 31.9.
template <typename T>
MOE_DEVICE float gate_of(float v) {
  if constexpr (sizeof(T) == 4) return sigmoid_of(v);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  return rcp_approx(1.0f + e);
}

// W: vectors of V elements per thread.  The row's loads are all issued before the first sum.  ROUTED: y is the
// weighted sum of the token's routed rows.
template <typename T, int V, int W, int THREADS, int CTAS, bool ROUTED>
__global__ void __launch_bounds__(THREADS, CTAS) k_block_norm(NormArgs a) {
  __shared__ float red[2][32];
  const int t = blockIdx.x, nv = a.H / V;
  const size_t off = size_t(t) * a.H;
  const float inv_h = 1.0f / float(a.H);
  Pack<T, V> xp[W], gp[W];
  float y[W][V];
  const float gate = a.gate_tok ? a.gate_tok[t] : 1.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    xp[i] = Pack<T, V>::zero();
    if (v < nv) {
      xp[i] = load_vec<T, V>(static_cast<const T*>(a.x) + off, v);
      if (a.gate_full) gp[i] = load_vec_once<T, V>(static_cast<const T*>(a.gate_full) + off, v);
    }
  }
  if (a.y) {
    if (!ROUTED) {
      Pack<T, V> yp[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        yp[i] = Pack<T, V>::zero();
        if (v < nv) yp[i] = load_vec_once<T, V>(static_cast<const T*>(a.y) + off, v);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) yp[i].unpack(y[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) y[i][e] = 0.0f;
      // the token's rows, kNormSlots at a time, in slot order
      for (int j0 = 0; j0 < a.k; j0 += kNormSlots) {
        int row[kNormSlots];
        float w[kNormSlots];
#pragma unroll
        for (int j = 0; j < kNormSlots; ++j) {
          const size_t p = size_t(t) * a.k + j0 + j;
          row[j] = j0 + j < a.k ? a.p2r[p] : -1;
          w[j] = a.topk_w && j0 + j < a.k ? a.topk_w[p] : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int v = threadIdx.x + i * blockDim.x;
          if (v >= nv) continue;
          Pack<T, V> r[kNormSlots];
#pragma unroll
          for (int j = 0; j < kNormSlots; ++j)
            if (row[j] >= 0) r[j] = load_vec_once<T, V>(static_cast<const T*>(a.y) + size_t(row[j]) * a.H, v);
#pragma unroll
          for (int j = 0; j < kNormSlots; ++j) {
            if (row[j] < 0) continue;
            float f[V];
            r[j].unpack(f);
#pragma unroll
            for (int e = 0; e < V; ++e) y[i][e] = fmaf(w[j], f[e], y[i][e]);
          }
        }
      }
    }
    float scale = a.alpha;
    if (a.gate_tok) scale *= a.sigmoid ? sigmoid_of(gate) : gate;
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
      float m[V], xf[V];
#pragma unroll
      for (int e = 0; e < V; ++e) m[e] = scale;
      if (a.w_post && v < nv) {
        float w[V];
        load_vec<T, V>(static_cast<const T*>(a.w_post), v).unpack(w);
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] *= w[e];
      }
      if (a.gate_full && v < nv) {
        float g[V];
        gp[i].unpack(g);
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] *= a.sigmoid ? gate_of<T>(g[e]) : g[e];
      }
      xp[i].unpack(xf);
#pragma unroll
      for (int e = 0; e < V; ++e) y[i][e] = fmaf(m[e], y[i][e], xf[e]);  // z; zeros past the row's end
      if (v < nv) store_vec(static_cast<T*>(a.z) + off, v, Pack<T, V>::of(y[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) xp[i].unpack(y[i]);
  }
  if (!a.h) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] = fmaf(y[i][e], y[i][e], s[0]);
  block_sum<1>(s, red[1]);
  const float r = rsqrtf(s[0] * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    float w[V];
    load_vec<T, V>(static_cast<const T*>(a.w_next), v).unpack(w);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] *= y[i][e] * r;
    store_vec(static_cast<T*>(a.h) + off, v, Pack<T, V>::of(w));
  }
}

// The rows of the backward pass wait in shared memory: every thread copies its own vectors of the next rows
// (cp.async, no barrier: it reads back what it copied itself) while it works on the current one.
template <typename T, int V>
MOE_DEVICE void copy_vec(Pack<T, V>* dst, const T* row, int v) {
  if constexpr (sizeof(Pack<T, V>) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(row + size_t(v) * V) : "memory");
  else if constexpr (sizeof(Pack<T, V>) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(row + size_t(v) * V) : "memory");
  else
    *dst = load_vec<T, V>(row, v);
}

// Persistent CTAs per SM: 768 threads (80 registers each), one CTA of more.
__host__ __device__ constexpr int bwd_ctas(int threads) { return threads > 768 ? 1 : 768 / threads; }

enum { kZ, kDh, kDz, kY, kGate, kArrays };  // arrays of a stage

// bytes of a stage: a row of every array
template <typename T, int V, int W, int THREADS>
__host__ __device__ constexpr int bwd_stage_bytes(bool gate) {
  return (gate ? kArrays : kArrays - 1) * W * THREADS * int(sizeof(Pack<T, V>));
}

// FULL: a step with dz, dh, y, w_post and the gradients of x and y, and no elementwise gate, known to the compiler.  DIRECT: rows
// too long for two stages are read from global memory (the second reading from L2).
template <typename T, int V, int W, int THREADS, bool DIRECT, bool FULL>
__global__ void __launch_bounds__(THREADS, bwd_ctas(THREADS)) k_block_norm_bwd(NormArgs a, int depth) {
  const bool has_dh = FULL || a.dh, has_dz = FULL || a.dz, has_y = FULL || a.y, has_post = FULL || a.w_post;
  const bool has_dx = FULL || a.dx, has_dy = FULL || a.dy, has_gate = !FULL && a.gate_full;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red1[4 * 32], red2[4 * 32];
  const int nv = a.H / V, nth = blockDim.x;
  const int stage_bytes = bwd_stage_bytes<T, V, W, THREADS>(has_gate);
  const float inv_h = 1.0f / float(a.H);
  uint8_t* const mine = smem + threadIdx.x * sizeof(Pack<T, V>);
  // array and vector at offsets known to the compiler: spaced for THREADS threads, whatever the launch has
  auto slot = [&](int stage, int arr, int i) {
    return reinterpret_cast<Pack<T, V>*>(mine + stage * stage_bytes + (arr * W + i) * THREADS * int(sizeof(Pack<T, V>)));
  };
  auto get = [&](int stage, int arr, int i, size_t off) {
    if constexpr (DIRECT) {
      const void* const from[kArrays] = {a.x, a.dh, a.dz, a.y, a.gate_full};
      return load_vec<T, V>(static_cast<const T*>(from[arr]) + off, threadIdx.x + i * nth);
    } else {
      return *slot(stage, arr, i);
    }
  };
  auto fetch = [&](int t, int stage) {
    if (DIRECT) return;
    if (t < a.T) {
      const size_t off = size_t(t) * a.H;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int v = threadIdx.x + i * nth;
        if (v >= nv) continue;
        if (has_dh) {
          copy_vec(slot(stage, kZ, i), static_cast<const T*>(a.x) + off, v);
          copy_vec(slot(stage, kDh, i), static_cast<const T*>(a.dh) + off, v);
        }
        if (has_dz) copy_vec(slot(stage, kDz, i), static_cast<const T*>(a.dz) + off, v);
        if (has_y) copy_vec(slot(stage, kY, i), static_cast<const T*>(a.y) + off, v);
        if (has_gate) copy_vec(slot(stage, kGate, i), static_cast<const T*>(a.gate_full) + off, v);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Single 16-bit elements have no asynchronous copy: a row ahead waits in registers, from the start of one row's work to its
  // end (while there are registers).
  constexpr bool HOLD = !DIRECT && sizeof(Pack<T, V>) == 2 && W <= 4;
  Pack<T, V> held[HOLD ? kArrays : 1][W];
  auto hold = [&](int t) {
    if (t >= a.T) return;
    const size_t off = size_t(t) * a.H;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * nth;
      if (v >= nv) continue;
      if (has_dh) {
        held[kZ][i] = load_vec<T, V>(static_cast<const T*>(a.x) + off, v);
        held[kDh][i] = load_vec<T, V>(static_cast<const T*>(a.dh) + off, v);
      }
      if (has_dz) held[kDz][i] = load_vec<T, V>(static_cast<const T*>(a.dz) + off, v);
      if (has_y) held[kY][i] = load_vec<T, V>(static_cast<const T*>(a.y) + off, v);
      if (has_gate) held[kGate][i] = load_vec<T, V>(static_cast<const T*>(a.gate_full) + off, v);
    }
  };
  auto put = [&](int t, int stage) {
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (threadIdx.x + i * nth >= nv) continue;
      if (has_dh) {
        *slot(stage, kZ, i) = held[kZ][i];
        *slot(stage, kDh, i) = held[kDh][i];
      }
      if (has_dz) *slot(stage, kDz, i) = held[kDz][i];
      if (has_y) *slot(stage, kY, i) = held[kY][i];
      if (has_gate) *slot(stage, kGate, i) = held[kGate][i];
    }
  };
  Pack<T, V> wn[W], wp[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * nth;
    wn[i] = wp[i] = Pack<T, V>::zero();
    if (v < nv && has_dh) wn[i] = load_vec<T, V>(static_cast<const T*>(a.w_next), v);
    if (v < nv && has_post) wp[i] = load_vec<T, V>(static_cast<const T*>(a.w_post), v);
  }
  float gp[W][V], gn[W][V];  // this CTA's sums for dw_post, dw_next
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) gp[i][e] = gn[i][e] = 0.0f;
  // <z, z>, <z, w_next dh>, <y, y> of a row
  auto first_sums = [&](float* s, int stage, size_t off) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (threadIdx.x + i * nth >= nv) continue;
      float zf[V], f[V], w[V];
      if (has_dh) {
        get(stage, kZ, i, off).unpack(zf);
        get(stage, kDh, i, off).unpack(f);
        wn[i].unpack(w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[0] = fmaf(zf[e], zf[e], s[0]);
          s[1] = fmaf(zf[e], w[e] * f[e], s[1]);
        }
      }
      if (has_post) {
        get(stage, kY, i, off).unpack(f);
#pragma unroll
        for (int e = 0; e < V; ++e) s[2] = fmaf(f[e], f[e], s[2]);
      }
    }
  };
  float r = 0.0f, q = 1.0f, zc = 0.0f;  // d = dz + r (w dh - z zc)
  auto statistics = [&](const float* s) {
    if (has_dh) r = rsqrtf(s[0] * inv_h + a.eps);
    if (has_post) q = rsqrtf(s[2] * inv_h + a.eps);
    zc = r * (r * (s[1] * inv_h));  // r * r alone overflows for eps below 2^-128
  };
  // One barrier per row: the second sum of row t and the first sums of the CTA's next row are joined together.
  // the kernel that joins the partial sums may be launched; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int stage = 0, ahead = 1;
  // the gate of the next row, read a row ahead: reading it in its own row cost a fifth of the time (97 against 76 us)
  float gate = a.gate_tok ? a.gate_tok[blockIdx.x] : 1.0f;
  fetch(blockIdx.x, 0);
  fetch(blockIdx.x + gridDim.x, 1);
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    first_sums(s, 0, size_t(blockIdx.x) * a.H);
    block_sum<4>(s, red1);
    statistics(s);
  }
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, ahead ^= 1) {
    const int after = stage + 1 == depth ? 0 : stage + 1;  // the next row's stage
    if constexpr (HOLD)
      hold(t + 2 * gridDim.x);
    else if (depth == 3)
      fetch(t + 2 * gridDim.x, after + 1 == depth ? 0 : after + 1);
    const size_t off = size_t(t) * a.H;
    float at = gate, dat = 1.0f;  // the token's gate and its derivative
    if (a.gate_tok) {
      if (t + gridDim.x < a.T) gate = a.gate_tok[t + gridDim.x];
      if (a.sigmoid) sigmoid_grad(at, at, dat);
    }
    float d[W][V];
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // [3]: <y, w_post d> (with the elementwise gate: <y, w_post a d>)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int v = threadIdx.x + i * nth;
      if (v >= nv) continue;
      if (has_dz) {
        get(stage, kDz, i, off).unpack(d[i]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) d[i][e] = 0.0f;
      }
      if (has_dh) {
        float zf[V], f[V], w[V];
        get(stage, kZ, i, off).unpack(zf);
        get(stage, kDh, i, off).unpack(f);
        wn[i].unpack(w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          gn[i][e] = fmaf(f[e], zf[e] * r, gn[i][e]);
          d[i][e] = fmaf(r, w[e] * f[e] - zf[e] * zc, d[i][e]);
        }
      }
      if (has_dx) store_vec(static_cast<T*>(a.dx) + off, v, Pack<T, V>::of(d[i]));
      if (!has_y) continue;
      float yf[V], w[V];
      get(stage, kY, i, off).unpack(yf);
      if (has_post) {
        wp[i].unpack(w);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = 1.0f;
      }
      if (has_gate) {
        float g[V], dg[V];
        get(stage, kGate, i, off).unpack(g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float c = g[e], dc = 1.0f;
          if (a.sigmoid) sigmoid_grad(g[e], c, dc);
          dg[e] = a.alpha * dc * d[i][e] * (yf[e] * q * w[e]);
          d[i][e] *= c;
        }
        if (a.dgate_full) store_vec(static_cast<T*>(a.dgate_full) + off, v, Pack<T, V>::of(dg));
      }
#pragma unroll
      for (int e = 0; e < V; ++e) s[3] = fmaf(yf[e], w[e] * d[i][e], s[3]);
    }
    if (depth == 3)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (t + gridDim.x < a.T) first_sums(s, after, off + size_t(gridDim.x) * a.H);
    block_sum<4>(s, ahead ? red2 : red1);
    if (a.dgate_tok && threadIdx.x == 0) a.dgate_tok[t] = a.alpha * dat * q * s[3];
    if (has_y) {
      const float c = a.alpha * at;
      const float yc = q * (q * (s[3] * inv_h));  // dy = c q (w_post d - y yc)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int v = threadIdx.x + i * nth;
        if (v >= nv) continue;
        float o[V];
        if (has_post) {
          float yf[V], w[V];
          get(stage, kY, i, off).unpack(yf);
          wp[i].unpack(w);
          const float cq = c * q;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            gp[i][e] = fmaf(cq * d[i][e], yf[e], gp[i][e]);
            o[e] = cq * (w[e] * d[i][e] - yf[e] * yc);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = c * d[i][e];
        }
        if (has_dy) store_vec(static_cast<T*>(a.dy) + off, v, Pack<T, V>::of(o));
      }
    }
    statistics(s);
    if constexpr (HOLD)
      put(t + 2 * gridDim.x, depth == 2 ? stage : after + 1 == depth ? 0 : after + 1);
    else if (depth == 2)
      fetch(t + 2 * gridDim.x, stage);
    stage = after;
  }
  // partial rows: [gridDim.x][2][H]
  float* part = a.part + size_t(blockIdx.x) * 2 * a.H;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int v = threadIdx.x + i * nth;
    if (v >= nv) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (has_post) part[size_t(v) * V + e] = gp[i][e];
      if (has_dh) part[a.H + size_t(v) * V + e] = gn[i][e];
    }
  }
}

// out[c] = sum over g of part[g][which][c], 32 columns per CTA, 32 row groups joined in shared memory.  Launched while the
// kernel that writes `part` still runs (512 x 2048: 11.1 -> 10.4 us for both), so it waits for that one to be complete first,
// and `part` is no const __restrict__: it changes during this kernel, and is read through L2 (__ldcg), behind the wait.
__global__ void __launch_bounds__(1024) k_norm_weight_sum(const float* part, int G, int H, float* dw_post, float* dw_next) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g0 = threadIdx.x >> 5;
  float* out = blockIdx.y == 0 ? dw_post : dw_next;
  if (!out) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v = 0.0f;
  if (c < H)
#pragma unroll 8
    for (int g = g0; g < G; g += 32) v += __ldcg(part + (size_t(g) * 2 + blockIdx.y) * H + c);
  s[g0][threadIdx.x & 31] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x & 31][g0]);
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + g0 < H) out[blockIdx.x * 32 + g0] = v;
}

// ---------------------------------------------------------------- launchers
int round32(int n) { return (n + 31) / 32 * 32; }

constexpr int kSms = 148;

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

template <typename T, int V, bool ROUTED>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st) {
  const int nv = a.H / V;
  const unsigned rows = unsigned(a.T);
  // Few rows: a vector per thread, the shortest path through the row.  Many: two vectors per thread, so that
  // several CTAs share an SM and one's loads run during the others' sums.  Up to 384 threads three CTAs of 55 registers fit an SM by
  // themselves; beyond, 40 registers make room for the third (4096 x 7168 50 -> 46 us; at 1000 x 4096 it would cost 7.1 -> 8.5 us).
  // Routed rows keep two: their slots' indices and weights fill 64 registers as it is.
  constexpr int wide_ctas = ROUTED ? 2 : 3;
  if (nv <= 1024 && (a.T < 2 * kSms || nv <= 64)) {
    k_block_norm<T, V, 1, 1024, 1, ROUTED><<<rows, round32(nv), 0, st>>>(a);
  } else if (nv <= 768) {
    k_block_norm<T, V, 2, 512, 2, ROUTED><<<rows, round32((nv + 1) / 2), 0, st>>>(a);
  } else if (nv <= 1024) {
    k_block_norm<T, V, 2, 512, wide_ctas, ROUTED><<<rows, round32((nv + 1) / 2), 0, st>>>(a);
  } else if (nv <= 4096) {
    k_block_norm<T, V, 4, V == 8 ? 512 : 1024, 1, ROUTED><<<rows, round32((nv + 3) / 4), 0, st>>>(a);
  } else if constexpr (V == 1) {
    if (nv <= 8192)
      k_block_norm<T, V, 8, 1024, 1, ROUTED><<<rows, round32((nv + 7) / 8), 0, st>>>(a);
    else
      k_block_norm<T, V, 16, 1024, 1, ROUTED><<<rows, round32((nv + 15) / 16), 0, st>>>(a);
  } else {
    return cudaErrorInvalidValue;  // H <= 16384: at most 4096 vectors
  }
  return cudaGetLastError();
}

// CTAs: one or more per SM.  A CTA's rows follow one another, and its partial sums cost 8 H bytes written and read, so their
// number goes with sqrt(T / H); single elements take longer over a row.  512 x 2048 bf16: 148 CTAs 11.5, 444 CTAs 16.1 us;
// 4096 x 2048: 148, 296 and 444 CTAs 35, 29 and 32 us; 4000 x 511: 444 and 888 CTAs 35 and 25 us.
int bwd_grid(int T, int H, int threads, bool single) {
  int c = 1;
  while (c < bwd_ctas(threads) && int64_t(2 * c + 1) * (2 * c + 1) * H <= int64_t(single ? 36 : 12) * T) ++c;
  return T < kSms * c ? T : kSms * c;
}
constexpr int kSmemMax = 224 * 1024;

template <typename T, int V, int W, int THREADS, bool DIRECT, bool FULL>
cudaError_t run_bwd_as(const NormArgs& a, int grid, cudaStream_t st) {
  // raised once per device, so no later call (e.g. one inside a stream capture) sets attributes
  static std::atomic<bool> done[128] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(k_block_norm_bwd<T, V, W, THREADS, DIRECT, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (err != cudaSuccess) return err;
    done[dev].store(true, std::memory_order_release);
  }
  const int threads = round32((a.H / V + W - 1) / W), stage = bwd_stage_bytes<T, V, W, THREADS>(a.gate_full != nullptr);
  const int depth = DIRECT || 3 * stage > kSmemMax / bwd_ctas(THREADS) ? 2 : 3;
  k_block_norm_bwd<T, V, W, THREADS, DIRECT, FULL><<<unsigned(grid), threads, DIRECT ? 0 : size_t(depth) * stage, st>>>(a, depth);
  return cudaGetLastError();
}

template <typename T, int V, int W, int THREADS, bool DIRECT>
cudaError_t run_bwd(const NormArgs& a, int grid, cudaStream_t st) {
  // the usual step of rows that fill vectors gets a kernel of its own: 12% less time at 4096 x 7168
  if constexpr (V > 1 && W <= 2) {
    if (a.dh && a.dz && a.y && a.w_post && a.dx && a.dy && !a.gate_full) return run_bwd_as<T, V, W, THREADS, DIRECT, true>(a, grid, st);
  }
  return run_bwd_as<T, V, W, THREADS, DIRECT, false>(a, grid, st);
}

template <int N>
using Int = std::integral_constant<int, N>;

template <typename T, int V>
cudaError_t norm_bwd(const NormArgs& a, int* grid, cudaStream_t st) {
  const int nv = a.H / V;
  auto run = [&](auto w, auto threads, auto direct) {
    *grid = bwd_grid(a.T, a.H, threads.value, V == 1);
    return run_bwd<T, V, w.value, threads.value, direct.value>(a, *grid, st);
  };
  constexpr std::false_type staged;
  constexpr std::true_type direct;
  if (nv <= 128) return run(Int<1>(), Int<128>(), staged);
  if (nv <= 256) return run(Int<1>(), Int<256>(), staged);
  if constexpr (V > 1) {
    if (nv <= 512) return run(Int<1>(), Int<512>(), staged);
    if (nv <= 1024) return run(Int<2>(), Int<512>(), staged);
    // Rows too long for two stages in shared memory are read directly: two stages of 1792 vectors fit (four arrays), of 1024
    // threads' two no longer.  Two vectors per thread and more threads rather than four of 512 or 1024, which spill (4096 x
    // 7168 fp32 118 against 340 us, 1000 x 9216 bf16 67 against 101 us).
    if constexpr (V == 4) {
      if (nv <= 1792 && !a.gate_full) return run(Int<2>(), Int<896>(), staged);
    }
    if (nv <= 2048) return run(Int<2>(), Int<1024>(), direct);
    if constexpr (V == 4) return run(Int<4>(), Int<1024>(), direct);
    return cudaErrorInvalidValue;  // H <= 16384: at most 2048 vectors of eight
  } else {
    // single elements: four per thread, so that several rows share an SM (4000 x 1001 bf16: 43 us, two of 512 threads 52)
    if (nv <= 512) return run(Int<4>(), Int<128>(), staged);
    if (nv <= 1024) return run(Int<4>(), Int<256>(), staged);
    if (nv <= 2048) return run(Int<4>(), Int<512>(), staged);
    if (nv <= 4096) return run(Int<4>(), Int<1024>(), staged);
    if (nv <= 8192) return run(Int<8>(), Int<1024>(), std::bool_constant<sizeof(T) == 4>());
    return run(Int<16>(), Int<1024>(), direct);
  }
}

// grid NULL: forward; else backward, and the number of partial rows is stored there
template <typename T>
cudaError_t norm_of(const NormArgs& a, int* grid, cudaStream_t st) {
  constexpr int V = vec_width<T>();
  bool wide = a.H % V == 0;
  const void* ps[] = {a.x, a.y, a.w_post, a.w_next, a.gate_full, a.z, a.h, a.dz, a.dh, a.dx, a.dy, a.dgate_full};
  for (const void* p : ps) wide = wide && vec_aligned(p);
  if (grid) return wide ? norm_bwd<T, V>(a, grid, st) : norm_bwd<T, 1>(a, grid, st);
  if (a.p2r) return wide ? norm_fwd<T, V, true>(a, st) : norm_fwd<T, 1, true>(a, st);
  return wide ? norm_fwd<T, V, false>(a, st) : norm_fwd<T, 1, false>(a, st);
}

cudaError_t norm_any(const NormArgs& a, moe_dtype_t dt, int* grid, cudaStream_t st) {
  if (dt == MOE_BF16) return norm_of<__nv_bfloat16>(a, grid, st);
  if (dt == MOE_F16) return norm_of<__half>(a, grid, st);
  return norm_of<float>(a, grid, st);
}

}  // namespace

cudaError_t launch_block_norm(const moe_block_norm_t& b, const void* x, int T, int H, moe_dtype_t dt, void* z, void* h,
                              cudaStream_t st) {
  NormArgs a = args_of(b, T, H);
  a.x = x;
  a.z = z;
  a.h = h;
  return norm_any(a, dt, nullptr, st);
}

// The largest grid over the element types and alignments: the fewest threads that a row can have, an eighth of its length
// (rows of single elements have a quarter, 128 at least).
size_t block_norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  const int t = T < INT_MAX ? int(T) : INT_MAX;
  const int threads = H <= 1024 ? 128 : H <= 2048 ? 256 : 512;
  return size_t(bwd_grid(t, int(H < 16384 ? H : 16384), threads, true)) * 2 * size_t(H) * sizeof(float);
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
  int grid = 0;
  cudaError_t err = norm_any(a, dt, &grid, st);
  if (err != cudaSuccess || (!g.dw_post && !g.dw_next)) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((H + 31) / 32), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_weight_sum, static_cast<const float*>(a.part), grid, H, g.dw_post, g.dw_next);
}

}  // namespace moe
