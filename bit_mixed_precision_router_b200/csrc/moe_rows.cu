// Tokens sorted by expert and back, with routing weights, and the gradients.  With p = t*k + j
// a (token, slot) pair, r(p) = pair_to_row[p] its row (negative: the pair was dropped and has no
// row) and w_p its weight (1 where the call is unweighted):
//   sort      rows[r(p)] = w_p x[t]                      back      out[t] = sum_j w_p rows[r(p)] (+ residual[t])
//   d sort    dx[t] = sum_j w_p drows[r(p)]              d back    drows[r(p)] = w_p dout[t]
//             dw_p = <drows[r(p)], x[t]>                           dw_p = <dout[t], rows[r(p)]>
// Each gradient is the other direction plus one dot product per pair, so two kernels cover all four:
//   k_spread  token-major: reads a[t] once, writes its k rows (and reads k rows for the dots);
//   k_gather  token-major: reads k rows, writes one (and reads one more for the dots).
// Token-major needs no atomics (a token's k pairs belong to one CTA) and reads the token's row once.
// Sums run in fp32 in slot order, each result rounded once to the element type; the dots stay fp32.
// Bound by HBM: (k + 1) rows per token, (2k + 1) or (k + 2) with the dots.
//   k_route_bwd  the gradient of the softmax over the k chosen logits.
//   k_permute_cap  the stable counting sort behind it, with dropped pairs and a row limit per expert.
#include <cooperative_groups.h>

#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kRowThreads = 256;
constexpr int kSlots = 8;  // rows of a token in flight per thread
// Vectors of a row in flight per thread, of V elements each: with few rows per token, or single elements, a thread takes
// several (one row per token, 4096 x 4096 bf16: sort 15.7 -> 9.7 us; 4 x 2048 x 2047: 25 -> 13, back 32 -> 17.5).
// With eight single elements and their dots the registers run out (511 to 8191 of them, back's gradient: 20% to 50% slower).
__host__ __device__ constexpr int vectors_of(int V, int slots, bool dots) {
  return slots <= 2 ? 4 : V == 1 && slots <= 4 ? 4 : slots <= 4 ? 2 : V == 1 && slots <= kSlots && !dots ? 4 : 1;
}

// Sums of N values over the CTA (at most kRowThreads threads), in one fixed order; value j is returned to thread j < N.
// `red`: 8 N floats of shared memory.
template <int N>
MOE_DEVICE float block_sums(float (&v)[N], float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const float w = warp_sums<N>(v);
  if (lane % (32 / N) == 0) red[(lane / (32 / N)) * 8 + warp] = w;
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x < N) {
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; ++i) s += i < nw ? red[threadIdx.x * 8 + i] : 0.0f;
  }
  return s;
}

// KB: slots unrolled (k_spread: at a time; k_gather: all, k <= KB).
template <typename T, int V, bool DOT, int KB>
__global__ void __launch_bounds__(kRowThreads, DOT ? 3 : 0)
    k_spread(const T* a, const T* __restrict__ b, const float* __restrict__ w, const int32_t* __restrict__ p2r, int H, int k,
             T* __restrict__ rows, float* __restrict__ dw) {
  constexpr int U = vectors_of(V, KB, DOT);
  __shared__ float red[KB * 8];
  const int t = blockIdx.x, nv = H / V;
  const T* arow = a + size_t(t) * H;
  const int step = DOT ? int(blockDim.x) : int(blockDim.x * gridDim.y);
  const int v0 = DOT ? int(threadIdx.x) : int(blockIdx.y * blockDim.x + threadIdx.x);
  for (int j0 = 0; j0 < k; j0 += KB) {
    int row[KB];
    float wj[KB], dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const size_t p = size_t(t) * k + j0 + j;
      row[j] = j0 + j < k ? p2r[p] : -1;
      wj[j] = w && j0 + j < k ? w[p] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int v = v0; v < nv; v += U * step) {
      Pack<T, V> av[U], bv[U][KB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v + u * step >= nv) break;
        av[u] = load_vec<T, V>(arow, v + u * step);
        if (DOT) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (row[j] >= 0) bv[u][j] = load_vec_once<T, V>(b + size_t(row[j]) * H, v + u * step);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v + u * step >= nv) break;
        float f[V];
        av[u].unpack(f);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (row[j] < 0) continue;
          if (DOT) {
            float g[V];
            bv[u][j].unpack(g);
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = fmaf(f[i], g[i], dot[j]);
          }
          if (w) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = wj[j] * f[i];
            store_vec(rows + size_t(row[j]) * H, v + u * step, Pack<T, V>::of(o));
          } else {
            store_vec(rows + size_t(row[j]) * H, v + u * step, av[u]);
          }
        }
      }
    }
    if (DOT) {
      const float s = block_sums<KB>(dot, red);
      const int j = j0 + int(threadIdx.x);
      if (threadIdx.x < KB && j < k) dw[size_t(t) * k + j] = s;
      __syncthreads();
    }
  }
}

template <typename T, int V, bool DOT, int KB>
__global__ void __launch_bounds__(kRowThreads, DOT && KB <= kSlots ? 3 : 0)
    k_gather(const T* __restrict__ rows, const T* x, const float* __restrict__ w, const int32_t* __restrict__ p2r, int H, int k,
             T* out, float* __restrict__ dw) {
  constexpr int U = vectors_of(V, KB, DOT), SB = KB < kSlots ? KB : kSlots;  // slots in flight
  __shared__ float red[KB * 8];
  __shared__ int srow[KB];
  __shared__ float sw[KB];
  const int t = blockIdx.x, nv = H / V;
  if (threadIdx.x < KB) {
    const bool in = int(threadIdx.x) < k;
    const size_t p = size_t(t) * k + threadIdx.x;
    srow[threadIdx.x] = in ? p2r[p] : -1;
    sw[threadIdx.x] = in && w ? w[p] : 1.0f;
  }
  __syncthreads();
  float dot[KB];
#pragma unroll
  for (int j = 0; j < KB; ++j) dot[j] = 0.0f;
  const int step = DOT ? int(blockDim.x) : int(blockDim.x * gridDim.y);
  for (int v = DOT ? int(threadIdx.x) : int(blockIdx.y * blockDim.x + threadIdx.x); v < nv; v += U * step) {
    float acc[U][V];
    Pack<T, V> xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < V; ++i) acc[u][i] = 0.0f;
      if (x && v + u * step < nv) xv[u] = load_vec<T, V>(x + size_t(t) * H, v + u * step);
    }
#pragma unroll
    for (int j0 = 0; j0 < KB; j0 += SB) {
      if (j0 >= k) break;
      Pack<T, V> r[U][SB];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < SB; ++j)
          if (srow[j0 + j] >= 0 && v + u * step < nv) r[u][j] = load_vec_once<T, V>(rows + size_t(srow[j0 + j]) * H, v + u * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v + u * step >= nv) break;
        float xf[V];
        if (DOT) xv[u].unpack(xf);
#pragma unroll
        for (int j = 0; j < SB; ++j) {
          if (srow[j0 + j] < 0) continue;
          float f[V];
          r[u][j].unpack(f);
          const float wj = sw[j0 + j];
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u][i] = fmaf(wj, f[i], acc[u][i]);
          if (DOT) {
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j0 + j] = fmaf(xf[i], f[i], dot[j0 + j]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v + u * step >= nv) break;
      if (!DOT && x) {  // the residual, added last
        float xf[V];
        xv[u].unpack(xf);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] += xf[i];
      }
      store_vec(out + size_t(t) * H, v + u * step, Pack<T, V>::of(acc[u]));
    }
  }
  if (DOT) {
    const float s = block_sums<KB>(dot, red);
    if (threadIdx.x < KB && int(threadIdx.x) < k) dw[size_t(t) * k + threadIdx.x] = s;
  }
}

// One warp per token: dl_j = w_j (dw_j - sum_i w_i dw_i), scattered into a row of zeros.  Pairs
// are added in slot order by one lane, so an expert chosen twice gets both parts, in one order.
constexpr int kRouteWarps = 4;
__global__ void __launch_bounds__(32 * kRouteWarps) k_route_bwd(const float* __restrict__ dw, const float* __restrict__ w,
                                                                const int32_t* __restrict__ ids, int T, int E, int k,
                                                                float* __restrict__ dl) {
  extern __shared__ float smem_f[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= T) return;
  float* row = smem_f + warp * E;
  for (int e = lane; e < E; e += 32) row[e] = 0.0f;
  const size_t p = size_t(t) * k + lane;
  const float wj = lane < k ? w[p] : 0.0f, d = lane < k ? dw[p] : 0.0f;
  const int id = lane < k ? ids[p] : -1;
  const float g = wj * (d - warp_sum(wj * d));
  __syncwarp();
  for (int j = 0; j < k; ++j) {
    if (lane == j && id >= 0 && id < E) row[id] += g;
    __syncwarp();
  }
  for (int e = lane; e < E; e += 32) dl[size_t(t) * E + e] = row[e];
}

// ---------------------------------------------------------------- permutation with dropped pairs
// A stable counting sort of P pairs by expert over one cluster of C CTAs (C = 1 for small P): warp
// q of the cluster (CTA rank * NW + warp) owns pairs [q P / (C NW), (q+1) P / (C NW)).
//   1. each warp counts its pairs per expert (bin E: ids outside 0..E-1);
//   2. per expert, the counts of earlier warps (own CTA) and earlier CTAs (distributed shared
//      memory) give the pair's index inside its expert; the kept totals give the expert's first row;
//   3. a pair whose index is below the limit takes row first + index, any other is dropped: it gets
//      row -1 and follows the last kept row in sorted_pair, in ascending order.  The number of
//      dropped pairs ahead of a warp follows from the same counts.
// `cnt` is [NW][E + 1] ints of shared memory.
constexpr int kPermThreads = 1024;
constexpr int kPermCntInts = 8192;  // 32 KiB of counts: NW = min(32, 8192 / (E + 1))

// The bins of kPermAhead pairs p, p + 32, ... (all loads in flight); -1 past the end.
constexpr int kPermAhead = 4;
MOE_DEVICE void load_ids(const int32_t* ids, int p, int end, int E, int (&id)[kPermAhead]) {
#pragma unroll
  for (int r = 0; r < kPermAhead; ++r) id[r] = p + 32 * r < end ? ids[p + 32 * r] : -2;
#pragma unroll
  for (int r = 0; r < kPermAhead; ++r) id[r] = p + 32 * r >= end ? -1 : id[r] >= 0 && id[r] < E ? id[r] : E;
}

template <int C>
__global__ void __launch_bounds__(kPermThreads) k_permute_cap(const int32_t* __restrict__ ids, int P, int E, int cap,
                                                              int NW, moe_routing_t out) {
  __shared__ int cnt[kPermCntInts];
  __shared__ int tot[MOE_MAX_EXPERTS + 1];   // this CTA's pairs per bin
  __shared__ int base[MOE_MAX_EXPERTS + 1];  // pairs of the bin in earlier CTAs
  __shared__ int first[MOE_MAX_EXPERTS];     // the expert's first row
  __shared__ int dropped[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwb = blockDim.x >> 5;
  const int B = E + 1;
  const int rank = C > 1 ? int(cg::this_cluster().block_rank()) : 0;
  for (int i = threadIdx.x; i < NW * B; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int64_t q = int64_t(rank) * NW + warp, Q = int64_t(C) * NW;
  const int beg = int(q * P / Q), end = int((q + 1) * P / Q);
  int* mine = cnt + warp * B;
  if (warp < NW) {
    for (int p0 = beg; p0 < end; p0 += 32 * kPermAhead) {
      int id[kPermAhead];
      load_ids(ids, p0 + lane, end, E, id);
#pragma unroll
      for (int r = 0; r < kPermAhead; ++r)
        if (id[r] >= 0) atomicAdd(&mine[id[r]], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < B; e += blockDim.x) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < NW; ++w) {
      const int c = cnt[w * B + e];
      cnt[w * B + e] = run;
      run += c;
    }
    tot[e] = run;
  }
  if (C > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
  // pairs of bin e in earlier CTAs, and in all
  const int limit = cap > 0 ? cap : 0x7fffffff;
  int all_of[2] = {0, 0};  // B <= 1025 bins over 1024 threads
  for (int i = 0, e = threadIdx.x; e < B; e += blockDim.x, ++i) {
    int before = 0, all = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {  // all reads in flight at once
      const int v = C > 1 ? *cg::this_cluster().map_shared_rank(&tot[e], c) : tot[e];
      before += c < rank ? v : 0;
      all += v;
    }
    base[e] = before;
    all_of[i] = all;
  }
  if (C > 1)
    cg::this_cluster().sync();  // every CTA has read the totals; from here each is on its own
  else
    __syncthreads();
  for (int i = 0, e = threadIdx.x; e < B; e += blockDim.x, ++i) tot[e] = all_of[i];
  __syncthreads();
  // dropped pairs ahead of each warp: its own earlier pairs past the limit, bin E whole
  for (int w = warp; w < NW; w += nwb) {
    int s = 0;
    for (int e = lane; e < B; e += 32) {
      const int c = base[e] + cnt[w * B + e];
      s += e == E ? c : max(0, c - limit);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) dropped[w] = s;
  }
  if (warp == 0) {  // dropped[32]: kept rows
    const int per = (E + 31) / 32;
    const int b = min(E, lane * per), en = min(E, b + per);
    int sum = 0, act = 0;
    for (int e = b; e < en; ++e) {
      sum += min(tot[e], limit);
      act += tot[e] > 0;
    }
    int isum = sum, iact = act;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v1 = __shfl_up_sync(0xffffffffu, isum, d), v2 = __shfl_up_sync(0xffffffffu, iact, d);
      if (lane >= d) {
        isum += v1;
        iact += v2;
      }
    }
    int run = isum - sum, pos = iact - act;
    for (int e = b; e < en; ++e) {
      const int n = min(tot[e], limit);
      first[e] = run;
      if (rank == 0) {
        out.expert_offsets[e] = run;
        if (n > 0) out.expert_list[1 + pos] = e;
      }
      pos += n > 0;
      run += n;
    }
    if (lane == 31) {
      dropped[32] = isum;
      if (rank == 0) {
        out.expert_offsets[E] = isum;
        out.expert_list[0] = iact;
      }
    }
  }
  __syncthreads();
  if (warp >= NW) return;
  const int kept_rows = dropped[32];
  int drop_at = kept_rows + dropped[warp];
  const unsigned lt = (1u << lane) - 1u;
  for (int p0 = beg; p0 < end; p0 += 32 * kPermAhead) {
    int ahead[kPermAhead];
    load_ids(ids, p0 + lane, end, E, ahead);
#pragma unroll
    for (int r = 0; r < kPermAhead; ++r) {
      const int p = p0 + 32 * r + lane, id = ahead[r];
      const unsigned peers = __match_any_sync(0xffffffffu, id);
      int idx = 0;
      if (id >= 0) idx = base[id] + mine[id] + __popc(peers & lt);
      __syncwarp();
      if (id >= 0 && (__ffs(peers) - 1) == lane) mine[id] += __popc(peers);
      __syncwarp();
      const bool keep = id >= 0 && id < E && idx < limit;
      const unsigned lost = __ballot_sync(0xffffffffu, id >= 0 && !keep);
      if (id >= 0) {
        const int row = keep ? first[id] + idx : drop_at + __popc(lost & lt);
        out.sorted_pair[row] = p;
        out.pair_to_row[p] = keep ? row : -1;
      }
      drop_at += __popc(lost);
    }
  }
}

// ---------------------------------------------------------------- launchers
int row_threads(int nv) {  // as many threads as the row has vectors, at most kRowThreads
  const int t = (nv + 31) / 32 * 32;
  return t < kRowThreads ? t : kRowThreads;
}

template <typename T, int V, bool DOT, int KB>
cudaError_t spread_of(const RowArgs& g, cudaStream_t st) {
  const int nv = (g.H / V + vectors_of(V, KB, DOT) - 1) / vectors_of(V, KB, DOT), threads = row_threads(nv);
  const dim3 grid(unsigned(g.T), DOT ? 1u : unsigned((nv + threads - 1) / threads));
  k_spread<T, V, DOT, KB><<<grid, threads, 0, st>>>(static_cast<const T*>(g.a), static_cast<const T*>(g.b), g.w, g.p2r, g.H, g.k,
                                                    static_cast<T*>(g.out), g.dw);
  return cudaGetLastError();
}

template <typename T, int V, bool DOT, int KB>
cudaError_t gather_of(const RowArgs& g, cudaStream_t st) {
  const int nv = (g.H / V + vectors_of(V, KB, DOT) - 1) / vectors_of(V, KB, DOT), threads = row_threads(nv);
  const dim3 grid(unsigned(g.T), DOT ? 1u : unsigned((nv + threads - 1) / threads));
  k_gather<T, V, DOT, KB><<<grid, threads, 0, st>>>(static_cast<const T*>(g.a), static_cast<const T*>(g.b), g.w, g.p2r, g.H, g.k,
                                                    static_cast<T*>(g.out), g.dw);
  return cudaGetLastError();
}

template <typename T, int V, bool DOT>
cudaError_t spread(const RowArgs& g, cudaStream_t st) {
  return g.k <= 2   ? spread_of<T, V, DOT, 2>(g, st)
         : g.k <= 4 ? spread_of<T, V, DOT, 4>(g, st)
                    : spread_of<T, V, DOT, kSlots>(g, st);
}

template <typename T, int V, bool DOT>
cudaError_t gather(const RowArgs& g, cudaStream_t st) {
  return g.k <= 2        ? gather_of<T, V, DOT, 2>(g, st)
         : g.k <= 4      ? gather_of<T, V, DOT, 4>(g, st)
         : g.k <= kSlots ? gather_of<T, V, DOT, kSlots>(g, st)
                         : gather_of<T, V, DOT, MOE_MAX_TOPK>(g, st);
}

template <typename T>
cudaError_t rows_of(const RowArgs& g, bool is_spread, cudaStream_t st) {
  constexpr int V = vec_width<T>();
  // 128-bit accesses where every row starts on 16 bytes; else one element at a time
  const bool wide = g.H % V == 0 && vec_aligned(g.a) && vec_aligned(g.b) && vec_aligned(g.out);
  if (is_spread && g.dw) return wide ? spread<T, V, true>(g, st) : spread<T, 1, true>(g, st);
  if (is_spread) return wide ? spread<T, V, false>(g, st) : spread<T, 1, false>(g, st);
  if (g.dw) return wide ? gather<T, V, true>(g, st) : gather<T, 1, true>(g, st);
  return wide ? gather<T, V, false>(g, st) : gather<T, 1, false>(g, st);
}

cudaError_t rows_any(const RowArgs& g, moe_dtype_t dt, bool is_spread, cudaStream_t st) {
  if (dt == MOE_BF16) return rows_of<__nv_bfloat16>(g, is_spread, st);
  if (dt == MOE_F16) return rows_of<__half>(g, is_spread, st);
  return rows_of<float>(g, is_spread, st);
}

}  // namespace

cudaError_t launch_spread_rows(const RowArgs& g, moe_dtype_t dt, cudaStream_t st) { return rows_any(g, dt, true, st); }
cudaError_t launch_gather_sum(const RowArgs& g, moe_dtype_t dt, cudaStream_t st) { return rows_any(g, dt, false, st); }

cudaError_t launch_route_bwd(const float* dw, const float* w, const int32_t* ids, int T, int E, int k, float* dlogits,
                             cudaStream_t st) {
  k_route_bwd<<<unsigned((T + kRouteWarps - 1) / kRouteWarps), 32 * kRouteWarps, kRouteWarps * E * sizeof(float), st>>>(
      dw, w, ids, T, E, k, dlogits);
  return cudaGetLastError();
}

cudaError_t launch_permute_capacity(const int32_t* ids, int P, int E, int cap, const moe_routing_t& out,
                                    cudaStream_t st) {
  const int most = kPermCntInts / (E + 1) < 32 ? kPermCntInts / (E + 1) : 32;
  const int C = P > 1024 ? 8 : 1;  // pairs enough for several CTAs (4096 pairs: one CTA 12.3, eight 5.7 us)
  const int want = (P + 32 * C - 1) / (32 * C);
  const int NW = want < most ? want : most;
  // the bins are walked by all threads, two per thread at most
  const int bins = ((E + 2) / 2 + 31) / 32 * 32;
  const int threads = 32 * NW > bins ? 32 * NW : bins;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(C));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(C);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (C == 1) return cudaLaunchKernelEx(&cfg, k_permute_cap<1>, ids, P, E, cap, NW, out);
  return cudaLaunchKernelEx(&cfg, k_permute_cap<8>, ids, P, E, cap, NW, out);
}

}  // namespace moe
