// Matrix-vector products with 4-bit weights and group scales: y[t][n] = sum_k x[t][k] w[n][k] for a few
// tokens, w one W4G128 or NVFP4 matrix as the quantisers write it; SwiGLU or a residual in the epilogue.
//
// Bound by the weight stream (half a byte per weight plus scales) up to some 32 tokens, so each weight is
// read once per pass of 64 tokens, dequantised in registers, and meets all of the pass's tokens on
// mma.sync m16n8k16 (16 weight rows x 16 k x 8 tokens; with one token a tcgen05 tile would be 1/128
// used and its operands would have to be written to shared memory first).
//
// One warp owns 16 rows.  Lane (g, c) = (lane / 4, lane % 4) reads 16 bytes (32 codes) of rows g and g+8 per
// group of 128: four lanes cover a row's group, and word j of the 16 bytes feeds two MMA steps.  The k order
// inside a group is free as long as both operands agree, so the codes are used as the words hold them
// (nibbles i and i+4 make a pair) and the tokens are staged in that order instead:
//   - W4: pair = bf16/fp16 128|u or 1024|u by one lop3, minus 136 or 1032: q exactly.  Products q x are
//     exact in fp32; a group's sum is scaled once by its bf16 scale in fp32, so no weight is rounded.
//   - NVFP4: e2m1 * e4m3 has at most 2 + 4 significant bits: exact in bf16 and fp16; the scale differs per lane
//     within an MMA step, so it multiplies the weights; the per-tensor scale multiplies the result.
// Accumulation is fp32 throughout: within a group by the tensor core (whose additions truncate), the groups by
// rounded additions, so the error does not grow with K; results are rounded once.
//
// Eight warps per CTA, RW of them on different rows and KW = 8 / RW on different groups of the same rows, and S
// CTAs of a cluster on different parts of K: enough warps for the memory system also when N is small.  The
// partial sums are joined in shared memory, across the cluster through distributed shared memory, in a fixed
// order: deterministic, without a workspace and in one launch.
#pragma once

#include <cooperative_groups.h>

#include <atomic>

#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {

struct LinearArgs {
  const uint8_t* w;      // [N][K/2]
  const uint8_t* scale;  // bf16 [N][K/128] or e4m3 [N][K/16]
  const float* gscale;   // NVFP4: [1]
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  int y_dtype;
  int T, N, K, swiglu;
  int S;
};

namespace {

namespace cg = cooperative_groups;

constexpr int kPassTokens = 64;  // tokens per pass over the weights


// The eight W4 codes of a word as q = u - 8, pairs p of nibbles (p, p + 4).  A code is put into the mantissa of a
// constant whose last place is one unit: bf16 128 + u, fp16 1024 + u; fp16 has room for a nibble four bits up
// (1024 + 16 u, then times 1/16), which saves two shifts.
MOE_DEVICE uint32_t and_or(uint32_t v, uint32_t mask, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(magic));
  return d;
}
template <bool BF16>
MOE_DEVICE void w4_word(uint32_t word, uint32_t (&q)[4]) {
  if (BF16) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(q[p]) : "r"(and_or(word >> (4 * p), 0x000F000Fu, 0x43004300u)), "r"(0x43084308u));
  } else {
#pragma unroll
    for (int p = 0; p < 4; p += 2) {
      const uint32_t w = word >> (4 * p);
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(q[p]) : "r"(and_or(w, 0x000F000Fu, 0x64006400u)), "r"(0x64086408u));
      asm("fma.rn.f16x2 %0, %1, %2, %3;"  // / 16 - 72
          : "=r"(q[p + 1])
          : "r"(and_or(w, 0x00F000F0u, 0x64006400u)), "r"(0x2C002C00u), "r"(0xD480D480u));
    }
  }
}

// Pair i of a word of E2M1 codes times their block's scale.  fp16: pairs are nibbles (2i, 2i + 1).  bf16: nibbles (i, i + 4);
// the code's magnitude is placed on the exponent's and mantissa's low bits (its value times 2^-126), and
// the scale carries 2^118, so the product is the weight times 2^-8.
template <bool BF16>
MOE_DEVICE uint32_t e2m1_pair(uint32_t word, int i, uint32_t scale2) {
  uint32_t d;
  if (BF16) {
    const uint32_t mag = (i < 2 ? word << (6 - 4 * i) : word >> (4 * i - 6)) & 0x01C001C0u;
    const uint32_t v = ((word << (12 - 4 * i)) & 0x80008000u) | mag;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(scale2));
  } else {
    d = hmul2(e2m1x2_to_h2((word >> (8 * i)) & 0xFFu), scale2);
  }
  return d;
}

// an E4M3 block scale as the multiplier of e2m1_pair
template <bool BF16>
MOE_DEVICE uint32_t e4m3_pair(uint32_t byte) {
  const uint32_t h2 = e4m3_to_h2(byte);
  if (!BF16) return h2;
  const float f = __half2float(__ushort_as_half(uint16_t(h2))) * 0x1p118f;
  const uint32_t b = float_to_bf16_bits(f);
  return b | (b << 16);
}

template <bool BF16>
MOE_DEVICE void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    mma_bf16(d, a0, a1, a2, a3, b0, b1);
  else
    mma_f16(d, a0, a1, a2, a3, b0, b1);
}

// 16 bytes global -> shared, asynchronous, L1 bypassed; the issuing thread sees them after cp_wait
MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEVICE void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEVICE void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The shape of a CTA for NT token tiles (8 tokens each) per pass, KW warps on different groups of the same rows.
template <int NT, int KW>
struct Lin {
  static constexpr int kWarps = NT <= 2 ? 8 : 16;             // more rows per staged token where tokens are many
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRW = kWarps / KW;                     // warps on different rows
  static constexpr int kCG = NT == 1 ? 8 : NT == 8 ? 2 : 4;   // groups of K staged at a time: four 16-byte units a thread
  static constexpr int kCI = kCG / KW;                        // of them each warp's
  static constexpr int kTokStride = kCG * 256 + 64;           // bytes per staged token; 64: no bank conflicts
  static constexpr int kTokBytes = 8 * NT * kTokStride;
  static constexpr int kDepth = 4;                            // groups of weights in flight per warp
  static constexpr int kRing = kDepth * 1024;                 // bytes per warp
  static constexpr int kSmem = 2 * kTokBytes + kWarps * kRing;
  static constexpr int kCtas = NT == 1 ? 3 : NT == 2 ? 2 : 1; // per SM
};

template <bool BF16, int FMT, int NT, int KW>
__global__ void __launch_bounds__(Lin<NT, KW>::kThreads, Lin<NT, KW>::kCtas) k_linear_w4(LinearArgs a) {
  using L = Lin<NT, KW>;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr bool W4 = FMT == MOE_FMT_W4G128;
  constexpr int CG = L::kCG, CI = L::kCI, STRIDE = L::kTokStride, LD = 8 * NT, RW = L::kRW, D = L::kDepth;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int wr = warp / KW, kw = warp % KW;
  const int part = blockIdx.y;  // K part of this CTA (its rank in the cluster)
  const int t0 = blockIdx.z * kPassTokens, nt = min(a.T - t0, 8 * NT);
  const int G = a.K / 128;
  const int gb = int(int64_t(part) * G / a.S), ge = int(int64_t(part + 1) * G / a.S);
  const int chunks = (ge - gb + CG - 1) / CG;
  const int ni = ge - gb > kw ? (ge - gb - kw + KW - 1) / KW : 0;  // this warp's groups: gb + kw + i KW

  // rows of this lane; rows past the end repeat the last one and are not stored
  const int tile = blockIdx.x * RW + wr, half = a.N / 2;
  const int r0 = a.swiglu ? min(tile * 8 + g, half - 1) : min(tile * 16 + g, a.N - 1);
  const int r1 = a.swiglu ? r0 + half : min(tile * 16 + g + 8, a.N - 1);
  const uint8_t* w0 = a.w + size_t(r0) * (a.K / 2) + c * 16 + size_t(gb + kw) * 64;
  const uint8_t* w1 = a.w + size_t(r1) * (a.K / 2) + c * 16 + size_t(gb + kw) * 64;
  // W4: one bf16 per group; NVFP4: eight bytes per group, two of them (32 codes) this lane's
  constexpr int SB = W4 ? 2 : 8;
  const uint8_t* s0 = a.scale + (size_t(r0) * G + gb + kw) * SB + (W4 ? 0 : 2 * c);
  const uint8_t* s1 = a.scale + (size_t(r1) * G + gb + kw) * SB + (W4 ? 0 : 2 * c);

  // weights: a ring of D groups per warp; each lane copies and reads its own 2 x 16 bytes of a slot
  uint8_t* ring = smem + 2 * L::kTokBytes + warp * L::kRing + lane * 16;
  const uint32_t ring_at = smem_addr(ring);
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (d < ni) {
      cp_async16(ring_at + d * 1024, w0 + d * (KW * 64));
      cp_async16(ring_at + d * 1024 + 512, w1 + d * (KW * 64));
    }
    cp_commit();
  }
  // scales: registers, SR groups ahead
  constexpr int SR = CI >= 4 ? 4 : 2;
  uint32_t sa[SR] = {}, sb[SR] = {};
#pragma unroll
  for (int d = 0; d < SR; ++d) {
    if (d < ni) {
      sa[d] = __ldg(reinterpret_cast<const uint16_t*>(s0 + d * (KW * SB)));
      sb[d] = __ldg(reinterpret_cast<const uint16_t*>(s1 + d * (KW * SB)));
    }
  }

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

  // tokens: chunks of CG groups, double buffered; the next chunk's units are in registers while this one is used.
  // A thread's four units are 16 bytes (8 elements) u of tokens t, t + TS, t + 2 TS, t + 3 TS.
  constexpr int TS = L::kThreads / (CG * 16);
  const int tu = threadIdx.x % (CG * 16), tt = threadIdx.x / (CG * 16);
  const uint16_t* xp = static_cast<const uint16_t*>(a.x) + size_t(t0 + tt) * a.ldx + size_t(gb) * 128 + tu * 8;
  const int64_t xrow = a.ldx * TS;
  // unit u of a group goes to word j = u % 4 of lane c = u / 4
  uint8_t* const tok_at = smem + tt * STRIDE + (tu >> 4) * 256 + (tu & 3) * 64 + ((tu >> 2) & 3) * 16;
  uint4 xu[4];
  auto load_tokens = [&](int ch) {
    if (gb + ch * CG + (tu >> 4) >= ge) return;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (tt + r * TS < nt) xu[r] = *reinterpret_cast<const uint4*>(xp + r * xrow + ch * (CG * 128));
  };
  auto store_tokens = [&](int ch) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint4 o = make_uint4(0, 0, 0, 0);  // tokens past the last one are zeros
      if (tt + r * TS < nt) {
        o = xu[r];
        if (W4 || BF16) {  // pairs (i, i + 4)
          o.x = __byte_perm(xu[r].x, xu[r].z, 0x5410);
          o.y = __byte_perm(xu[r].x, xu[r].z, 0x7632);
          o.z = __byte_perm(xu[r].y, xu[r].w, 0x5410);
          o.w = __byte_perm(xu[r].y, xu[r].w, 0x7632);
        }
      } else if (ch > 1) {
        continue;  // both buffers hold their zeros
      }
      *reinterpret_cast<uint4*>(tok_at + (ch & 1) * L::kTokBytes + r * TS * STRIDE) = o;
    }
  };
  load_tokens(0);
  store_tokens(0);
  __syncthreads();
  int i0 = 0;  // first group of the chunk
  for (int ch = 0; ch < chunks; ++ch, i0 += CI) {
    if (ch + 1 < chunks) load_tokens(ch + 1);
    const uint8_t* xs = smem + (ch & 1) * L::kTokBytes + kw * 256 + c * 16 + g * STRIDE;
    const int slot0 = CI >= D ? 0 : (i0 & (D - 1)) * 1024;  // CI divides D or is a multiple of it
#pragma unroll
    for (int ii = 0; ii < CI; ++ii) {
      if (i0 + ii >= ni) break;
      const int slot = slot0 + (ii & (D - 1)) * 1024;
      cp_wait<D - 1>();
      const uint4 wa = *reinterpret_cast<const uint4*>(ring + slot);
      const uint4 wb = *reinterpret_cast<const uint4*>(ring + slot + 512);
      const uint32_t ua[4] = {wa.x, wa.y, wa.z, wa.w}, ub[4] = {wb.x, wb.y, wb.z, wb.w};
      const uint32_t qa = sa[ii % SR], qb = sb[ii % SR];
      uint32_t pa[4][4], pb[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (W4) {
          w4_word<BF16>(ua[j], pa[j]);
          w4_word<BF16>(ub[j], pb[j]);
        } else {
          const uint32_t fa = e4m3_pair<BF16>((qa >> (j < 2 ? 0 : 8)) & 0xFFu);
          const uint32_t fb = e4m3_pair<BF16>((qb >> (j < 2 ? 0 : 8)) & 0xFFu);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            pa[j][p] = e2m1_pair<BF16>(ua[j], p, fa);
            pb[j][p] = e2m1_pair<BF16>(ub[j], p, fb);
          }
        }
      }
      // the slot just read (its words are in registers) takes the group D ahead
      if (i0 + ii + D < ni) {
        cp_async16(ring_at + slot, w0 + (ii + D) * (KW * 64));
        cp_async16(ring_at + slot + 512, w1 + (ii + D) * (KW * 64));
      }
      cp_commit();
      if (CI == 1) {
        sa[0] = sa[1];
        sb[0] = sb[1];
      }
      if (i0 + ii + SR < ni) {
        sa[CI == 1 ? 1 : ii % SR] = __ldg(reinterpret_cast<const uint16_t*>(s0 + (ii + SR) * (KW * SB)));
        sb[CI == 1 ? 1 : ii % SR] = __ldg(reinterpret_cast<const uint16_t*>(s1 + (ii + SR) * (KW * SB)));
      }
      const float fa = W4 ? __uint_as_float(qa << 16) : 1.0f, fb = W4 ? __uint_as_float(qb << 16) : 1.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 b = *reinterpret_cast<const uint4*>(xs + n * 8 * STRIDE + ii * (KW * 256) + j * 64);
          mma16<BF16>(d, pa[j][0], pb[j][0], pa[j][1], pb[j][1], b.x, b.y);
          mma16<BF16>(d, pa[j][2], pb[j][2], pa[j][3], pb[j][3], b.z, b.w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = W4 ? fmaf(e < 2 ? fa : fb, d[e], acc[n][e]) : acc[n][e] + d[e];
      }
    }
    w0 += CI * KW * 64;
    w1 += CI * KW * 64;
    s0 += CI * KW * SB;
    s1 += CI * KW * SB;
    if (ch + 1 < chunks) store_tokens(ch + 1);
    __syncthreads();
  }
  // partial sums: [KW][RW * 16][LD] floats (every copy into the ring has landed: the last groups were waited for)
  float* red = reinterpret_cast<float*>(smem);
  constexpr int RB = RW * 16;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* o = red + (kw * RB + wr * 16 + g) * LD + 8 * n + 2 * c;
    *reinterpret_cast<float2*>(o) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(o + 8 * LD) = make_float2(acc[n][2], acc[n][3]);
  }
  cg::cluster_group cl = cg::this_cluster();
  if (a.S > 1)
    cl.sync();
  else
    __syncthreads();
  // each CTA of the cluster finishes its share of the rows
  const int FR = a.swiglu ? RB / 2 : RB, M = a.swiglu ? half : a.N;
  const int fb = part * FR / a.S, fn = (part + 1) * FR / a.S - fb;
  float post = 1.0f;
  if (!W4) post = *a.gscale * (BF16 ? 256.0f : 1.0f);
  for (int q = threadIdx.x; q < fn * nt; q += L::kThreads) {
    const int f = fb + q % fn, t = q / fn;
    const int n = blockIdx.x * FR + f;
    if (n >= M) continue;
    const int m = a.swiglu ? (f >> 3) * 16 + (f & 7) : f;
    float v = 0.0f, up = 0.0f;
    for (int s = 0; s < a.S; ++s) {
      const float* rs = a.S > 1 ? cl.map_shared_rank(red, s) : red;
      for (int k = 0; k < KW; ++k) {
        v += rs[(k * RB + m) * LD + t];
        if (a.swiglu) up += rs[(k * RB + m + 8) * LD + t];
      }
    }
    v *= post;
    if (a.swiglu) v = silu(v) * (up * post);
    const size_t tr = size_t(t0 + t);
    if (a.y_dtype == MOE_F32) {
      if (a.residual) v += static_cast<const float*>(a.residual)[tr * a.ldr + n];
      static_cast<float*>(a.y)[tr * a.ldy + n] = v;
    } else if (a.y_dtype == MOE_BF16) {
      if (a.residual) v += to_float(static_cast<const __nv_bfloat16*>(a.residual)[tr * a.ldr + n]);
      static_cast<__nv_bfloat16*>(a.y)[tr * a.ldy + n] = from_float<__nv_bfloat16>(v);
    } else {
      if (a.residual) v += to_float(static_cast<const __half*>(a.residual)[tr * a.ldr + n]);
      static_cast<__half*>(a.y)[tr * a.ldy + n] = from_float<__half>(v);
    }
  }
  if (a.S > 1) cl.sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------- launcher
template <bool BF16, int FMT, int NT, int KW>
cudaError_t run_linear(const LinearArgs& a, cudaStream_t st) {
  using L = Lin<NT, KW>;
  static_assert(L::kWarps * 16 * 8 * NT * int(sizeof(float)) <= 2 * L::kTokBytes, "the partial sums reuse the token stage");
  // raised once per device, so no later call (e.g. one inside a stream capture) sets attributes
  static std::atomic<bool> done[128] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(k_linear_w4<BF16, FMT, NT, KW>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (err != cudaSuccess) return err;
    done[dev].store(true, std::memory_order_release);
  }
  const int tiles = (a.N + 15) / 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((tiles + L::kRW - 1) / L::kRW), unsigned(a.S), unsigned((a.T + kPassTokens - 1) / kPassTokens));
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = unsigned(a.S);
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear_w4<BF16, FMT, NT, KW>, a);
}

}  // namespace

template <bool BF16, int FMT>
cudaError_t pick_linear(LinearArgs a, cudaStream_t st) {
  const int tok = a.T < kPassTokens ? a.T : kPassTokens;
  const int NT = tok <= 8 ? 1 : tok <= 16 ? 2 : tok <= 32 ? 4 : 8;
  // split K until there are warps enough for the machine, two groups per warp at least: first among the
  // warps of a CTA, then over the CTAs of a cluster
  const int tiles = (a.N + 15) / 16, G = a.K / 128, want = 148 * 16;
  const int kw_most = NT == 1 ? 8 : NT == 8 ? 2 : 4;
  int KW = 1, S = 1;
  while (KW < kw_most && tiles * KW < want && KW * 4 <= G) KW *= 2;
  while (S < 8 && int64_t(tiles) * KW * S < want && KW * S * 4 <= G) S *= 2;
  a.S = S;
  // LIN_OVERRIDE
  switch (NT * 16 + KW) {
    case 1 * 16 + 1: return run_linear<BF16, FMT, 1, 1>(a, st);
    case 1 * 16 + 2: return run_linear<BF16, FMT, 1, 2>(a, st);
    case 1 * 16 + 4: return run_linear<BF16, FMT, 1, 4>(a, st);
    case 1 * 16 + 8: return run_linear<BF16, FMT, 1, 8>(a, st);
    case 2 * 16 + 1: return run_linear<BF16, FMT, 2, 1>(a, st);
    case 2 * 16 + 2: return run_linear<BF16, FMT, 2, 2>(a, st);
    case 2 * 16 + 4: return run_linear<BF16, FMT, 2, 4>(a, st);
    case 4 * 16 + 1: return run_linear<BF16, FMT, 4, 1>(a, st);
    case 4 * 16 + 2: return run_linear<BF16, FMT, 4, 2>(a, st);
    case 4 * 16 + 4: return run_linear<BF16, FMT, 4, 4>(a, st);
    case 8 * 16 + 1: return run_linear<BF16, FMT, 8, 1>(a, st);
    case 8 * 16 + 2: return run_linear<BF16, FMT, 8, 2>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
