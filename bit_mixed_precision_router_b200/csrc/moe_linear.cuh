// Matrix-vector products with 4-bit weights and group scales: y[t][n] = sum_k x[t][k] w[n][k], w one W4G128 or NVFP4
// matrix as the quantisers write it, SwiGLU or a residual in the epilogue.  This kernel serves up to 16 tokens, and small
// matrices in passes of 16; the rest goes to the tcgen05 kernel (moe_linear_umma.cuh).
//
// Bound by the weight stream (half a byte per weight plus scales): each weight is read once, dequantised in registers, and
// meets all tokens on mma.sync m16n8k16 (16 weight rows x 16 k x 8 tokens).  A tcgen05 tile would be mostly empty, and its
// operand has to be written to tensor memory first: a group's eight MMAs take about 0.4 us there whatever the tokens.
//
// One warp owns 16 rows.  Lane (g, c) = (lane / 4, lane % 4) reads 16 bytes (32 codes) of rows g and g+8 per group of 128:
// four lanes cover a row's group, and word j of the 16 bytes feeds two MMA steps.  The k order inside a group is free as long
// as both operands agree, so the codes are used as the words hold them (nibbles i and i+4 make a pair) and the tokens are
// staged in that order instead:
//   - W4: pair = bf16/fp16 128|u or 1024|u by one lop3, minus 136 or 1032: q exactly.  Products q x are exact in fp32; a
//     group's sum is scaled once by its bf16 scale in fp32, so no weight is rounded.
//   - NVFP4: e2m1 * e4m3 has at most 2 + 4 significant bits: exact in bf16 and fp16; the scale differs per lane within an MMA
//     step, so it multiplies the weights; the per-tensor scale multiplies the result.
// Accumulation is fp32 throughout: within a group by the tensor core (whose additions truncate), the groups by rounded
// additions, so the error does not grow with K; results are rounded once.
//
// Eight warps per CTA, RW of them on different rows and KW = 8 / RW on different groups of the same rows, and S CTAs of a
// cluster on different parts of K: enough warps for the memory system also when N is small.  The partial sums are joined in
// shared memory, across the cluster through distributed shared memory, in a fixed order: deterministic, without a workspace
// and in one launch.
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

MOE_DEVICE void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
MOE_DEVICE void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Bytes of finish_linear's shared memory: the CTA's partial sums and what its cluster sends it.
__host__ __device__ constexpr int finish_bytes(int KW, int RB, int LD) { return (KW * RB + RB + 16) * LD * 4; }

// Joins the partial sums red[KW][RB][LD] (rows, tokens) of this CTA, then those of the cluster's CTAs in rank order, applies
// the epilogue and stores.  Each CTA finishes its share of the rows; the others send it theirs (stores into its shared
// memory, which do not wait, behind one cluster barrier; reading them from there took longer than the products of a small
// matrix).  With SwiGLU the rows alternate: UP gate rows, then their UP up rows.
template <int KW, int RB, int LD, int UP>
MOE_DEVICE void finish_linear(const LinearArgs& a, float* red, int part, int t0, int nt, float post) {
  const int S = a.S, sw = a.swiglu ? 1 : 0;
  const int FR = RB >> sw, M = a.N >> sw, FS = (FR + S - 1) / S;
  if (S > 1) cluster_arrive();  // this CTA's rings are free: its cluster may write
  __syncthreads();
  float* recv = red + KW * RB * LD;  // [S][gate, up][FS][LD]
  if (S > 1) {
    cluster_wait();
    cg::cluster_group cl = cg::this_cluster();
    for (int q = threadIdx.x; q < RB * nt; q += blockDim.x) {
      const int m = q % RB, t = q / RB;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) v += red[(k * RB + m) * LD + t];
      const int f = sw ? (m / (2 * UP)) * UP + m % UP : m, up = sw ? (m / UP) & 1 : 0;
      const int to = ((f + 1) * S - 1) / FR;  // the last CTA whose first row, to * FR / S, is not past f
      cl.map_shared_rank(recv, to)[(((part << sw) + up) * FS + f - to * FR / S) * LD + t] = v;
    }
    cluster_arrive();
    cluster_wait();
  }
  const int fb = part * FR / S, fn = (part + 1) * FR / S - fb;
  for (int q = threadIdx.x; q < fn * nt; q += blockDim.x) {
    const int f = q % fn, t = q / fn;
    const int n = blockIdx.x * FR + fb + f;
    if (n >= M) continue;
    float v = 0.0f, up = 0.0f;
    if (S > 1) {
      for (int s = 0; s < S; ++s) {
        v += recv[((s << sw) * FS + f) * LD + t];
        if (sw) up += recv[((s * 2 + 1) * FS + f) * LD + t];
      }
    } else {
      const int m = sw ? (f / UP) * (2 * UP) + f % UP : f;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        v += red[(k * RB + m) * LD + t];
        if (sw) up += red[(k * RB + m + UP) * LD + t];
      }
    }
    v *= post;
    if (sw) v = silu(v) * (up * post);
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
}

// The shape of a CTA for NT token tiles (8 tokens each) per pass, KW warps on different groups of the same rows.
template <int NT, int KW>
struct Lin {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRW = kWarps / KW;                     // warps on different rows
  static constexpr int kCG = NT == 1 ? 8 : 4;                // groups of K staged at a time: four 16-byte units a thread
  static constexpr int kCI = kCG / KW;                        // of them each warp's
  static constexpr int kTokStride = kCG * 256 + 64;           // bytes per staged token; 64: no bank conflicts
  static constexpr int kTokBytes = 8 * NT * kTokStride;
  // groups of weights in flight per warp; with three CTAs per SM every one more is taken from L1, which holds the scales' lines
  // (50304 x 7168, 1 token: two 44, four 49 us before the scales were read as vectors); launches of one CTA per SM have the same
  static constexpr int kDepth = NT == 1 ? 2 : 4;
  static constexpr int kRing = kDepth * 1024;                 // bytes per warp
  static constexpr int kSmem = 2 * kTokBytes + kWarps * kRing;
  static constexpr int kCtas = NT == 1 ? 3 : 2;           // per SM
};

// bf16 scale i of a vector of them
MOE_DEVICE float scale_of(const uint4& v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return i & 1 ? bf16_hi(w) : bf16_lo(w);
}
MOE_DEVICE float scale_of(const uint2& v, int i) { return i & 1 ? bf16_hi(i < 2 ? v.x : v.y) : bf16_lo(i < 2 ? v.x : v.y); }
MOE_DEVICE float scale_of(uint32_t, int) { return 0.0f; }

// VS: a chunk's scales of a row are one aligned vector (W4, KW = 1): one load where single scales took a sector each from
// L2, L1 being shared memory's (50304 x 7168: 1 token 49 -> 44 us, 16 tokens 68 -> 64 us).
template <bool BF16, int FMT, int NT, int KW, bool VS>
__global__ void __launch_bounds__(Lin<NT, KW>::kThreads, Lin<NT, KW>::kCtas) k_linear_w4(LinearArgs a) {
  using L = Lin<NT, KW>;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr bool W4 = FMT == MOE_FMT_W4G128;
  constexpr int CG = L::kCG, CI = L::kCI, STRIDE = L::kTokStride, LD = 8 * NT, RW = L::kRW, D = L::kDepth;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int wr = warp / KW, kw = warp % KW;
  const int part = blockIdx.y;  // K part of this CTA (its rank in the cluster)
  const int t0 = blockIdx.z * (8 * NT), nt = min(a.T - t0, 8 * NT);  // this pass's tokens
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
  // groups copied together: with two tiles of tokens the two halves of the rows' 128-byte lines
  constexpr int PAIR = NT == 2 && CI >= 2 ? 2 : 1;
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (d < ni) {
      cp_async16(ring_at + d * 1024, w0 + d * (KW * 64));
      cp_async16(ring_at + d * 1024 + 512, w1 + d * (KW * 64));
    }
    if (d % PAIR == PAIR - 1) cp_commit();
  }
  // scales: a chunk ahead as one vector per row, or SR groups ahead in registers
  using ScaleVec = typename RawOf<VS ? 2 * CG : 4>::type;
  ScaleVec va = {}, vb = {}, na = {}, nb = {};
  constexpr int SR = CI >= 4 ? 4 : 2;
  uint32_t sa[SR] = {}, sb[SR] = {};
  if (VS) {
    na = __ldg(reinterpret_cast<const ScaleVec*>(s0));
    nb = __ldg(reinterpret_cast<const ScaleVec*>(s1));
  } else {
#pragma unroll
    for (int d = 0; d < SR; ++d) {
      if (d < ni) {
        sa[d] = __ldg(reinterpret_cast<const uint16_t*>(s0 + d * (KW * SB)));
        sb[d] = __ldg(reinterpret_cast<const uint16_t*>(s1 + d * (KW * SB)));
      }
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
    if (VS) {
      va = na;
      vb = nb;
      if (ch + 1 < chunks) {
        na = __ldg(reinterpret_cast<const ScaleVec*>(s0 + CI * SB));
        nb = __ldg(reinterpret_cast<const ScaleVec*>(s1 + CI * SB));
      }
    }
#pragma unroll
    for (int ii = 0; ii < CI; ++ii) {
      if (i0 + ii >= ni) break;
      const int slot = slot0 + (ii & (D - 1)) * 1024;
      if (ii % PAIR == 0) cp_wait<D / PAIR - 1>();
      const uint4 wa = *reinterpret_cast<const uint4*>(ring + slot);
      const uint4 wb = *reinterpret_cast<const uint4*>(ring + slot + 512);
      const uint32_t ua[4] = {wa.x, wa.y, wa.z, wa.w}, ub[4] = {wb.x, wb.y, wb.z, wb.w};
      const uint32_t qa = sa[ii % SR], qb = sb[ii % SR];
      // The operands of word j; with one tile of tokens all four words are dequantised first (10% less time at
      // 50304 x 7168, 1 token), with more each word meets its tokens at once, which needs fewer registers (6% less with 16
      // tokens).
      constexpr int HELD = NT == 1 ? 4 : 1;
      uint32_t pa[HELD][4], pb[HELD][4];
      auto dequantise = [&](int j) {
        if (W4) {
          w4_word<BF16>(ua[j], pa[j % HELD]);
          w4_word<BF16>(ub[j], pb[j % HELD]);
        } else {
          const uint32_t fa = e4m3_pair<BF16>((qa >> (j < 2 ? 0 : 8)) & 0xFFu);
          const uint32_t fb = e4m3_pair<BF16>((qb >> (j < 2 ? 0 : 8)) & 0xFFu);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            pa[j % HELD][p] = e2m1_pair<BF16>(ua[j], p, fa);
            pb[j % HELD][p] = e2m1_pair<BF16>(ub[j], p, fb);
          }
        }
      };
      if (HELD == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) dequantise(j);
      }
      // the slots just read (their words are in registers) take the groups D ahead
      if (ii % PAIR == PAIR - 1) {
#pragma unroll
        for (int b = PAIR - 1; b >= 0; --b) {
          if (i0 + ii - b + D < ni) {
            cp_async16(ring_at + slot - b * 1024, w0 + (ii - b + D) * (KW * 64));
            cp_async16(ring_at + slot - b * 1024 + 512, w1 + (ii - b + D) * (KW * 64));
          }
        }
        cp_commit();
      }
      if (!VS && CI == 1) {
        sa[0] = sa[1];
        sb[0] = sb[1];
      }
      if (!VS && i0 + ii + SR < ni) {
        sa[CI == 1 ? 1 : ii % SR] = __ldg(reinterpret_cast<const uint16_t*>(s0 + (ii + SR) * (KW * SB)));
        sb[CI == 1 ? 1 : ii % SR] = __ldg(reinterpret_cast<const uint16_t*>(s1 + (ii + SR) * (KW * SB)));
      }
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (HELD == 1) dequantise(j);
        const uint32_t(&ra)[4] = pa[j % HELD], (&rb)[4] = pb[j % HELD];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 b = *reinterpret_cast<const uint4*>(xs + n * 8 * STRIDE + ii * (KW * 256) + j * 64);
          mma16<BF16>(d[n], ra[0], rb[0], ra[1], rb[1], b.x, b.y);
          mma16<BF16>(d[n], ra[2], rb[2], ra[3], rb[3], b.z, b.w);
        }
      }
      const float fa = VS ? scale_of(va, ii) : W4 ? __uint_as_float(qa << 16) : 1.0f;
      const float fb = VS ? scale_of(vb, ii) : W4 ? __uint_as_float(qb << 16) : 1.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = W4 ? fmaf(e < 2 ? fa : fb, d[n][e], acc[n][e]) : acc[n][e] + d[n][e];
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
  finish_linear<KW, RB, LD, 8>(a, red, part, t0, nt, W4 ? 1.0f : *a.gscale * (BF16 ? 256.0f : 1.0f));
}

// ---------------------------------------------------------------- launcher
template <bool BF16, int FMT, int NT, int KW, bool VS = false>
cudaError_t run_linear(const LinearArgs& a, cudaStream_t st) {
  using L = Lin<NT, KW>;
  static_assert(finish_bytes(KW, L::kRW * 16, 8 * NT) <= L::kSmem, "the partial sums reuse the stage and the rings");
  // raised once per device, so no later call (e.g. one inside a stream capture) sets attributes
  static std::atomic<bool> done[128] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(k_linear_w4<BF16, FMT, NT, KW, VS>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (err != cudaSuccess) return err;
    done[dev].store(true, std::memory_order_release);
  }
  const int tiles = (a.N + 15) / 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((tiles + L::kRW - 1) / L::kRW), unsigned(a.S), unsigned((a.T + 8 * NT - 1) / (8 * NT)));
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
  return cudaLaunchKernelEx(&cfg, k_linear_w4<BF16, FMT, NT, KW, VS>, a);
}

}  // namespace

// Where K is split: warps on the same rows (KW), then CTAs of a cluster (S).  The machine wants at least a
// hundred CTAs, and rows that share their staged tokens want to be many per CTA.  Up to 2048 k the warps of a CTA split a
// group each before a cluster does (joining a cluster costs about 0.4 us); longer rows leave the warps longer runs when the
// cluster splits first.  Measured at 512 .. 50304 rows of 2048 .. 7168 k; against the best of all splits at most 8% slower.
template <bool BF16, int FMT>
cudaError_t pick_linear(LinearArgs a, cudaStream_t st) {
  const int NT = a.T <= 8 ? 1 : 2, kw_most = NT == 1 ? 8 : 4;
  const int tiles = (a.N + 15) / 16, G = a.K / 128, enough = 100;
  const int passes = (a.T + 15) / 16;
  auto blocks = [&](int kw) { return (tiles + 8 / kw - 1) / (8 / kw) * passes; };
  int KW = 1, S = 1;
  if (G <= 16) {
    while (KW < kw_most && blocks(KW) < enough && KW * 2 <= G) KW *= 2;
    while (S < 8 && blocks(KW) * S < enough && KW * S * 4 <= G) S *= 2;
  } else {
    while (KW < kw_most && blocks(KW) * 4 < enough) KW *= 2;
    const int most = NT == 1 ? 444 : 148;  // CTAs: three per SM, or one
    while (S < 4 && blocks(KW) * S * 2 <= most) S *= 2;
  }
  a.S = S;
  // every part of K starts a chunk's scales on a vector's boundary
  constexpr bool W4 = FMT == MOE_FMT_W4G128;
  const int chunk = NT == 1 ? 8 : 4;
  const bool vs = W4 && G % (chunk * a.S) == 0;
  switch (NT * 16 + KW) {
    case 1 * 16 + 1: return vs ? run_linear<BF16, FMT, 1, 1, W4>(a, st) : run_linear<BF16, FMT, 1, 1>(a, st);
    case 1 * 16 + 2: return run_linear<BF16, FMT, 1, 2>(a, st);
    case 1 * 16 + 4: return run_linear<BF16, FMT, 1, 4>(a, st);
    case 1 * 16 + 8: return run_linear<BF16, FMT, 1, 8>(a, st);
    case 2 * 16 + 1: return vs ? run_linear<BF16, FMT, 2, 1, W4>(a, st) : run_linear<BF16, FMT, 2, 1>(a, st);
    case 2 * 16 + 2: return run_linear<BF16, FMT, 2, 2>(a, st);
    case 2 * 16 + 4: return run_linear<BF16, FMT, 2, 4>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
