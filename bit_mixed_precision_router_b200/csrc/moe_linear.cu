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
#include <cooperative_groups.h>

#include <atomic>

#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kLinWarps = 8;
constexpr int kPassTokens = 64;  // tokens per pass over the weights

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
  int RW, S;
};

// pair i of a word of eight W4 codes (nibbles i and i + 4) as q values
template <bool BF16>
MOE_DEVICE uint32_t w4_pair(uint32_t word, int i) {
  constexpr uint32_t magic = BF16 ? 0x43004300u : 0x64006400u;  // 128 or 1024, one unit per code step
  uint32_t v, d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "n"(0x000F000F), "r"(magic));
  if (BF16)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x43084308u));  // 136
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x64086408u));  // 1032
  return d;
}

// the same for E2M1 codes times the block's scale.  fp16: pairs are nibbles (2i, 2i + 1).  bf16: nibbles (i, i + 4);
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

MOE_DEVICE uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__host__ __device__ constexpr int kChunkGroups(int NT) { return NT <= 2 ? 16 : 32 / NT; }  // groups of K staged at a time
__host__ __device__ constexpr int kTokStride(int NT) { return kChunkGroups(NT) * 256 + 64; }  // bytes per staged token; 64: no bank conflicts

// NT: 8-token tiles per pass; D: groups of weights in flight per warp.
template <bool BF16, int FMT, int NT, int D>
__global__ void __launch_bounds__(32 * kLinWarps) k_linear_w4(LinearArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool W4 = FMT == MOE_FMT_W4G128;
  constexpr int CG = kChunkGroups(NT), STRIDE = kTokStride(NT), LD = 8 * NT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int RW = a.RW, KW = kLinWarps / RW, wr = warp / KW, kw = warp % KW;
  const int part = blockIdx.y;  // K part of this CTA (its rank in the cluster)
  const int t0 = blockIdx.z * kPassTokens, nt = min(a.T - t0, 8 * NT);
  const int G = a.K / 128;
  const int gb = int(int64_t(part) * G / a.S), ge = int(int64_t(part + 1) * G / a.S);
  const int chunks = (ge - gb + CG - 1) / CG, CI = CG / KW;
  const int ni = ge - gb > kw ? (ge - gb - kw + KW - 1) / KW : 0;  // this warp's groups: gb + kw + i KW

  // rows of this lane; rows past the end repeat the last one and are not stored
  const int tile = blockIdx.x * RW + wr, half = a.N / 2;
  const int r0 = a.swiglu ? min(tile * 8 + g, half - 1) : min(tile * 16 + g, a.N - 1);
  const int r1 = a.swiglu ? r0 + half : min(tile * 16 + g + 8, a.N - 1);
  const uint8_t* w0 = a.w + size_t(r0) * (a.K / 2) + c * 16 + size_t(gb + kw) * 64;
  const uint8_t* w1 = a.w + size_t(r1) * (a.K / 2) + c * 16 + size_t(gb + kw) * 64;
  // W4: one bf16 per group; NVFP4: eight bytes per group, two of them (32 codes) this lane's
  const uint8_t* s0 = a.scale + (W4 ? (size_t(r0) * G + gb + kw) * 2 : (size_t(r0) * G + gb + kw) * 8 + 2 * c);
  const uint8_t* s1 = a.scale + (W4 ? (size_t(r1) * G + gb + kw) * 2 : (size_t(r1) * G + gb + kw) * 8 + 2 * c);

  uint4 wa[D], wb[D];
  uint32_t sa[D], sb[D];
  auto fetch = [&](int i, int d) {
    if (i >= ni) return;
    const size_t o = size_t(i) * KW;
    wa[d] = ldg_stream(w0 + o * 64);
    wb[d] = ldg_stream(w1 + o * 64);
    sa[d] = __ldg(reinterpret_cast<const uint16_t*>(s0 + o * (W4 ? 2 : 8)));
    sb[d] = __ldg(reinterpret_cast<const uint16_t*>(s1 + o * (W4 ? 2 : 8)));
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, d);

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

  const uint16_t* x = static_cast<const uint16_t*>(a.x) + size_t(t0) * a.ldx;
  for (int ch = 0; ch < chunks; ++ch) {
    // stage the chunk's tokens: 16 bytes (8 elements) q of a group go to word j = q % 4 of lane c = q / 4
    if (ch) __syncthreads();
    const int g0 = gb + ch * CG, units = min(CG, ge - g0) * 16;
    for (int b = threadIdx.x; b < nt * units; b += 4 * 32 * kLinWarps) {
      uint4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int q = b + r * 32 * kLinWarps, t = q / units, u = q - t * units;
        if (t < nt) v[r] = *reinterpret_cast<const uint4*>(x + size_t(t) * a.ldx + size_t(g0) * 128 + u * 8);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int q = b + r * 32 * kLinWarps, t = q / units, u = q - t * units;
        if (t >= nt) continue;
        uint4 o = v[r];
        if (W4 || BF16) {  // pairs (i, i + 4)
          o.x = __byte_perm(v[r].x, v[r].z, 0x5410);
          o.y = __byte_perm(v[r].x, v[r].z, 0x7632);
          o.z = __byte_perm(v[r].y, v[r].w, 0x5410);
          o.w = __byte_perm(v[r].y, v[r].w, 0x7632);
        }
        *reinterpret_cast<uint4*>(smem + t * STRIDE + (u >> 4) * 256 + (u & 3) * 64 + ((u >> 2) & 3) * 16) = o;
      }
    }
    __syncthreads();
    for (int i0 = ch * CI; i0 < min((ch + 1) * CI, ni); i0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int i = i0 + d;
        if (i >= ni) break;
        const uint8_t* xs = smem + ((i - ch * CI) * KW + kw) * 256 + c * 16 + g * STRIDE;
        float part_acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) part_acc[n][e] = 0.0f;
        const uint32_t ua[4] = {wa[d].x, wa[d].y, wa[d].z, wa[d].w}, ub[4] = {wb[d].x, wb[d].y, wb[d].z, wb[d].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t pa[4], pb[4];
          if (W4) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              pa[p] = w4_pair<BF16>(ua[j], p);
              pb[p] = w4_pair<BF16>(ub[j], p);
            }
          } else {
            const uint32_t fa = e4m3_pair<BF16>((sa[d] >> (j < 2 ? 0 : 8)) & 0xFFu);
            const uint32_t fb = e4m3_pair<BF16>((sb[d] >> (j < 2 ? 0 : 8)) & 0xFFu);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              pa[p] = e2m1_pair<BF16>(ua[j], p, fa);
              pb[p] = e2m1_pair<BF16>(ub[j], p, fb);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 b = make_uint4(0, 0, 0, 0);
            if (8 * n + g < nt) b = *reinterpret_cast<const uint4*>(xs + n * 8 * STRIDE + j * 64);
            mma16<BF16>(part_acc[n], pa[0], pb[0], pa[1], pb[1], b.x, b.y);
            mma16<BF16>(part_acc[n], pa[2], pb[2], pa[3], pb[3], b.z, b.w);
          }
        }
        const float fa = W4 ? __uint_as_float(sa[d] << 16) : 1.0f, fb = W4 ? __uint_as_float(sb[d] << 16) : 1.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[n][e] = W4 ? fmaf(e < 2 ? fa : fb, part_acc[n][e], acc[n][e]) : acc[n][e] + part_acc[n][e];
        }
        fetch(i + D, d);
      }
    }
  }
  // partial sums: [KW][RW * 16][LD] floats
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  const int RB = RW * 16;
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
  for (int q = threadIdx.x; q < fn * nt; q += 32 * kLinWarps) {
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
template <bool BF16, int FMT, int NT, int D>
cudaError_t run_linear(const LinearArgs& a, cudaStream_t st) {
  const int tok = a.T < 8 * NT ? a.T : 8 * NT;
  size_t smem = size_t(tok) * kTokStride(NT);
  const size_t red = size_t(kLinWarps) * 16 * 8 * NT * sizeof(float);
  if (smem < red) smem = red;
  constexpr int most = 8 * NT * kTokStride(NT);
  if constexpr (most > 48 * 1024) {
    // raised once per device, so no later call (e.g. one inside a stream capture) sets attributes
    static std::atomic<bool> done[128] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
      err = cudaFuncSetAttribute(k_linear_w4<BF16, FMT, NT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (err != cudaSuccess) return err;
      done[dev].store(true, std::memory_order_release);
    }
  }
  const int tiles = (a.N + 15) / 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((tiles + a.RW - 1) / a.RW), unsigned(a.S), unsigned((a.T + kPassTokens - 1) / kPassTokens));
  cfg.blockDim = dim3(32 * kLinWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = unsigned(a.S);
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear_w4<BF16, FMT, NT, D>, a);
}

template <bool BF16, int FMT>
cudaError_t pick_linear(LinearArgs a, cudaStream_t st) {
  const int tok = a.T < kPassTokens ? a.T : kPassTokens;
  const int NT = tok <= 8 ? 1 : tok <= 16 ? 2 : tok <= 32 ? 4 : 8;
  // split K until there are warps enough for the machine, two groups per warp at least: first among the
  // warps of a CTA, then over the CTAs of a cluster
  const int tiles = (a.N + 15) / 16, G = a.K / 128, want = 148 * 16;
  const int kw_most = NT <= 2 ? 8 : NT == 4 ? 4 : 2;
  int KW = 1, S = 1;
  while (KW < kw_most && tiles * KW < want && KW * 4 <= G) KW *= 2;
  while (S < 8 && int64_t(tiles) * KW * S < want && KW * S * 4 <= G) S *= 2;
  a.RW = kLinWarps / KW;
  a.S = S;
  const bool deep = kChunkGroups(NT) / KW >= 4;
  if (NT == 1) return deep ? run_linear<BF16, FMT, 1, 4>(a, st) : run_linear<BF16, FMT, 1, 2>(a, st);
  if (NT == 2) return deep ? run_linear<BF16, FMT, 2, 4>(a, st) : run_linear<BF16, FMT, 2, 2>(a, st);
  if (NT == 4) return deep ? run_linear<BF16, FMT, 4, 4>(a, st) : run_linear<BF16, FMT, 4, 2>(a, st);
  return deep ? run_linear<BF16, FMT, 8, 4>(a, st) : run_linear<BF16, FMT, 8, 2>(a, st);
}

}  // namespace

cudaError_t launch_linear_w4(const moe_linear_t& w, const void* x, int64_t ldx, moe_dtype_t x_dtype, int T, int N, int K,
                             moe_act_t act, const void* residual, int64_t ldr, void* y, int64_t ldy, moe_dtype_t y_dtype,
                             cudaStream_t st) {
  LinearArgs a = {};
  a.w = static_cast<const uint8_t*>(w.w);
  a.scale = static_cast<const uint8_t*>(w.scale);
  a.gscale = w.gscale;
  a.x = x;
  a.ldx = ldx;
  a.residual = residual;
  a.ldr = ldr;
  a.y = y;
  a.ldy = ldy;
  a.y_dtype = int(y_dtype);
  a.T = T;
  a.N = N;
  a.K = K;
  a.swiglu = act == MOE_ACT_SWIGLU;
  const bool bf16 = x_dtype == MOE_BF16;
  if (w.fmt == MOE_FMT_W4G128)
    return bf16 ? pick_linear<true, MOE_FMT_W4G128>(a, st) : pick_linear<false, MOE_FMT_W4G128>(a, st);
  return bf16 ? pick_linear<true, MOE_FMT_NVFP4>(a, st) : pick_linear<false, MOE_FMT_NVFP4>(a, st);
}

}  // namespace moe
