// moe_linear_w4 on the fifth-generation tensor cores, for more than 16 tokens of a larger matrix.
//
// A CTA owns 128 weight rows (the lanes of tensor memory, MMA M) and one part of K; the tokens are MMA N = 32 or 64, larger
// batches take passes of 64.  Roles:
//   warps 0-7   dequantise: set s = warp / 4 takes the groups n = s, s + 2, ... of 128 k.  A warp copies its 32 rows' codes (2 KiB a
//               group) into a private ring with cp.async, four lanes to a row so that whole sectors are read; then a thread is a
//               row: its 64 bytes become 64 columns of tensor memory (tcgen05.st), never shared memory.  When the group's MMAs
//               are done it reads its row of the group's sums (tcgen05.ld) and adds them, times the group's scale, to its fp32
//               registers: as in the mma.sync kernel no weight is rounded, and the tensor core only ever adds up one group;
//   warp 8      one thread loads the tokens of each group by TMA (two boxes of 64 k, 128-byte swizzle) into a ring;
//   warp 9      one thread issues eight tcgen05.mma (A from tensor memory, B from shared memory) per group.
// An MMA with A from tensor memory takes about 100 cycles however few its tokens, eight a group; with one operand and one
// accumulator per set a group's store, MMAs, load and additions follow one another (0.43 us per group and SM with two CTAs of two
// sets, 0.72 with one CTA of 4 to 6; issuing the MMAs of several sets in turn, dequantising ahead of them or a deeper token ring
// changed nothing or lost).  Half of the time at 50304 x 7168 and 64 tokens (125 us) would be MMAs alone if every SM had the same
// share (62 us); the rest is that chain, and 393 blocks of rows on 296 resident CTAs, so that some CTAs take two.  mma.sync has no
// such chain but reads every token from shared memory per 16 rows: 125 against 87 us with 32 tokens and 233 against 125 us with 64.
// The sets' sums, and those of the cluster's CTAs on other parts of K, are joined in shared memory in a fixed order.
// Every wait is bounded (mbar_wait): one that runs out sets the device error word and its role stops; the CTA still frees its
// tensor memory.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "moe_linear.cuh"

namespace moe {
namespace {

constexpr int kPassTokens = 64;  // tokens per pass over the weights

template <int NTOK>
struct Um {
  static constexpr int kSets = 2;
  static constexpr int kDeqWarps = 4 * kSets;
  static constexpr int kThreads = 32 * (kDeqWarps + 2);
  static constexpr int kCtas = 2;  // per SM
  static constexpr int kTmemCols = 256;
  static constexpr int kACol = 0, kDCol = 64 * kSets;  // set s: A at 64 s, sums at kDCol + NTOK s
  static constexpr int kDepth = 4;                     // groups of weights in flight per warp
  static constexpr int kRing = kDepth * 2048;
  static constexpr int kXStages = NTOK == 64 ? 2 : 4;
  static constexpr int kAtom = NTOK * 128;  // 64 k of the tokens, 128 bytes each
  static constexpr int kXStage = 2 * kAtom;
  static constexpr int kOffW = kXStages * kXStage;
  static constexpr int kOffBar = kOffW + kDeqWarps * kRing;
  static constexpr int kBars = 2 * kXStages + 2 * kSets;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;  // + alignment slack
  static_assert(kDCol + kSets * NTOK <= kTmemCols, "tensor-memory plan");
  static_assert(finish_bytes(1, 128, NTOK + 1) <= kOffBar, "the partial sums reuse the rings");
  static_assert(kSmem * kCtas <= 226 * 1024, "shared-memory plan");
};

// ---------------------------------------------------------------- PTX wrappers
MOE_DEVICE void um_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
MOE_DEVICE void um_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
MOE_DEVICE void um_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T, M = 128, N from idesc, K = 16
MOE_DEVICE void um_mma(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
// 16 consecutive 32-bit columns of this thread's lane
MOE_DEVICE void um_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
MOE_DEVICE void um_ld16(uint32_t at, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(at)
      : "memory");
}
MOE_DEVICE void um_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
MOE_DEVICE void um_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
MOE_DEVICE void um_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
MOE_DEVICE void um_tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar))
      : "memory");
}
// K-major, 128-byte swizzle, rows of 128 bytes, 8-row groups 1024 bytes apart (base 1024-aligned; the start may advance by
// 32 bytes per K = 16 step inside the row)
MOE_DEVICE uint64_t um_desc(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}

// ---------------------------------------------------------------- codes to operand pairs in k order
// Four words (32 codes) of a row -> 16 registers of two 16-bit weights each (k ascending).
template <bool BF16>
MOE_DEVICE void w4_words_in_order(const uint4& q, uint32_t (&v)[16]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  constexpr uint32_t high = BF16 ? 0x43434343u : 0x64646464u;   // high byte of bf16 128, fp16 1024
  constexpr uint32_t bias = BF16 ? 0x43084308u : 0x64086408u;   // 136, 1032
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x0F0F0F0Fu, hi = (w[i] >> 4) & 0x0F0F0F0Fu;
    const uint32_t a = __byte_perm(lo, hi, 0x5140), b = __byte_perm(lo, hi, 0x7362);  // codes 0..3, 4..7
    const uint32_t p[4] = {__byte_perm(a, high, 0x4140), __byte_perm(a, high, 0x4342), __byte_perm(b, high, 0x4140),
                           __byte_perm(b, high, 0x4342)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[4 * i + j]) : "r"(p[j]), "r"(bias));
      else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[4 * i + j]) : "r"(p[j]), "r"(bias));
    }
  }
}
// E2M1 codes times the block scales of their words 0..1 and 2..3.  bf16: the fp16 pattern shifted right by three has the
// same exponent field under bf16's bias, the value times 2^-112, and the scale carries 2^104, so the product is the weight times
// 2^-8, as in the mma.sync kernel: tokens overflow at the same sizes whatever their number.
template <bool BF16>
MOE_DEVICE void e2m1_words_in_order(const uint4& q, uint32_t scales, uint32_t (&v)[16]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h2 = e4m3_to_h2((scales >> (8 * (i >> 1))) & 0xFFu);
    uint32_t s2 = h2;
    if (BF16) {
      s2 = float_to_bf16_bits(__half2float(__ushort_as_half(uint16_t(h2))) * 0x1p104f);
      s2 |= s2 << 16;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = e2m1x2_to_h2((w[i] >> (8 * j)) & 0xFFu);
      if (BF16)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[4 * i + j]) : "r"(((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u)), "r"(s2));
      else
        v[4 * i + j] = hmul2(h, s2);
    }
  }
}

template <bool BF16, int FMT, int NTOK>
__global__ void __launch_bounds__(Um<NTOK>::kThreads, Um<NTOK>::kCtas)
    k_linear_umma(const __grid_constant__ CUtensorMap tm_x, LinearArgs a, unsigned* err) {
  using U = Um<NTOK>;
  constexpr bool W4 = FMT == MOE_FMT_W4G128;
  constexpr int SETS = U::kSets, D = U::kDepth;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  uint64_t* fullX = reinterpret_cast<uint64_t*>(smem + U::kOffBar);
  uint64_t* emptyX = fullX + U::kXStages;
  uint64_t* fullA = emptyX + U::kXStages;  // a set's operand is in tensor memory (and its sums have been read)
  uint64_t* done = fullA + SETS;           // its MMAs are complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + SETS);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.y, t0 = blockIdx.z * kPassTokens, nt = min(a.T - t0, NTOK);
  const int G = a.K / 128, half = a.N / 2;
  const int gb = int(int64_t(part) * G / a.S), ng = int(int64_t(part + 1) * G / a.S) - gb;
  const bool deq = warp < U::kDeqWarps;
  const int set = warp >> 2, quarter = warp & 3;

  // ---- weights: this warp's 32 rows; rows past the end repeat the last one and are not stored
  const int ns = deq && ng > set ? (ng - set + SETS - 1) / SETS : 0;  // this set's groups
  const int row0 = a.swiglu ? (quarter < 2 ? 0 : half) + blockIdx.x * 64 + (quarter & 1) * 32 : blockIdx.x * 128 + quarter * 32;
  const int last = a.swiglu && quarter < 2 ? half - 1 : a.N - 1;
  const int first = min(row0, last);
  const uint8_t* wp = a.w + size_t(first) * (a.K / 2) + size_t(gb + set) * 64 + (lane & 3) * 16;
  uint32_t roff[4];  // copies: lane / 4 + 8 i is the row, lane % 4 the 16 bytes of its 64
#pragma unroll
  for (int i = 0; i < 4; ++i) roff[i] = uint32_t(min(row0 + (lane >> 2) + 8 * i, last) - first) * uint32_t(a.K / 2);
  const uint32_t ring = sbase + U::kOffW + (deq ? warp : 0) * U::kRing;
  int fetched = 0;
  auto fetch = [&]() {
    if (fetched < ns) {
      const uint32_t d = ring + (fetched & (D - 1)) * 2048;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 2) + 8 * i;  // 16-byte chunks exchanged by row, so that a thread per row reads without conflicts
        cp_async16(d + r * 64 + (((lane & 3) ^ (r >> 1)) & 3) * 16, wp + roff[i]);
      }
      wp += SETS * 64;
    }
    ++fetched;
    cp_commit();
  };
  if (deq) {
#pragma unroll
    for (int d = 0; d < D; ++d) fetch();
  }

  if (threadIdx.x == 32 * U::kDeqWarps) {
    for (int i = 0; i < U::kXStages; ++i) {
      mbar_init(&fullX[i], 1);
      mbar_init(&emptyX[i], 1);
    }
    for (int i = 0; i < SETS; ++i) {
      mbar_init(&fullA[i], 4);
      mbar_init(&done[i], 1);
    }
    fence_mbar_init();
  } else if (warp == U::kDeqWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(U::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  um_fence_before();
  __syncthreads();
  um_fence_after();
  const uint32_t tmem = *tmem_slot;

  float acc[NTOK];
#pragma unroll
  for (int i = 0; i < NTOK; ++i) acc[i] = 0.0f;

  if (deq) {
    constexpr int SB = W4 ? 2 : 8;  // scale bytes per group and row
    const int row = min(row0 + lane, last);
    const uint8_t* sp = a.scale + (size_t(row) * G + gb + set) * SB;
    auto scale_at = [&](int m) {  // the m-th of this set's groups
      uint2 v = make_uint2(0u, 0u);
      if (m < ns) {
        if (W4)
          v.x = __ldg(reinterpret_cast<const uint16_t*>(sp + size_t(m) * (SETS * SB)));
        else
          v = __ldg(reinterpret_cast<const uint2*>(sp + size_t(m) * (SETS * SB)));
      }
      return v;
    };
    const uint32_t at = tmem + (uint32_t(quarter * 32) << 16);
    uint2 sc = scale_at(0), sc1 = scale_at(1);
    // 32 codes j of this thread's row of group m, as operand registers
    auto codes = [&](int m, int j, const uint2& s, uint32_t (&v)[16]) {
      uint4 q;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                   : "r"(ring + (m & (D - 1)) * 2048 + lane * 64 + ((j ^ (lane >> 1)) & 3) * 16));
      if (W4)
        w4_words_in_order<BF16>(q, v);
      else
        e2m1_words_in_order<BF16>(q, (j < 2 ? s.x : s.y) >> (16 * (j & 1)), v);
    };
    for (int m = 0; m < ns; ++m) {
      cp_wait<D - 1>();
      __syncwarp();  // the warp's copies of this group are visible to all its lanes
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t v[16];
        codes(m, j, sc, v);
        um_st16(at + uint32_t(U::kACol + set * 64 + j * 16), v);
      }
      __syncwarp();  // every lane has read the slot
      fetch();
      um_wait_st();
      um_fence_before();
      __syncwarp();
      if (lane == 0) um_arrive(&fullA[set]);
      const float f = W4 ? __uint_as_float(sc.x << 16) : 1.0f;
      sc = sc1;
      sc1 = scale_at(m + 2);
      const bool ok = mbar_wait(&done[set], m & 1, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      um_fence_after();
#pragma unroll
      for (int c = 0; c < NTOK; c += 16) {
        uint32_t v[16];
        um_ld16(at + uint32_t(U::kDCol + set * NTOK + c), v);
        um_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c + i] = fmaf(f, __uint_as_float(v[i]), acc[c + i]);
      }
    }
    cp_wait<0>();
  } else if (warp == U::kDeqWarps) {
    if (lane == 0) {
      int issued = 0;
      for (int n = 0; n < ng; ++n) {
        const int st = n % U::kXStages;
        if (!mbar_wait(&emptyX[st], ((n / U::kXStages) & 1) ^ 1, err)) break;
        mbar_arrive_expect_tx(&fullX[st], uint32_t(U::kXStage));
        const uint32_t d = sbase + st * U::kXStage;
        um_tma_2d(d, &tm_x, (gb + n) * 128, t0, &fullX[st]);
        um_tma_2d(d + U::kAtom, &tm_x, (gb + n) * 128 + 64, t0, &fullX[st]);
        issued = n + 1;
      }
      // every load has landed before the CTA moves on (also when a wait ran out)
      for (int n = max(0, issued - U::kXStages); n < issued; ++n) mbar_wait(&fullX[n % U::kXStages], (n / U::kXStages) & 1, err);
    }
    __syncwarp();
  } else {
    if (lane == 0) {
      // fp32 sums, A and B both bf16 or both fp16, K-major
      const uint32_t ab = BF16 ? 1u : 0u;
      const uint32_t idesc = (1u << 4) | (ab << 7) | (ab << 10) | (uint32_t(NTOK >> 3) << 17) | (uint32_t(128 >> 4) << 24);
      const uint64_t desc0 = um_desc(sbase);
      int issued = 0;
      for (int n = 0; n < ng; ++n) {
        const int st = n % U::kXStages, s = n % SETS;
        if (!mbar_wait(&fullX[st], (n / U::kXStages) & 1, err) || !mbar_wait(&fullA[s], (n / SETS) & 1, err)) break;
        um_fence_after();
        const uint64_t desc = desc0 + uint64_t((st * U::kXStage) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // atom kk / 4, 32 bytes per K = 16 step inside it
          um_mma(tmem + uint32_t(U::kDCol + s * NTOK), tmem + uint32_t(U::kACol + s * 64 + kk * 8),
                 desc + uint64_t((kk >> 2) * (U::kAtom >> 4) + 2 * (kk & 3)), idesc, kk != 0);
        um_commit(&emptyX[st]);
        um_commit(&done[s]);
        issued = n + 1;
      }
      // the MMAs are complete before tensor memory is freed (also when a wait ran out)
      for (int n = max(0, issued - SETS); n < issued; ++n) mbar_wait(&done[n % SETS], (n / SETS) & 1, err);
    }
    __syncwarp();
  }
  um_fence_before();
  __syncthreads();  // all sums are in registers, all copies have landed and been used
  um_fence_after();
  if (warp == U::kDeqWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(U::kTmemCols) : "memory");
  // sums: [128][NTOK + 1] floats (odd row length: a column of rows spreads over the banks), set 1's plus set 0's
  float* red = reinterpret_cast<float*>(smem);
  constexpr int LD = NTOK + 1;
  float* o = red + (quarter * 32 + lane) * LD;
  if (deq && set == 1) {
#pragma unroll
    for (int i = 0; i < NTOK; ++i) o[i] = acc[i];
  }
  __syncthreads();
  if (deq && set == 0) {
#pragma unroll
    for (int i = 0; i < NTOK; ++i) o[i] += acc[i];
  }
  finish_linear<1, 128, LD, 64>(a, red, part, t0, nt, W4 ? 1.0f : *a.gscale * (BF16 ? 256.0f : 1.0f));
}

cudaError_t encode_tokens(CUtensorMap* map, const LinearArgs& a, bool bf16, int box_rows);

template <bool BF16, int FMT, int NTOK>
cudaError_t run_umma(const LinearArgs& a, unsigned* err_word, cudaStream_t st) {
  using U = Um<NTOK>;
  // raised once per device, so no later call (e.g. one inside a stream capture) sets attributes
  static std::atomic<bool> ready[128] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(k_linear_umma<BF16, FMT, NTOK>, cudaFuncAttributeMaxDynamicSharedMemorySize, U::kSmem);
    if (err != cudaSuccess) return err;
    ready[dev].store(true, std::memory_order_release);
  }
  CUtensorMap map;
  if ((err = encode_tokens(&map, a, BF16, NTOK)) != cudaSuccess) return err;
  const int blocks = a.swiglu ? (a.N / 2 + 63) / 64 : (a.N + 127) / 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks), unsigned(a.S), unsigned((a.T + kPassTokens - 1) / kPassTokens));
  cfg.blockDim = dim3(U::kThreads);
  cfg.dynamicSmemBytes = U::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = unsigned(a.S);
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear_umma<BF16, FMT, NTOK>, map, a, err_word);
}

}  // namespace
}  // namespace moe
