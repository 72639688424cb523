// moe_linear_w4 for W4G128 matrices, and the choice between the formats (the kernel: moe_linear.cuh).
#include "moe_linear.cuh"

namespace moe {

cudaError_t linear_nvfp4(const LinearArgs& a, bool bf16, cudaStream_t st);                    // moe_linear_nvfp4.cu
cudaError_t linear_umma(const LinearArgs& a, moe_format_t fmt, bool bf16, cudaStream_t st);  // moe_linear_umma.cu

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
  // A tcgen05 pass takes 64 tokens in about the time of one; a pass here takes 16, but in a tenth of the latency, and
  // several passes fill the machine that a small matrix leaves empty.  The unit is one warp's: 16 rows x 128 k x 16 tokens.
  // Up to 30000 of them (200 per SM) passes take 0.4 .. 0.95 of tcgen05's time, 1.09 at worst (128 x 2048, 64 tokens: 5.5
  // against 13.6 us; 512 x 7168: 8.6 against 17.0; 7168 x 2048: 16.0 against 20.3; 4096 x 7168, 20 tokens: 16.7 against
  // 15.5); at 43000 they take 1.1 .. 1.3 of it (4096 x 7168, 40 tokens: 25.6 against 20.0 us).
  const int64_t units = int64_t((T + 15) / 16) * ((N + 15) / 16) * (K / 128);
  if (T > 16 && units > 30000) return linear_umma(a, w.fmt, bf16, st);
  if (w.fmt == MOE_FMT_W4G128)
    return bf16 ? pick_linear<true, MOE_FMT_W4G128>(a, st) : pick_linear<false, MOE_FMT_W4G128>(a, st);
  return linear_nvfp4(a, bf16, st);
}

}  // namespace moe
