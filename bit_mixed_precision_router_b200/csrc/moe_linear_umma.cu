// The tcgen05 form of moe_linear_w4 (the kernel: moe_linear_umma.cuh) and the tensor map of its tokens.
#include "moe_linear_umma.cuh"

namespace moe {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  // looked up once, through the runtime (host threads may race to store the same value)
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn fn = cached.load(std::memory_order_acquire);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
    cached.store(fn, std::memory_order_release);
  }
  return fn;
}

// x [T][K] (rows ldx elements apart) in boxes of box_rows tokens x 64 k, 128-byte swizzle; tokens past T read as zeros
cudaError_t encode_tokens(CUtensorMap* map, const LinearArgs& a, bool bf16, int box_rows) {
  const EncodeFn enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cuuint64_t(a.K), cuuint64_t(a.T)};
  const cuuint64_t strides[1] = {cuuint64_t(a.ldx) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(a.x),
                         dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Parts of K: as many CTAs as SMs (a call with few blocks has many groups: it would not come here otherwise); with a block
// of rows for every other SM the split costs more than it gives (4096 x 7168, 64 tokens: 4 parts 23.6, 2 parts 30 us; 12288 x 4096: 1 part 31.7, 2 parts
// 36 us).  Six rather than eight where eight would not fill the machine either (2048 x 7168: 20.5 against 25.7 us).
int umma_parts(int blocks) { return blocks > 73 ? 1 : blocks > 36 ? 2 : blocks > 18 ? 4 : blocks > 9 ? 6 : 8; }

template <bool BF16, int FMT>
cudaError_t pick_umma(LinearArgs a, unsigned* err, cudaStream_t st) {
  const int rows = a.swiglu ? (a.N / 2 + 63) / 64 : (a.N + 127) / 128, passes = (a.T + kPassTokens - 1) / kPassTokens;
  a.S = umma_parts(rows > 1000 || passes > 1000 ? 1000 : rows * passes);
  return a.T <= 32 ? run_umma<BF16, FMT, 32>(a, err, st) : run_umma<BF16, FMT, 64>(a, err, st);
}

}  // namespace

cudaError_t linear_umma(const LinearArgs& a, moe_format_t fmt, bool bf16, cudaStream_t st) {
  unsigned* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  if (fmt == MOE_FMT_W4G128) return bf16 ? pick_umma<true, MOE_FMT_W4G128>(a, err, st) : pick_umma<false, MOE_FMT_W4G128>(a, err, st);
  return bf16 ? pick_umma<true, MOE_FMT_NVFP4>(a, err, st) : pick_umma<false, MOE_FMT_NVFP4>(a, err, st);
}

}  // namespace moe
