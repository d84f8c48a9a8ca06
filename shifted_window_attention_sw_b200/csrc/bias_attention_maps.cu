// Tensor maps of the attention's tiles.
#include "bias_attention.cuh"

namespace vswin {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeFn) nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

}  // namespace

bool make_head_map(HeadMap* m, const Heads& v, int B, int L, int H, int d, int dtype, int rows) {
  m->use = 0;
  m->hmul = m->bmul = 1;
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  long long st = v.st * 2, sh = v.sh * 2, sb = v.sb * 2;
  if (L > 1 && st == 0) return false;
  if (H == 1 || sh == 0) H = 1, m->hmul = 0, sh = 16;
  if (B == 1 || sb == 0) B = 1, m->bmul = 0, sb = 16;
  if (L == 1) st = 16;
  if (st >= (1LL << 40) || sh >= (1LL << 40) || sb >= (1LL << 40)) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)st, (cuuint64_t)sh, (cuuint64_t)sb};
  const cuuint32_t box[4] = {(cuuint32_t)(d == 32 ? 32 : 64), (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
  m->use = fn(&m->map, dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, v.p, dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              d == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  return m->use != 0;
}

}  // namespace vswin
