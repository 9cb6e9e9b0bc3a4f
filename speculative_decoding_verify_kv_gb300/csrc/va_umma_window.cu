// Tensor-core partial kernel: the instantiations of windowed calls.
#include "va_umma.cuh"

namespace va {

// Maps over a bf16 cache for the kernels that take it page by page: one box is
// 16 tokens of one KV head, as D / 64 column blocks of 64 one after the other
// (the column block is a dimension of its own, outside the tokens), so that a
// page of one tensor is one copy.  Contiguous [64][capacity][D / 64][plane],
// paged [64][16][D / 64][KVH][block].
static bool make_page_map(CUtensorMap* map, const Params& p, const void* base) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t D = (cuuint64_t)p.D, nb = D / 64, row = D * 2;
  const cuuint32_t box[5] = {64, (cuuint32_t)kPage, (cuuint32_t)nb, 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r;
  if (p.page_size == 0) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)p.capacity, nb, (cuuint64_t)p.num_seqs * p.KVH};
    const cuuint64_t strides[3] = {row, 128, (cuuint64_t)p.capacity * row};
    r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[5] = {64, (cuuint64_t)kPage, nb, (cuuint64_t)p.KVH, (cuuint64_t)p.num_blocks};
    const cuuint64_t strides[4] = {row, 128, kPage * row, (cuuint64_t)p.KVH * kPage * row};
    r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return r == CUDA_SUCCESS;
}

bool make_page_maps(const Params& p, CUtensorMap* k, CUtensorMap* v) {
  return make_page_map(k, p, p.k) && make_page_map(v, p, p.v);
}

cudaError_t launch_umma_window(Params& p, dim3 grid, cudaStream_t st) {
#define VA_U_WIN(DD)                                                                             \
  if (p.D == DD)                                                                                 \
    return p.kv_dtype == VA_BF16 ? launch_umma_t<DD, VA_BF16, true, true>(p, grid, st)           \
                                 : launch_umma_t<DD, VA_Q8_0, true, true>(p, grid, st);
  if (p.kv_dtype != VA_F32) {
    VA_U_WIN(64) VA_U_WIN(128) VA_U_WIN(256)
  }
#undef VA_U_WIN
  return cudaErrorInvalidValue;
}

}  // namespace va
