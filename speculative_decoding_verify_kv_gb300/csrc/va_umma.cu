// Tensor-core partial kernel: the instantiations of the unwindowed calls.
#include "va_umma.cuh"

namespace va {

int umma_threads(int D, int kv_dtype) {
  (void)D;
  return kv_dtype == VA_Q8_0 ? UCfg<256, VA_Q8_0>::THREADS : UCfg<256, VA_BF16>::THREADS;
}

int umma_smem_bytes(int D, int kv_dtype) {
#define VA_U_SMEM(DD, KT) \
  if (D == DD && kv_dtype == KT) return UCfg<DD, KT>::SMEM;
  VA_U_SMEM(64, VA_BF16) VA_U_SMEM(64, VA_Q8_0) VA_U_SMEM(128, VA_BF16)
  VA_U_SMEM(128, VA_Q8_0) VA_U_SMEM(256, VA_BF16) VA_U_SMEM(256, VA_Q8_0)
#undef VA_U_SMEM
  return 0;
}

cudaError_t launch_umma_partial(const Params& p, dim3 grid, cudaStream_t st) {
#define VA_U_BF16(DD)                                                                     \
  if (p.D == DD && p.kv_dtype == VA_BF16)                                                 \
    return p.page_size != 0 ? launch_umma_t<DD, VA_BF16, true, false>(p, grid, st)              \
                            : launch_umma_t<DD, VA_BF16, false, false>(p, grid, st);
#define VA_U_Q8(DD)                                                                       \
  if (p.D == DD && p.kv_dtype == VA_Q8_0)                                                 \
    return p.page_size != 0 ? launch_umma_t<DD, VA_Q8_0, true, false>(p, grid, st)              \
                            : launch_umma_t<DD, VA_Q8_0, false, false>(p, grid, st);
  VA_U_BF16(64) VA_U_Q8(64) VA_U_BF16(128) VA_U_Q8(128) VA_U_BF16(256) VA_U_Q8(256)
#undef VA_U_BF16
#undef VA_U_Q8
  return cudaErrorInvalidValue;
}

}  // namespace va
