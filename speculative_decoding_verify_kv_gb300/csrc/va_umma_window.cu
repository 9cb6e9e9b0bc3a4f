// Tensor-core partial kernel: the instantiations of windowed calls.
#include "va_umma.cuh"

namespace va {

// Maps over a bf16 cache whose boxes are one page of 64 columns.
bool make_page_maps(const Params& p, CUtensorMap* k, CUtensorMap* v) {
  return make_map(k, p, p.k, true) && make_map(v, p, p.v, true);
}

cudaError_t launch_umma_window(const Params& p, dim3 grid, cudaStream_t st) {
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
