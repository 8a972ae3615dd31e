// swin_rows_bf16.cu -- the row kernels (swin_rows.cuh) on bf16 activations.
#include "swin_rows.cuh"

namespace swin {
namespace rows {

int launch_bf16(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  return launch_width<__nv_bfloat16>(a, bwd, branch, pre, ctas, st);
}

}  // namespace rows
}  // namespace swin
