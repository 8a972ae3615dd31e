// swin_rows_f32.cu -- the row kernels (swin_rows.cuh) on fp32 activations.
#include "swin_rows.cuh"

namespace swin {
namespace rows {

int launch_f32(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  return launch_width<float>(a, bwd, branch, pre, ctas, st);
}

}  // namespace rows
}  // namespace swin
