// swin_heads_f32.cu -- the head kernel (swin_heads.cuh) on fp32 activations.
#include "swin_heads.cuh"

namespace swin {
namespace heads {

int launch_f32(const Args &a, bool bwd, bool norm, bool beta, int ctas, size_t smem, cudaStream_t st) {
  return launch_heads<float>(a, bwd, norm, beta, ctas, smem, st);
}

}  // namespace heads
}  // namespace swin
