// swin_heads_bf16.cu -- the head kernel (swin_heads.cuh) on bf16 activations.
#include "swin_heads.cuh"

namespace swin {
namespace heads {

int launch_bf16(const Args &a, bool bwd, bool norm, bool beta, int ctas, size_t smem, cudaStream_t st) {
  return launch_heads<__nv_bfloat16>(a, bwd, norm, beta, ctas, smem, st);
}

}  // namespace heads
}  // namespace swin
