// ggrn_norms_bf16.cu -- the kernels of ggrn_norms.cuh for T = bf16.
#include "ggrn_norms.cuh"

namespace ggrn {
namespace norms {

int launch_bf16(int kind, const Params& p, const Plan& k, cudaStream_t s) {
  switch (kind) {
    case kLayerNorm: return launch_kind<kLayerNorm, __nv_bfloat16>(p, k, s);
    case kLayerNormGrad: return launch_kind<kLayerNormGrad, __nv_bfloat16>(p, k, s);
    default: return launch_kind<kMamba2Grad, __nv_bfloat16>(p, k, s);
  }
}

}  // namespace norms
}  // namespace ggrn
