// ggrn_norms_f32.cu -- the kernels of ggrn_norms.cuh for T = f32.
#include "ggrn_norms.cuh"

namespace ggrn {
namespace norms {

int launch_f32(int kind, const Params& p, const Plan& k, cudaStream_t s) {
  switch (kind) {
    case kLayerNorm: return launch_kind<kLayerNorm, float>(p, k, s);
    case kLayerNormGrad: return launch_kind<kLayerNormGrad, float>(p, k, s);
    case kOnnxGrad: return launch_kind<kOnnxGrad, float>(p, k, s);
    default: return launch_kind<kMamba2Grad, float>(p, k, s);
  }
}

}  // namespace norms
}  // namespace ggrn
