// ggrn_norms_f16.cu -- the kernels of ggrn_norms.cuh for T = f16.
#include "ggrn_norms.cuh"

namespace ggrn {
namespace norms {

int launch_f16(int kind, const Params& p, const Plan& k, cudaStream_t s) {
  switch (kind) {
    case kLayerNorm: return launch_kind<kLayerNorm, __half>(p, k, s);
    case kLayerNormGrad: return launch_kind<kLayerNormGrad, __half>(p, k, s);
    case kOnnxGrad: return launch_kind<kOnnxGrad, __half>(p, k, s);
    default: return launch_kind<kMamba2Grad, __half>(p, k, s);
  }
}

}  // namespace norms
}  // namespace ggrn
