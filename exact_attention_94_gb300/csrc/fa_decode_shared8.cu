// The main kernel of decode_shared.cuh over pages of 8-bit codes.
#include "decode_shared.cuh"

namespace fa {

cudaError_t launch_shared_main8(const CUtensorMap (&maps)[5], const SharedParams& p, int D, cudaLaunchConfig_t& cfg) {
  return D == 64 ? launch_shared_main<64, true>(maps, p, cfg) : launch_shared_main<128, true>(maps, p, cfg);
}

}  // namespace fa
