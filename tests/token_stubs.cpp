// Stand-ins for the launchers of the kernels on token rows in a host-only
// build of their entry points.  Calls that pass every argument check end here.
#include "../bmmc_affine_index_amd/csrc/tokens/tokens.h"

namespace bmmc {

int launch_expert_order(const OrderArgs &, int, hipStream_t) { return BMMC_ERR_HIP; }
int launch_expert_gather(const MoveArgs &, int, hipStream_t) { return BMMC_ERR_HIP; }
int launch_expert_combine(const MoveArgs &, int, hipStream_t) { return BMMC_ERR_HIP; }
int launch_expert_combine_backward(const MoveArgs &, int, hipStream_t) { return BMMC_ERR_HIP; }
int launch_rotary(const HeadsArgs &, const bmmc_rotation &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_cache_append(const AppendArgs &, hipStream_t) { return BMMC_ERR_HIP; }

}  // namespace bmmc
