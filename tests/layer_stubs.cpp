// Stand-ins for the launchers of a layer's kernels in a host-only build of their
// entry points.  Calls that pass every argument check end here.
#include "../bmmc_affine_index_amd/csrc/layer/layer.h"

namespace bmmc {

int launch_attend_few(const AttendArgs &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_attend_many(const AttendArgs &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_attend_join(const AttendArgs &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_cache_quantize(const QuantizeArgs &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_cache_read(const ReadArgs &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_expert_balance(const BalanceArgs &, hipStream_t) { return BMMC_ERR_HIP; }
int launch_expert_balance_backward(const BalanceArgs &, hipStream_t) { return BMMC_ERR_HIP; }

}  // namespace bmmc
