// The team decode's kernels over a cache of int8 codes.
#include "pkv_team_impl.cuh"

namespace pkv {
TeamKernel team_kernel_int8(int head_dim, int group) {
    return head_dim == 64 ? team_kernel_info<kTeamInt8, 64>(group) : team_kernel_info<kTeamInt8, 128>(group);
}
}  // namespace pkv
