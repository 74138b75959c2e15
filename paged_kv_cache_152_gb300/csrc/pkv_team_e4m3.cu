// The team decode's kernels over a cache of e4m3 codes.
#include "pkv_team_impl.cuh"

namespace pkv {
TeamKernel team_kernel_e4m3(int head_dim, int group) {
    return head_dim == 64 ? team_kernel_info<kTeamE4m3, 64>(group) : team_kernel_info<kTeamE4m3, 128>(group);
}
}  // namespace pkv
