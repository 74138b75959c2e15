// The team decode's kernels over an fp16 cache (listed blocks).
#include "pkv_team_impl.cuh"

namespace pkv {
TeamKernel team_kernel_f16(int head_dim, int group) {
    return head_dim == 64 ? team_kernel_info<kTeamF16, 64>(group) : team_kernel_info<kTeamF16, 128>(group);
}
}  // namespace pkv
