// pkv_team_params.h -- parameters and workspace of the team decode.
#ifndef PKV_TEAM_PARAMS_H
#define PKV_TEAM_PARAMS_H

#include <cuda_fp16.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

constexpr int kTeamMaxGroup = 16;

struct TeamParams {
    __half *out;                  // [N][H][D]
    const __half *query;          // [N][H][D]
    const void *key_cache;        // [NB][Hkv][BS][D]
    const void *value_cache;
    const float *key_scale;       // [NB] rows of Hkv, scale_stride apart; 8-bit caches only
    const float *value_scale;
    const int32_t *block_tables;  // [N][MB]
    const int32_t *context_lens;  // [N]
    const int32_t *selected;      // [N][Hkv][max_selected], NULL: every block
    const int32_t *num_selected;  // [N][Hkv]
    int2 *cut;                    // [C] segments that CTA c's first and last piece are cut of, or -1
    float2 *part_ml;              // [C][2][G] a cut piece's (maximum, sum)
    float *part_o;                // [C][2][G][D] and its output
    int32_t *status;
    int num_seqs;
    int num_heads;
    int num_kv_heads;
    int group;
    int max_blocks_per_seq;
    int max_selected;
    int num_blocks;
    int block_shift;
    int scale_stride;
    float scale_log2;             // scale * log2(e)
};

// Workspace carve-up (byte offsets).  It carries nothing from call to call.
struct TeamWorkspace {
    size_t ml, o, total;
    static TeamWorkspace plan(int64_t ctas, int group, int head_dim) {
        auto up = [](size_t x) { return (x + 255) / 256 * 256; };
        TeamWorkspace w;
        w.ml = up(sizeof(int2) * (size_t)ctas);
        w.o = w.ml + up(sizeof(float2) * (size_t)ctas * 2 * group);
        w.total = w.o + up(sizeof(float) * (size_t)ctas * 2 * group * head_dim);
        return w;
    }
};

// One compiled kernel.
struct TeamKernel {
    const void *fn;
    size_t smem_fixed;    // dynamic shared memory without the prefix sums (8 bytes per sequence)
    int threads;
    int ctas_per_sm;
    int step_rows;
};

// pkv_team_{f16,int8,e4m3}.cu; head_dim 64 or 128, group 1 to 16.
TeamKernel team_kernel_f16(int head_dim, int group);
TeamKernel team_kernel_int8(int head_dim, int group);
TeamKernel team_kernel_e4m3(int head_dim, int group);

}  // namespace pkv

#endif  // PKV_TEAM_PARAMS_H
