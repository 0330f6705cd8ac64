// The tcgen05 ragged-attention kernel: fp8, head_dim 128.
#include "attend_prompt_launch.cuh"

namespace pkd {

cudaError_t launch_prompt_fp8_d128(const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p, bool partials,
                               bool overlap, int grid, cudaStream_t stream) {
    return launch_prompt_typed<128, kPtFP8>(kvmap, qmap, p, partials, overlap, grid, stream);
}

}  // namespace pkd
