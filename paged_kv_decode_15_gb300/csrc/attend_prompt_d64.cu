// The tcgen05 ragged-attention kernel at head_dim 64.
#include "attend_prompt_launch.cuh"

namespace pkd {

cudaError_t launch_prompt_d64(bool bf16, const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p,
                               bool partials, int grid, cudaStream_t stream) {
    return bf16 ? launch_prompt_typed<64, true>(kvmap, qmap, p, partials, grid, stream)
                : launch_prompt_typed<64, false>(kvmap, qmap, p, partials, grid, stream);
}

}  // namespace pkd
