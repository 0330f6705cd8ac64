// The tcgen05 ragged-attention kernel at head_dim 128.
#include "attend_prompt_launch.cuh"

namespace pkd {

cudaError_t launch_prompt_d128(bool bf16, const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p,
                               bool partials, int grid, cudaStream_t stream) {
    return bf16 ? launch_prompt_typed<128, true>(kvmap, qmap, p, partials, grid, stream)
                : launch_prompt_typed<128, false>(kvmap, qmap, p, partials, grid, stream);
}

}  // namespace pkd
