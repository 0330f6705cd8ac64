// The tcgen05 ragged-attention kernel: bf16, head_dim 64.
#include "attend_prompt_launch.cuh"

namespace pkd {

cudaError_t launch_prompt_bf16_d64(const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p, bool partials,
                               bool overlap, int grid, cudaStream_t stream) {
    return launch_prompt_typed<64, kPtBF16>(kvmap, qmap, p, partials, overlap, grid, stream);
}

}  // namespace pkd
