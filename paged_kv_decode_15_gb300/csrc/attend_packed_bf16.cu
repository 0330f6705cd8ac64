// The tcgen05 ragged-attention kernel on packed keys and values: bf16.
#include "attend_prompt_launch.cuh"

namespace pkd {

cudaError_t launch_packed_bf16(int D, const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                              const AttendParams& p, int grid, cudaStream_t stream) {
    const bool cap = p.cap_log2 > 0.f;
    if (D == 128)
        return cap ? launch_packed_one<128, kPtBF16, true>(kmap, vmap, qmap, p, grid, stream)
                   : launch_packed_one<128, kPtBF16, false>(kmap, vmap, qmap, p, grid, stream);
    return cap ? launch_packed_one<64, kPtBF16, true>(kmap, vmap, qmap, p, grid, stream)
               : launch_packed_one<64, kPtBF16, false>(kmap, vmap, qmap, p, grid, stream);
}

}  // namespace pkd
