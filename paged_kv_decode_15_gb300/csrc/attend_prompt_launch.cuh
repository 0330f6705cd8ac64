// Launch of the tcgen05 ragged-attention kernel for one head_dim and type.
#pragma once

#include "attend_launch.h"
#include "attend_prompt.cuh"

namespace pkd {

template <int D, int kType, bool kCap, bool kBias>
static cudaError_t launch_prompt_one(const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p,
                                     bool partials, bool overlap, int grid, cudaStream_t stream) {
    auto kern = attend_prompt_kernel<D, kType, kCap, kBias>;
    static PerDevice state;
    cudaError_t e = kernel_setup(state, kern, kPtThreads, PtShape<D, kType>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(grid), kPtThreads, PtShape<D, kType>::SMEM, overlap, stream, kvmap, kvmap, qmap, p,
                         partials ? 1 : 0);
}

template <int D, int kType>
static cudaError_t launch_prompt_typed(const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p,
                                       bool partials, bool overlap, int grid, cudaStream_t stream) {
    const bool cap = p.cap_log2 > 0.f, bias = p.slopes != nullptr;
    if (cap)
        return bias ? launch_prompt_one<D, kType, true, true>(kvmap, qmap, p, partials, overlap, grid, stream)
                    : launch_prompt_one<D, kType, true, false>(kvmap, qmap, p, partials, overlap, grid, stream);
    return bias ? launch_prompt_one<D, kType, false, true>(kvmap, qmap, p, partials, overlap, grid, stream)
                : launch_prompt_one<D, kType, false, false>(kvmap, qmap, p, partials, overlap, grid, stream);
}

template <int D, int kType, bool kCap>
static cudaError_t launch_packed_one(const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                                     const AttendParams& p, int grid, cudaStream_t stream) {
    auto kern = attend_prompt_kernel<D, kType, kCap, false, true>;
    static PerDevice state;
    cudaError_t e = kernel_setup(state, kern, kPtThreads, PtShape<D, kType, true>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(grid), kPtThreads, PtShape<D, kType, true>::SMEM, false, stream, kmap, vmap, qmap, p, 0);
}

}  // namespace pkd
