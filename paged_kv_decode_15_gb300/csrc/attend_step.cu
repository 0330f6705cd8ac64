// Instantiations of the step kernel of ragged paged attention.
#include "attend_launch.h"
#include "attend_step.cuh"

namespace pkd {

constexpr int kStepNbuf = 2;  // stages per warp ring, as in the decode grid

template <class W, int D, int ELT>
static cudaError_t launch_one(const CUtensorMap& tmap, const AttendParams& a, const DecodeParams& d, dim3 grid,
                              bool overlap, cudaStream_t stream) {
    using S = StepShape<W, D, ELT, kStepNbuf>;
    // e4m3 stages let four CTAs into an SM (as for the decode grid's five, one fewer
    // for the rows' masks and biases)
    auto kern = attend_step_kernel<W, D, ELT, kStepNbuf, ELT == 1 ? 4 : 1>;
    static PerDevice state;
    cudaError_t e = kernel_setup(state, kern, kNW * 32, S::SMEM);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, kNW * 32, S::SMEM, overlap, stream, tmap, a, d);
}

// NT: 8-row tiles of the P.V product (1 for at most 8 rows)
cudaError_t launch_attend_step(int D, int kv_dtype, int NT, const CUtensorMap& tmap, const AttendParams& a,
                               const DecodeParams& d, dim3 grid, bool overlap, cudaStream_t stream) {
    if (kv_dtype == PKD_FP8_E4M3) {
        if (D != 128) return cudaErrorInvalidValue;
        return NT == 1 ? launch_one<Fp8MmaWarp<1, 1>, 128, 1>(tmap, a, d, grid, overlap, stream)
                       : launch_one<Fp8MmaWarp<1, 2>, 128, 1>(tmap, a, d, grid, overlap, stream);
    }
    const bool bf16 = kv_dtype == PKD_BF16;
#define PKD_STEP(dd, nt)                                                                              \
    if (D == dd && NT == nt)                                                                          \
        return bf16 ? launch_one<MmaWarp<dd, true, 1, nt>, dd, 2>(tmap, a, d, grid, overlap, stream)           \
                    : launch_one<MmaWarp<dd, false, 1, nt>, dd, 2>(tmap, a, d, grid, overlap, stream);
    PKD_STEP(128, 1) PKD_STEP(128, 2) PKD_STEP(64, 1) PKD_STEP(64, 2)
#undef PKD_STEP
    return cudaErrorInvalidValue;
}

}  // namespace pkd
