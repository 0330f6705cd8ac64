// Instantiations of the tcgen05 kernel of pkd_key_weights.
#include "attend_launch.h"
#include "key_weights_tc05.cuh"

namespace pkd {

template <int D, int kType, bool kCap>
static cudaError_t launch_tc05(const CUtensorMap& kvmap, const CUtensorMap& qmap, const WeighParams& w, long long items,
                               cudaStream_t stream) {
    auto kern = key_weights_tc05_kernel<D, kType, kCap>;
    static PerDevice state;
    int grid = 1;
    cudaError_t e = persistent_grid(1, static_cast<int>(items < 152 ? items : 152), grid);
    if (e == cudaSuccess) e = kernel_setup(state, kern, kWtThreads, WtShape<D, kType>::SMEM);
    if (e != cudaSuccess) return e;
    // the roles' registers come out of those of the launch: a kernel that got fewer would wait for ever
    static const bool fits = [&] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs * kWtThreads >= 512 * kWtRegsExp + 128 * kWtRegsOther;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    return launch_kernel(kern, dim3(grid), kWtThreads, WtShape<D, kType>::SMEM, false, stream, kvmap, qmap, w);
}

cudaError_t launch_key_weights_tc05(int D, int kv_dtype, const CUtensorMap& kvmap, const CUtensorMap& qmap,
                                    const WeighParams& w, long long items, cudaStream_t stream) {
    const bool cap = w.a.cap_log2 > 0.f;
#define PKD_WT(d, t)                                                                            \
    if (D == d && kv_dtype == t)                                                                \
        return cap ? launch_tc05<d, t, true>(kvmap, qmap, w, items, stream) : launch_tc05<d, t, false>(kvmap, qmap, w, items, stream);
    PKD_WT(128, 0) PKD_WT(128, 1) PKD_WT(128, 2) PKD_WT(64, 0) PKD_WT(64, 1)
#undef PKD_WT
    return cudaErrorInvalidValue;
}

}  // namespace pkd
