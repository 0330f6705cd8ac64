// Host-side entry points of the ragged paged-attention kernels.
#pragma once

#include "launch.h"

namespace pkd {

struct AttendParams;

// Launch `kern`; with overlap as a programmatic dependent of the launch before it
// on the stream: it may start once every CTA of that one has started, and the
// kernel itself waits (griddepcontrol.wait) before it uses that one's results --
// at the latest before it ends, so that its own end implies the other's.
template <class... P, class... A>
cudaError_t launch_kernel(void (*kern)(P...), dim3 grid, int threads, size_t smem, bool overlap, cudaStream_t stream,
                          const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Steps (at most 16 query rows per kv head and request): chunked grid
// (max_splits, Hkv, B).  NT: 8-row tiles of the P.V product.
cudaError_t launch_attend_step(int D, int kv_dtype, int NT, const CUtensorMap& tmap, const AttendParams& a,
                               const DecodeParams& d, dim3 grid, bool overlap, cudaStream_t stream);

// Query blocks of any length on tcgen05 tensor cores: at most `items`
// persistent CTAs.  partials: leave every result as a partial one.  overlap: as
// for launch_kernel.
cudaError_t launch_attend_prompt(int D, int kv_dtype, const CUtensorMap& kvmap, const CUtensorMap& qmap,
                                 const AttendParams& p, bool partials, bool overlap, long long items,
                                 cudaStream_t stream);
#define PKD_PROMPT(name)                                                                                       \
    cudaError_t launch_prompt_##name(const CUtensorMap& kvmap, const CUtensorMap& qmap, const AttendParams& p, \
                                     bool partials, bool overlap, int grid, cudaStream_t stream);
PKD_PROMPT(bf16_d128) PKD_PROMPT(fp16_d128) PKD_PROMPT(fp8_d128) PKD_PROMPT(bf16_d64) PKD_PROMPT(fp16_d64)
#undef PKD_PROMPT

// Joins the partial results of the shared prefix with those of the requests' own keys.
struct PrefixMergeParams {
    const float* part_lse;        // [splits, rows] log2 domain, rows = B * sq * Hq
    const float* part_out;        // [splits, rows, D]
    const float* own_lse;         // [rows] natural log
    const float* own_out;         // [rows, D]
    const int32_t* group_start;   // [groups + 1]
    const int32_t* prefix_lens;   // [groups]
    void* out;
    float* lse;
    int groups, rows, rows_per_request, chunk, max_prefix_len, max_splits, out_dtype;
    float v_scale;
};
cudaError_t launch_prefix_merge(int D, const PrefixMergeParams& p, cudaStream_t stream);

// Tensor maps (cached by value; abi.cu).
pkd_status stage_map(CUtensorMap& out, const void* cache, uint64_t rows, int row_bytes, pkd_dtype dt);
pkd_status half_stage_map(CUtensorMap& out, const void* cache, uint64_t rows, int row_bytes, pkd_dtype dt);
pkd_status query_map(CUtensorMap& out, const void* q, int D, int Hq, uint64_t tokens, int64_t token_stride, int G,
                     int box_tokens, pkd_dtype dt);

}  // namespace pkd
