// Launch parameters of the choice of the keys that stay and of the compaction.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkd {

struct SelectParams {
    const float* weights;         // [B, H, keys], strides
    const int32_t* positions;     // the same with strides of its own, or null: key t at position t
    const int32_t* seq_lens;      // [B]
    const int32_t* context_lens;  // [B] with positions, else null: seq_lens
    int32_t* kept;                // [B, H, budget]
    int32_t* kept_lens;           // [B]
    int32_t* status;              // or null
    long long weights_b, weights_h, positions_b, positions_h;
    int B, H, keys, budget, sinks, recent, pool;
};

struct CompactParams {
    uint8_t* cache;
    const int32_t* block_table;   // [B, bt_stride]
    const int32_t* kept;          // [B, H, budget]
    const int32_t* kept_lens;     // [B]
    float* weights;               // [B, H, keys], strides, or null
    int32_t* positions;           // the same with strides of its own, or null
    int32_t* status;              // or null
    long long bt_stride, num_pages, weights_b, weights_h, positions_b, positions_h;
    int B, H, P, keys, budget, row_bytes;  // keys: those of the table (and of weights and positions)
    uint32_t pmagic;
    int pmshift;
};

cudaError_t launch_evict_select(const SelectParams& p, cudaStream_t stream);
cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream);

}  // namespace pkd
