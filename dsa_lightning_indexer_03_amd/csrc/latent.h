// Arguments and launchers of the operators on the latent cache: the write of
// both caches with its rotation, and attention over the latent rows.  (Apart
// from kernels.h, on whose text the traffic records of other kernels depend.)
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dsaidx {

// The layer's cache write: latent rows and index keys, rotated and appended.
struct AppendRopeArgs {
    const void* kv;              // [T] rows of E elements, kv_stride apart, bf16 or f32
    const void* index_k;         // nullable [T] rows of 128, index_stride apart, the same type
    int64_t kv_stride, index_stride;
    const float* cos_sin;        // [rope_len][R]: R/2 cosines, R/2 sines
    const int32_t* seq_ids;      // [T] sequence of each token (outside [0, B): not written)
    const int32_t* positions;    // [T] its position (outside the table or rope_len: not written)
    const int32_t* block_table;  // [B][max_pages] page ids (outside [0, num_pages): not written)
    void* latent;                // [num_pages][64][E] bf16 or E4M3FN codes
    float* latent_scale;         // [num_pages][64], fp8 rows only
    uint8_t* k_cache;            // [num_pages][64][128] E4M3FN codes
    float* k_scale;              // [num_pages][64]
    int T, B, max_pages, num_pages, E, R, rope_len;
    bool kv_pairs, index_pairs;  // pair i: columns (2i, 2i+1), else (i, i + R/2)
};

// Attention over the paged latent cache (selected rows, or prefix + own rows).
struct LatentArgs {
    const uint16_t* q;           // [T][H][E] bf16
    const void* cache;           // [num_pages][64][E] bf16 or E4M3FN codes
    const float* cache_scale;    // [num_pages][64], fp8 rows only
    const int32_t* block_table;  // [B][max_pages] page ids (outside [0, num_pages): no row)
    const int32_t* idx;          // [T][K] selected positions (outside the table: no row), or null:
    const int32_t* seq_ids;      //   nullable [T]: query t's row of the table (default t)
    const int32_t* prefix_table; // page ids of the shared prefix
    const int32_t* context_lens; // [T] each sequence's own positions
    uint16_t* out;               // [T][H][V] bf16
    float* lse;                  // nullable [T][H]
    void* workspace;
    float scale_log2;            // softmax scale times log2(e)
    int T, H, E, B, max_pages, num_pages, K, prefix_len, max_ctx;
};

hipError_t launch_cache_append_rope(const AppendRopeArgs& a, bool f32, bool fp8, hipStream_t stream);
size_t latent_topk_workspace_bytes(int T, int H, int K, bool fp8);
size_t latent_shared_workspace_bytes(int B, int H, int prefix_len, int max_ctx, bool fp8);
hipError_t launch_latent_attention(const LatentArgs& a, bool fp8, hipStream_t stream);

}  // namespace dsaidx
