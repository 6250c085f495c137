// Arguments and launchers of attention with keys and values of their own for G
// groups of query heads: the write of both paged caches, whole prompts, and one
// new token per sequence.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dsaidx {

// Rows of T tokens and some heads: element (t, h, d) is at t * row + h * head + d.
struct HeadRows {
    const void* p;
    int64_t row, head;
};

// The write of both caches: keys rotated, both appended.
struct KvAppendArgs {
    HeadRows in[2];              // keys, values: [T][G][D], bf16 or f32
    const float* cos_sin;        // nullable [rope_len][R]: R/2 cosines, R/2 sines
    const int32_t* seq_ids;      // [T] sequence of each token (outside [0, B): not written)
    const int32_t* positions;    // [T] its position (outside the table or rope_len: not written)
    const int32_t* block_table;  // [B][max_pages] page ids (outside [0, num_pages): not written)
    void* cache[2];              // [num_pages][G][64][D] bf16 or E4M3FN codes
    float* scale[2];             // [num_pages][G][64], fp8 rows only
    int T, G, B, max_pages, num_pages, R, rope_len;
    bool pairs;                  // pair i: columns (2i, 2i+1), else (i, i + R/2)
};

// Causal attention over whole packed sequences.
struct PromptArgs {
    HeadRows q, k, v;            // [T][H][D], [T][G][D], [T][G][V] bf16
    const int32_t* cu;           // [B+1] first row of each sequence
    uint16_t* out;               // [T][H][V] bf16
    float* lse;                  // nullable [T][H]
    float scale_log2;            // softmax scale times log2(e)
    int T, H, G, B;
};

// One new token per sequence over the paged caches.
struct KvDecodeArgs {
    const uint16_t* q;           // [B][H][D] bf16
    const void* cache[2];        // keys, values: [num_pages][G][64][D] bf16 or E4M3FN codes
    const float* scale[2];       // [num_pages][G][64], fp8 rows only
    const int32_t* block_table;  // [B][max_pages] page ids (outside [0, num_pages): a page without rows)
    const int32_t* lens;         // [B] positions of each sequence, clamped to [0, max_ctx]
    const int32_t* idx;          // nullable [B][K] positions (outside the sequence: no row)
    uint16_t* out;               // [B][H][D] bf16
    float* lse;                  // nullable [B][H]
    void* workspace;
    float scale_log2;
    int B, H, G, max_pages, num_pages, max_ctx, K;
};

hipError_t launch_kv_append_rope(const KvAppendArgs& a, int D, bool f32, bool fp8, hipStream_t stream);
int64_t prompt_blocks(int T, int B, int H);   // workgroups of a launch
hipError_t launch_prompt_attention(const PromptArgs& a, int D, hipStream_t stream);
size_t kv_decode_workspace_bytes(int B, int H, int G, int D, int max_ctx, int K, bool fp8);
hipError_t launch_kv_decode(const KvDecodeArgs& a, int D, bool fp8, hipStream_t stream);

}  // namespace dsaidx
