// C ABI of the lightning-indexer library: argument checks (all on the host,
// before any launch), workspace sizing and kernel dispatch.  The entry points
// are documented in include/dsaidx.h.
#include <stdarg.h>
#include <stdio.h>

#include "device_once.h"
#include "dsaidx.h"
#include "kernels.h"
#include "kv.h"
#include "latent.h"

namespace {

thread_local char g_err[320];

dsaidx_status fail(dsaidx_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return s;
}

dsaidx_status hip_fail(hipError_t e, const char* what) {
    return fail(DSAIDX_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

using dsaidx::kMaxTopk;
constexpr int kMaxL = 131072;
constexpr int kMaxSelectCols = 4194304;

bool prefill_is_fused(int dtype, int H, int D) {
    return (dtype == DSAIDX_BF16 || dtype == DSAIDX_FP8_E4M3) && D == 128 && H % 16 == 0 && H >= 16 && H <= 64;
}

size_t decode_score_stride(int max_ctx) { return (size_t)((max_ctx + 63) / 64) * 64; }

}  // namespace

extern "C" {

int dsaidx_version(void) { return 100; }

const char* dsaidx_status_string(int s) {
    switch (s) {
        case DSAIDX_OK: return "ok";
        case DSAIDX_ERR_NULL: return "required pointer is NULL";
        case DSAIDX_ERR_SHAPE: return "invalid or inconsistent size";
        case DSAIDX_ERR_DTYPE: return "unknown dtype";
        case DSAIDX_ERR_UNSUPPORTED: return "outside the supported ranges";
        case DSAIDX_ERR_WORKSPACE: return "workspace too small";
        case DSAIDX_ERR_HIP: return "HIP launch failed";
        default: return "unknown status";
    }
}

const char* dsaidx_last_error(void) { return g_err; }

dsaidx_status indexer_kcache_append(const void* k, int k_dtype, const int32_t* seq_ids,
                                    const int32_t* positions, const int32_t* block_table, int B,
                                    int max_pages_per_seq, uint8_t* k_cache, float* k_scale, int num_pages,
                                    int T, int D, int page_size, void* stream) {
    g_err[0] = 0;
    if (T < 0 || B < 1 || max_pages_per_seq < 1 || num_pages < 1 || D < 1 || page_size < 1)
        return fail(DSAIDX_ERR_SHAPE, "T=%d B=%d max_pages_per_seq=%d num_pages=%d D=%d page_size=%d", T, B,
                    max_pages_per_seq, num_pages, D, page_size);
    if (k_dtype != DSAIDX_F32 && k_dtype != DSAIDX_BF16 && k_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "k_dtype=%d", k_dtype);
    if (k_dtype == DSAIDX_FP8_E4M3) return fail(DSAIDX_ERR_UNSUPPORTED, "new keys must be bf16 or f32");
    if (D != 128) return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d (128)", D);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if (T == 0) return DSAIDX_OK;
    if (!k) return fail(DSAIDX_ERR_NULL, "k is NULL");
    if (!seq_ids) return fail(DSAIDX_ERR_NULL, "seq_ids is NULL");
    if (!positions) return fail(DSAIDX_ERR_NULL, "positions is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!k_cache) return fail(DSAIDX_ERR_NULL, "k_cache is NULL");
    if (!k_scale) return fail(DSAIDX_ERR_NULL, "k_scale is NULL");
    if (!aligned16(k) || ((uintptr_t)k_cache & 7u) != 0)
        return fail(DSAIDX_ERR_UNSUPPORTED, "k must be 16-byte and k_cache 8-byte aligned");
    dsaidx::KcacheArgs a{};
    a.k = k;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.block_table = block_table;
    a.k_cache = k_cache;
    a.k_scale = k_scale;
    a.T = T;
    a.B = B;
    a.max_pages = max_pages_per_seq;
    const hipError_t e = dsaidx::launch_kcache_append(a, k_dtype == DSAIDX_BF16 ? 1 : 0, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_kcache_append");
    return DSAIDX_OK;
}

dsaidx_status indexer_topk_gather(const void* latent_cache, int row_bytes, const int32_t* block_table,
                                  int max_pages_per_seq, int num_pages, int page_size,
                                  const int32_t* topk_idx, int B, int topk, void* out, void* stream) {
    g_err[0] = 0;
    if (!latent_cache) return fail(DSAIDX_ERR_NULL, "latent_cache is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!topk_idx) return fail(DSAIDX_ERR_NULL, "topk_idx is NULL");
    if (!out) return fail(DSAIDX_ERR_NULL, "out is NULL");
    if (B < 1 || topk < 1 || max_pages_per_seq < 1 || num_pages < 1 || page_size < 1 || row_bytes < 1)
        return fail(DSAIDX_ERR_SHAPE, "B=%d topk=%d max_pages_per_seq=%d num_pages=%d page_size=%d row_bytes=%d",
                    B, topk, max_pages_per_seq, num_pages, page_size, row_bytes);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if (row_bytes % 16 != 0 || row_bytes > 65536)
        return fail(DSAIDX_ERR_UNSUPPORTED, "row_bytes=%d (a multiple of 16, at most 65536)", row_bytes);
    if (!aligned16(latent_cache) || !aligned16(out))
        return fail(DSAIDX_ERR_UNSUPPORTED, "latent_cache and out must be 16-byte aligned");
    dsaidx::GatherArgs a{};
    a.cache = reinterpret_cast<const uint8_t*>(latent_cache);
    a.block_table = block_table;
    a.idx = topk_idx;
    a.out = reinterpret_cast<uint8_t*>(out);
    a.B = B;
    a.K = topk;
    a.max_pages = max_pages_per_seq;
    a.row_bytes = row_bytes;
    const hipError_t e = dsaidx::launch_topk_gather(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_topk_gather");
    return DSAIDX_OK;
}

dsaidx_status indexer_topk_gather_layers(const void* const* latent_caches, void* const* outs, int n_layers,
                                         int row_bytes, const int32_t* block_table, int max_pages_per_seq,
                                         int num_pages, int page_size, const int32_t* topk_idx, int B, int topk,
                                         void* stream) {
    g_err[0] = 0;
    if (!latent_caches) return fail(DSAIDX_ERR_NULL, "latent_caches is NULL");
    if (!outs) return fail(DSAIDX_ERR_NULL, "outs is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!topk_idx) return fail(DSAIDX_ERR_NULL, "topk_idx is NULL");
    if (n_layers < 1 || B < 1 || topk < 1 || max_pages_per_seq < 1 || num_pages < 1 || page_size < 1 ||
        row_bytes < 1)
        return fail(DSAIDX_ERR_SHAPE,
                    "n_layers=%d B=%d topk=%d max_pages_per_seq=%d num_pages=%d page_size=%d row_bytes=%d",
                    n_layers, B, topk, max_pages_per_seq, num_pages, page_size, row_bytes);
    if (n_layers > dsaidx::kMaxGatherLayers)
        return fail(DSAIDX_ERR_UNSUPPORTED, "n_layers=%d (at most %d per call)", n_layers,
                    dsaidx::kMaxGatherLayers);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if (row_bytes % 16 != 0 || row_bytes > 65536)
        return fail(DSAIDX_ERR_UNSUPPORTED, "row_bytes=%d (a multiple of 16, at most 65536)", row_bytes);
    dsaidx::GatherLayersArgs a{};
    for (int l = 0; l < n_layers; ++l) {
        if (!latent_caches[l]) return fail(DSAIDX_ERR_NULL, "latent_caches[%d] is NULL", l);
        if (!outs[l]) return fail(DSAIDX_ERR_NULL, "outs[%d] is NULL", l);
        if (!aligned16(latent_caches[l]) || !aligned16(outs[l]))
            return fail(DSAIDX_ERR_UNSUPPORTED, "latent_caches[%d] and outs[%d] must be 16-byte aligned", l, l);
        a.cache[l] = reinterpret_cast<const uint8_t*>(latent_caches[l]);
        a.out[l] = reinterpret_cast<uint8_t*>(outs[l]);
    }
    a.block_table = block_table;
    a.idx = topk_idx;
    a.B = B;
    a.K = topk;
    a.max_pages = max_pages_per_seq;
    a.row_bytes = row_bytes;
    a.n_layers = n_layers;
    const hipError_t e = dsaidx::launch_topk_gather_layers(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_topk_gather_layers");
    return DSAIDX_OK;
}

dsaidx_status indexer_cache_append_rope(const void* kv, int64_t kv_stride, int kv_interleaved, const void* index_k,
                                        int64_t index_stride, int index_interleaved, int in_dtype,
                                        const float* cos_sin, int rope_len, int rope_dim, const int32_t* seq_ids,
                                        const int32_t* positions, const int32_t* block_table, int B,
                                        int max_pages_per_seq, void* latent_cache, float* latent_scale,
                                        int latent_dtype, uint8_t* k_cache, float* k_scale, int num_pages, int T,
                                        int E, int D, int page_size, void* stream) {
    g_err[0] = 0;
    if (T < 0 || B < 1 || max_pages_per_seq < 1 || num_pages < 1 || E < 1 || D < 1 || page_size < 1 || rope_len < 1 ||
        rope_dim < 1)
        return fail(DSAIDX_ERR_SHAPE,
                    "T=%d B=%d max_pages_per_seq=%d num_pages=%d E=%d D=%d page_size=%d rope_len=%d rope_dim=%d", T, B,
                    max_pages_per_seq, num_pages, E, D, page_size, rope_len, rope_dim);
    if (in_dtype != DSAIDX_F32 && in_dtype != DSAIDX_BF16 && in_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "in_dtype=%d", in_dtype);
    if (latent_dtype != DSAIDX_F32 && latent_dtype != DSAIDX_BF16 && latent_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "latent_dtype=%d", latent_dtype);
    if (in_dtype == DSAIDX_FP8_E4M3) return fail(DSAIDX_ERR_UNSUPPORTED, "new rows must be bf16 or f32");
    if (latent_dtype == DSAIDX_F32) return fail(DSAIDX_ERR_UNSUPPORTED, "the latent cache must be bf16 or fp8");
    if (D != 128) return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d (128)", D);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if (E % 8 != 0 || E > 1024) return fail(DSAIDX_ERR_UNSUPPORTED, "E=%d (a multiple of 8, at most 1024)", E);
    if (rope_dim % 16 != 0 || rope_dim > 128 || rope_dim > E)
        return fail(DSAIDX_ERR_UNSUPPORTED, "rope_dim=%d (a multiple of 16, at most 128 and E)", rope_dim);
    if ((latent_dtype == DSAIDX_FP8_E4M3) != (latent_scale != nullptr))
        return fail(DSAIDX_ERR_SHAPE, "latent_scale goes with an fp8 latent cache, NULL with a bf16 one");
    if ((index_k != nullptr) != (k_cache != nullptr) || (index_k != nullptr) != (k_scale != nullptr))
        return fail(DSAIDX_ERR_SHAPE, "index_k, k_cache and k_scale are given together or not at all");
    // (a wave a token, and a launch holds less than 2^32 threads)
    if (T > 1 << 25) return fail(DSAIDX_ERR_UNSUPPORTED, "T=%d > 2^25", T);
    if (T == 0) return DSAIDX_OK;
    if (!kv) return fail(DSAIDX_ERR_NULL, "kv is NULL");
    if (!cos_sin) return fail(DSAIDX_ERR_NULL, "cos_sin is NULL");
    if (!seq_ids) return fail(DSAIDX_ERR_NULL, "seq_ids is NULL");
    if (!positions) return fail(DSAIDX_ERR_NULL, "positions is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!latent_cache) return fail(DSAIDX_ERR_NULL, "latent_cache is NULL");
    if (T > 1 && (kv_stride < E || (index_k && index_stride < D)))
        return fail(DSAIDX_ERR_SHAPE, "kv_stride=%lld < E=%d or index_stride=%lld < D=%d", (long long)kv_stride, E,
                    (long long)index_stride, D);
    const int per16 = in_dtype == DSAIDX_BF16 ? 8 : 4;  // elements of 16 bytes
    if (!aligned16(kv) || !aligned16(index_k) || !aligned16(cos_sin) || !aligned16(latent_cache) ||
        ((uintptr_t)k_cache & 7u) != 0 || (T > 1 && (kv_stride % per16 != 0 || (index_k && index_stride % per16 != 0))))
        return fail(DSAIDX_ERR_UNSUPPORTED,
                    "kv and index_k rows, cos_sin and latent_cache must be 16-byte, k_cache 8-byte aligned");
    dsaidx::AppendRopeArgs a{};
    a.kv = kv;
    a.index_k = index_k;
    a.kv_stride = kv_stride;
    a.index_stride = index_stride;
    a.cos_sin = cos_sin;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.block_table = block_table;
    a.latent = latent_cache;
    a.latent_scale = latent_scale;
    a.k_cache = k_cache;
    a.k_scale = k_scale;
    a.T = T;
    a.B = B;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.E = E;
    a.R = rope_dim;
    a.rope_len = rope_len;
    a.kv_pairs = kv_interleaved != 0;
    a.index_pairs = index_interleaved != 0;
    const hipError_t e = dsaidx::launch_cache_append_rope(a, in_dtype == DSAIDX_F32, latent_dtype == DSAIDX_FP8_E4M3,
                                                          (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_cache_append_rope");
    return DSAIDX_OK;
}

}  // extern "C"

namespace {

constexpr int kMaxLatentTokens = 1 << 27;  // longest list of keys of one query
constexpr int kMaxLatentHeads = 128;
constexpr float kLog2E = 1.44269504088896341f;

// The checks that both latent-attention entry points share; 0 when all pass.
dsaidx_status latent_check(const void* q, int q_dtype, const void* latent_cache, const float* latent_scale,
                           int latent_dtype, const int32_t* block_table, int max_pages_per_seq, int num_pages, int B,
                           int T, int H, int E, int V, int page_size, float scale, const void* out) {
    if (T < 0 || B < 1 || H < 1 || E < 1 || V < 1 || page_size < 1 || num_pages < 1 || max_pages_per_seq < 1)
        return fail(DSAIDX_ERR_SHAPE, "rows=%d B=%d H=%d E=%d V=%d page_size=%d num_pages=%d max_pages_per_seq=%d", T,
                    B, H, E, V, page_size, num_pages, max_pages_per_seq);
    if (q_dtype != DSAIDX_F32 && q_dtype != DSAIDX_BF16 && q_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "q_dtype=%d", q_dtype);
    if (latent_dtype != DSAIDX_F32 && latent_dtype != DSAIDX_BF16 && latent_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "latent_dtype=%d", latent_dtype);
    if (q_dtype != DSAIDX_BF16) return fail(DSAIDX_ERR_UNSUPPORTED, "queries must be bf16");
    if (latent_dtype == DSAIDX_F32) return fail(DSAIDX_ERR_UNSUPPORTED, "the latent cache must be bf16 or fp8");
    if ((latent_dtype == DSAIDX_FP8_E4M3) != (latent_scale != nullptr))
        return fail(DSAIDX_ERR_SHAPE, "latent_scale goes with an fp8 latent cache, NULL with a bf16 one");
    if (V != 512 || (E != 512 && E != 576))
        return fail(DSAIDX_ERR_UNSUPPORTED, "E=%d V=%d (E 512 or 576, V 512)", E, V);
    if (H > kMaxLatentHeads) return fail(DSAIDX_ERR_UNSUPPORTED, "H=%d > %d", H, kMaxLatentHeads);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if ((int64_t)max_pages_per_seq * page_size > kMaxLatentTokens || num_pages > kMaxLatentTokens / 64)
        return fail(DSAIDX_ERR_UNSUPPORTED, "max_pages_per_seq=%d num_pages=%d (tables and pools of at most %d tokens)",
                    max_pages_per_seq, num_pages, kMaxLatentTokens);
    // (a launch holds less than 2^32 threads; a query whose keys are not cut takes a
    // workgroup of 256 up to 16 heads, of 512 above, and plans with more parts are
    // taken only where they fit)
    if ((int64_t)T * H > (1 << 23)) return fail(DSAIDX_ERR_UNSUPPORTED, "rows * H = %lld > 2^23", (long long)T * H);
    const float in_base_2 = scale * kLog2E;
    if (!(in_base_2 - in_base_2 == 0.f)) return fail(DSAIDX_ERR_SHAPE, "scale * log2(e) must be finite");
    if (T == 0) return DSAIDX_OK;
    if (!q) return fail(DSAIDX_ERR_NULL, "q is NULL");
    if (!latent_cache) return fail(DSAIDX_ERR_NULL, "latent_cache is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!out) return fail(DSAIDX_ERR_NULL, "out is NULL");
    if (!aligned16(q) || !aligned16(latent_cache) || !aligned16(out))
        return fail(DSAIDX_ERR_UNSUPPORTED, "q, latent_cache and out must be 16-byte aligned");
    return DSAIDX_OK;
}

dsaidx_status latent_run(dsaidx::LatentArgs& a, int latent_dtype, float scale, void* workspace,
                         size_t workspace_bytes, size_t need, const char* name, void* stream) {
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSAIDX_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need > 0 && !aligned16(workspace)) return fail(DSAIDX_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    a.workspace = workspace;
    a.scale_log2 = scale * kLog2E;
    const hipError_t e = dsaidx::launch_latent_attention(a, latent_dtype == DSAIDX_FP8_E4M3, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, name);
    return DSAIDX_OK;
}

}  // namespace

extern "C" {

size_t indexer_latent_attention_topk_workspace_bytes(int T, int H, int E, int V, int topk, int latent_dtype) {
    (void)E; (void)V;
    if (T < 1 || H < 1 || topk < 1) return 0;
    return dsaidx::latent_topk_workspace_bytes(T, H, topk, latent_dtype == DSAIDX_FP8_E4M3);
}

dsaidx_status indexer_latent_attention_topk(const void* q, int q_dtype, const void* latent_cache,
                                            const float* latent_scale, int latent_dtype, const int32_t* block_table,
                                            int max_pages_per_seq, int num_pages, const int32_t* topk_idx,
                                            const int32_t* seq_ids, int B, int T, int H, int E, int V, int page_size,
                                            int topk, float scale, void* out, float* lse, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    g_err[0] = 0;
    const dsaidx_status st = latent_check(q, q_dtype, latent_cache, latent_scale, latent_dtype, block_table,
                                          max_pages_per_seq, num_pages, B, T, H, E, V, page_size, scale, out);
    if (st != DSAIDX_OK) return st;
    if (topk < 1) return fail(DSAIDX_ERR_SHAPE, "topk=%d must be >= 1", topk);
    if (topk > kMaxL) return fail(DSAIDX_ERR_UNSUPPORTED, "topk=%d > %d", topk, kMaxL);
    if (!seq_ids && T > B) return fail(DSAIDX_ERR_SHAPE, "T=%d > B=%d needs seq_ids", T, B);
    if (T == 0) return DSAIDX_OK;
    if (!topk_idx) return fail(DSAIDX_ERR_NULL, "topk_idx is NULL");
    dsaidx::LatentArgs a{};
    a.q = reinterpret_cast<const uint16_t*>(q);
    a.cache = latent_cache;
    a.cache_scale = latent_scale;
    a.block_table = block_table;
    a.idx = topk_idx;
    a.seq_ids = seq_ids;
    a.out = reinterpret_cast<uint16_t*>(out);
    a.lse = lse;
    a.T = T;
    a.H = H;
    a.E = E;
    a.B = B;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.K = topk;
    return latent_run(a, latent_dtype, scale, workspace, workspace_bytes,
                      indexer_latent_attention_topk_workspace_bytes(T, H, E, V, topk, latent_dtype),
                      "indexer_latent_attention_topk", stream);
}

size_t indexer_latent_attention_shared_workspace_bytes(int B, int H, int E, int V, int prefix_len,
                                                       int max_context_len, int latent_dtype) {
    (void)E; (void)V;
    if (B < 1 || H < 1 || prefix_len < 0 || max_context_len < 0) return 0;
    return dsaidx::latent_shared_workspace_bytes(B, H, prefix_len, max_context_len, latent_dtype == DSAIDX_FP8_E4M3);
}

dsaidx_status indexer_latent_attention_shared(const void* q, int q_dtype, const void* latent_cache,
                                              const float* latent_scale, int latent_dtype,
                                              const int32_t* prefix_table, int prefix_pages, int prefix_len,
                                              const int32_t* block_table, int max_pages_per_seq, int num_pages,
                                              const int32_t* context_lens, int max_context_len, int B, int H, int E,
                                              int V, int page_size, float scale, void* out, float* lse,
                                              void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = 0;
    const dsaidx_status st = latent_check(q, q_dtype, latent_cache, latent_scale, latent_dtype, block_table,
                                          max_pages_per_seq, num_pages, B < 1 ? 1 : B, B, H, E, V, page_size, scale,
                                          out);
    if (st != DSAIDX_OK) return st;
    if (prefix_pages < 0 || prefix_len < 0 || (int64_t)prefix_len > (int64_t)prefix_pages * page_size)
        return fail(DSAIDX_ERR_SHAPE, "prefix_len=%d in %d pages", prefix_len, prefix_pages);
    if (max_context_len < 0 || (int64_t)max_context_len > (int64_t)max_pages_per_seq * page_size)
        return fail(DSAIDX_ERR_SHAPE, "max_context_len=%d > max_pages_per_seq*page_size=%lld", max_context_len,
                    (long long)max_pages_per_seq * page_size);
    if (prefix_len > kMaxLatentTokens) return fail(DSAIDX_ERR_UNSUPPORTED, "prefix_len=%d > %d", prefix_len, kMaxLatentTokens);
    if (B == 0) return DSAIDX_OK;
    if (prefix_len > 0 && !prefix_table) return fail(DSAIDX_ERR_NULL, "prefix_table is NULL");
    if (!context_lens) return fail(DSAIDX_ERR_NULL, "context_lens is NULL");
    dsaidx::LatentArgs a{};
    a.q = reinterpret_cast<const uint16_t*>(q);
    a.cache = latent_cache;
    a.cache_scale = latent_scale;
    a.block_table = block_table;
    a.prefix_table = prefix_table;
    a.context_lens = context_lens;
    a.out = reinterpret_cast<uint16_t*>(out);
    a.lse = lse;
    a.T = B;
    a.H = H;
    a.E = E;
    a.B = B;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.prefix_len = prefix_len;
    a.max_ctx = max_context_len;
    return latent_run(a, latent_dtype, scale, workspace, workspace_bytes,
                      indexer_latent_attention_shared_workspace_bytes(B, H, E, V, prefix_len, max_context_len,
                                                                      latent_dtype),
                      "indexer_latent_attention_shared", stream);
}

}  // extern "C"

namespace {

constexpr int kMaxKvHeads = 128;
constexpr int kMaxKvRows = 1 << 23;        // query rows of a decode call: B * H

// Heads and scale of the attention calls with keys and values of G groups.
dsaidx_status kv_heads_check(int H, int G, float scale) {
    if (H < 1 || G < 1 || H % G != 0) return fail(DSAIDX_ERR_SHAPE, "H=%d G=%d (H a multiple of G)", H, G);
    if (H > kMaxKvHeads) return fail(DSAIDX_ERR_UNSUPPORTED, "H=%d > %d", H, kMaxKvHeads);
    const float in_base_2 = scale * kLog2E;
    if (!(in_base_2 - in_base_2 == 0.f)) return fail(DSAIDX_ERR_SHAPE, "scale * log2(e) must be finite");
    return DSAIDX_OK;
}

// The paged key and value caches; `empty`: a call without rows, whose pointers may be NULL.
dsaidx_status kv_caches_check(const void* k_cache, const float* k_scale, const void* v_cache, const float* v_scale,
                              int cache_dtype, int num_pages, int G, int D, int page_size, int max_pages_per_seq,
                              bool empty) {
    if (D < 1 || page_size < 1 || num_pages < 1)
        return fail(DSAIDX_ERR_SHAPE, "D=%d page_size=%d num_pages=%d", D, page_size, num_pages);
    if (cache_dtype != DSAIDX_F32 && cache_dtype != DSAIDX_BF16 && cache_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "cache_dtype=%d", cache_dtype);
    if (cache_dtype == DSAIDX_F32) return fail(DSAIDX_ERR_UNSUPPORTED, "the caches must be bf16 or fp8");
    if (D != 64 && D != 128) return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d (64 or 128)", D);
    if (G > kMaxKvHeads) return fail(DSAIDX_ERR_UNSUPPORTED, "G=%d > %d", G, kMaxKvHeads);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    // (rows of a pool are counted in 31 bits, positions of a table in 27)
    if ((int64_t)max_pages_per_seq * page_size > kMaxLatentTokens ||
        (int64_t)num_pages * G * page_size > 0x7FFFFFFF)
        return fail(DSAIDX_ERR_UNSUPPORTED, "max_pages_per_seq=%d num_pages=%d G=%d (tables of at most %d tokens, pools "
                    "of less than 2^31 rows)", max_pages_per_seq, num_pages, G, kMaxLatentTokens);
    if (empty) return DSAIDX_OK;
    if (!k_cache) return fail(DSAIDX_ERR_NULL, "k_cache is NULL");
    if (!v_cache) return fail(DSAIDX_ERR_NULL, "v_cache is NULL");
    const bool fp8 = cache_dtype == DSAIDX_FP8_E4M3;
    if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr))
        return fail(DSAIDX_ERR_SHAPE, "k_scale and v_scale go with fp8 caches, NULL with bf16 ones");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(DSAIDX_ERR_UNSUPPORTED, "k_cache and v_cache must be 16-byte aligned");
    return DSAIDX_OK;
}

// Every row of [T][heads] starts at 16 bytes (`per16` elements).
bool heads_ok(const void* p, int64_t stride, int64_t head_stride, int T, int heads, int per16) {
    return aligned16(p) && (T <= 1 || stride % per16 == 0) && (heads <= 1 || head_stride % per16 == 0);
}

}  // namespace

extern "C" {

dsaidx_status indexer_kv_append_rope(const void* k, int64_t k_stride, int64_t k_head_stride, const void* v,
                                     int64_t v_stride, int64_t v_head_stride, int in_dtype, const float* cos_sin,
                                     int rope_len, int rope_dim, int interleaved, const int32_t* seq_ids,
                                     const int32_t* positions, const int32_t* block_table, int B,
                                     int max_pages_per_seq, void* k_cache, float* k_scale, void* v_cache,
                                     float* v_scale, int cache_dtype, int num_pages, int T, int G, int D,
                                     int page_size, void* stream) {
    g_err[0] = 0;
    if (T < 0 || B < 1 || max_pages_per_seq < 1 || G < 1 || (cos_sin && (rope_len < 1 || rope_dim < 1)))
        return fail(DSAIDX_ERR_SHAPE, "T=%d B=%d max_pages_per_seq=%d G=%d rope_len=%d rope_dim=%d", T, B,
                    max_pages_per_seq, G, rope_len, rope_dim);
    if (in_dtype != DSAIDX_F32 && in_dtype != DSAIDX_BF16 && in_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "in_dtype=%d", in_dtype);
    if (in_dtype == DSAIDX_FP8_E4M3) return fail(DSAIDX_ERR_UNSUPPORTED, "new rows must be bf16 or f32");
    const dsaidx_status st = kv_caches_check(k_cache, k_scale, v_cache, v_scale, cache_dtype, num_pages, G, D,
                                             page_size, max_pages_per_seq, T == 0);
    if (st != DSAIDX_OK) return st;
    if (cos_sin && (rope_dim % 16 != 0 || rope_dim > D))
        return fail(DSAIDX_ERR_UNSUPPORTED, "rope_dim=%d (a multiple of 16, at most D)", rope_dim);
    // (16 lanes a token and head, and a launch holds less than 2^32 threads)
    if ((int64_t)T * G > 1 << 26) return fail(DSAIDX_ERR_UNSUPPORTED, "T * G = %lld > 2^26", (long long)T * G);
    if (T == 0) return DSAIDX_OK;
    if (!k) return fail(DSAIDX_ERR_NULL, "k is NULL");
    if (!v) return fail(DSAIDX_ERR_NULL, "v is NULL");
    if (!seq_ids) return fail(DSAIDX_ERR_NULL, "seq_ids is NULL");
    if (!positions) return fail(DSAIDX_ERR_NULL, "positions is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    const int per16 = in_dtype == DSAIDX_BF16 ? 8 : 4;  // elements of 16 bytes
    if (!heads_ok(k, k_stride, k_head_stride, T, G, per16) || !heads_ok(v, v_stride, v_head_stride, T, G, per16) ||
        !aligned16(cos_sin))
        return fail(DSAIDX_ERR_UNSUPPORTED, "rows of k and v and cos_sin must be 16-byte aligned");
    dsaidx::KvAppendArgs a{};
    a.in[0] = {k, k_stride, k_head_stride};
    a.in[1] = {v, v_stride, v_head_stride};
    a.cos_sin = cos_sin;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.block_table = block_table;
    a.cache[0] = k_cache;
    a.cache[1] = v_cache;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.T = T;
    a.G = G;
    a.B = B;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.R = cos_sin ? rope_dim : 0;
    a.rope_len = cos_sin ? rope_len : 0x7FFFFFFF;
    a.pairs = interleaved != 0;
    const hipError_t e = dsaidx::launch_kv_append_rope(a, D, in_dtype == DSAIDX_F32, cache_dtype == DSAIDX_FP8_E4M3,
                                                       (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_kv_append_rope");
    return DSAIDX_OK;
}

dsaidx_status indexer_prompt_attention(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k,
                                       int64_t k_stride, int64_t k_head_stride, const void* v, int64_t v_stride,
                                       int64_t v_head_stride, int dtype, const int32_t* cu_seqlens, int B, int T,
                                       int H, int G, int D, int V, float scale, void* out, float* lse, void* stream) {
    g_err[0] = 0;
    if (T < 0 || B < 1) return fail(DSAIDX_ERR_SHAPE, "T=%d B=%d", T, B);
    if (dtype != DSAIDX_F32 && dtype != DSAIDX_BF16 && dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "dtype=%d", dtype);
    if (dtype != DSAIDX_BF16) return fail(DSAIDX_ERR_UNSUPPORTED, "q, k and v must be bf16");
    const dsaidx_status st = kv_heads_check(H, G, scale);
    if (st != DSAIDX_OK) return st;
    if (!((D == 64 && V == 64) || ((D == 128 || D == 192) && V == 128)))
        return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d V=%d (64 and 64, 128 and 128, or 192 and 128)", D, V);
    // (a launch holds less than 2^32 threads, 256 a workgroup where there are many)
    if (dsaidx::prompt_blocks(T, B, H) >= 1 << 24)
        return fail(DSAIDX_ERR_UNSUPPORTED, "T=%d B=%d H=%d: 2^24 blocks of rows or more", T, B, H);
    if (T == 0) return DSAIDX_OK;
    if (!q) return fail(DSAIDX_ERR_NULL, "q is NULL");
    if (!k) return fail(DSAIDX_ERR_NULL, "k is NULL");
    if (!v) return fail(DSAIDX_ERR_NULL, "v is NULL");
    if (!cu_seqlens) return fail(DSAIDX_ERR_NULL, "cu_seqlens is NULL");
    if (!out) return fail(DSAIDX_ERR_NULL, "out is NULL");
    if (!heads_ok(q, q_stride, q_head_stride, T, H, 8) || !heads_ok(k, k_stride, k_head_stride, T, G, 8) ||
        !heads_ok(v, v_stride, v_head_stride, T, G, 8) || !aligned16(out))
        return fail(DSAIDX_ERR_UNSUPPORTED, "rows of q, k and v and out must be 16-byte aligned");
    // (a tile's rows are addressed with 32 bits)
    if (T > 1 && (q_stride < 0 || k_stride < 0 || v_stride < 0 || q_stride >= 1 << 24 || k_stride >= 1 << 24 ||
                  v_stride >= 1 << 24))
        return fail(DSAIDX_ERR_UNSUPPORTED, "q_stride=%lld k_stride=%lld v_stride=%lld (in [0, 2^24))",
                    (long long)q_stride, (long long)k_stride, (long long)v_stride);
    dsaidx::PromptArgs a{};
    a.q = {q, q_stride, q_head_stride};
    a.k = {k, k_stride, k_head_stride};
    a.v = {v, v_stride, v_head_stride};
    a.cu = cu_seqlens;
    a.out = reinterpret_cast<uint16_t*>(out);
    a.lse = lse;
    a.scale_log2 = scale * kLog2E;
    a.T = T;
    a.H = H;
    a.G = G;
    a.B = B;
    const hipError_t e = dsaidx::launch_prompt_attention(a, D, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_prompt_attention");
    return DSAIDX_OK;
}

size_t indexer_kv_attention_decode_workspace_bytes(int B, int H, int G, int D, int max_context_len, int topk,
                                                   int cache_dtype) {
    // (what the call refuses has no plan: its size is 0, and the call says why)
    if (B < 1 || G < 1 || H < G || H % G != 0 || H > kMaxKvHeads || (int64_t)B * H > kMaxKvRows ||
        (D != 64 && D != 128) || max_context_len < 0 || max_context_len > kMaxLatentTokens || topk < 0 ||
        topk > kMaxL || (cache_dtype != DSAIDX_BF16 && cache_dtype != DSAIDX_FP8_E4M3))
        return 0;
    return dsaidx::kv_decode_workspace_bytes(B, H, G, D, max_context_len, topk, cache_dtype == DSAIDX_FP8_E4M3);
}

dsaidx_status indexer_kv_attention_decode(const void* q, int q_dtype, const void* k_cache, const float* k_scale,
                                          const void* v_cache, const float* v_scale, int cache_dtype,
                                          const int32_t* block_table, int max_pages_per_seq, int num_pages,
                                          const int32_t* context_lens, int max_context_len, const int32_t* topk_idx,
                                          int topk, int B, int H, int G, int D, int page_size, float scale, void* out,
                                          float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = 0;
    if (B < 0 || max_pages_per_seq < 1) return fail(DSAIDX_ERR_SHAPE, "B=%d max_pages_per_seq=%d", B, max_pages_per_seq);
    if (q_dtype != DSAIDX_F32 && q_dtype != DSAIDX_BF16 && q_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "q_dtype=%d", q_dtype);
    if (q_dtype != DSAIDX_BF16) return fail(DSAIDX_ERR_UNSUPPORTED, "queries must be bf16");
    dsaidx_status st = kv_heads_check(H, G, scale);
    if (st != DSAIDX_OK) return st;
    st = kv_caches_check(k_cache, k_scale, v_cache, v_scale, cache_dtype, num_pages, G, D, page_size,
                         max_pages_per_seq, B == 0);
    if (st != DSAIDX_OK) return st;
    if (max_context_len < 0 || (int64_t)max_context_len > (int64_t)max_pages_per_seq * page_size)
        return fail(DSAIDX_ERR_SHAPE, "max_context_len=%d > max_pages_per_seq*page_size=%lld", max_context_len,
                    (long long)max_pages_per_seq * page_size);
    // (a list for no sequence has no address)
    if (topk < 0 || (topk_idx ? topk == 0 : topk > 0 && B > 0))
        return fail(DSAIDX_ERR_SHAPE, "topk=%d: at least 1 with topk_idx, 0 without", topk);
    if (topk > kMaxL) return fail(DSAIDX_ERR_UNSUPPORTED, "topk=%d > %d", topk, kMaxL);
    if ((int64_t)B * H > kMaxKvRows) return fail(DSAIDX_ERR_UNSUPPORTED, "B * H = %lld > 2^23", (long long)B * H);
    if (B == 0) return DSAIDX_OK;
    if (!q) return fail(DSAIDX_ERR_NULL, "q is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!context_lens) return fail(DSAIDX_ERR_NULL, "context_lens is NULL");
    if (!out) return fail(DSAIDX_ERR_NULL, "out is NULL");
    if (!aligned16(q) || !aligned16(out)) return fail(DSAIDX_ERR_UNSUPPORTED, "q and out must be 16-byte aligned");
    const size_t need = indexer_kv_attention_decode_workspace_bytes(B, H, G, D, max_context_len, topk, cache_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSAIDX_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need > 0 && !aligned16(workspace)) return fail(DSAIDX_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    dsaidx::KvDecodeArgs a{};
    a.q = reinterpret_cast<const uint16_t*>(q);
    a.cache[0] = k_cache;
    a.cache[1] = v_cache;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.block_table = block_table;
    a.lens = context_lens;
    a.idx = topk_idx;
    a.out = reinterpret_cast<uint16_t*>(out);
    a.lse = lse;
    a.workspace = workspace;
    a.scale_log2 = scale * kLog2E;
    a.B = B;
    a.H = H;
    a.G = G;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.max_ctx = max_context_len;
    a.K = topk;
    const hipError_t e = dsaidx::launch_kv_decode(a, D, cache_dtype == DSAIDX_FP8_E4M3, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_kv_attention_decode");
    return DSAIDX_OK;
}

dsaidx_status dsaidx_probe_mfma(int kind, int blocks, int iters, float* out, void* stream) {
    g_err[0] = 0;
    if (!out) return fail(DSAIDX_ERR_NULL, "out is NULL");
    if (kind < 0 || kind > 2) return fail(DSAIDX_ERR_UNSUPPORTED, "kind=%d (0, 1 or 2)", kind);
    if (blocks < 1 || blocks > 65536 || iters < 1 || iters > (1 << 20))
        return fail(DSAIDX_ERR_SHAPE, "blocks=%d iters=%d", blocks, iters);
    const hipError_t e = dsaidx::launch_probe_mfma(kind, blocks, iters, out, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "dsaidx_probe_mfma");
    return DSAIDX_OK;
}

dsaidx_status dsaidx_probe_page_read(const uint8_t* k_cache, const float* k_scale, const int32_t* page_ids, int n,
                                     int blocks, float* out, void* stream) {
    g_err[0] = 0;
    if (!k_cache || !k_scale || !page_ids || !out) return fail(DSAIDX_ERR_NULL, "a required pointer is NULL");
    if (n < 1 || blocks < 1 || blocks > 65536) return fail(DSAIDX_ERR_SHAPE, "n=%d blocks=%d", n, blocks);
    if (!aligned16(k_cache)) return fail(DSAIDX_ERR_UNSUPPORTED, "k_cache must be 16-byte aligned");
    const hipError_t e =
        dsaidx::launch_probe_page_read(k_cache, k_scale, page_ids, n, blocks, out, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "dsaidx_probe_page_read");
    return DSAIDX_OK;
}

size_t topk_select_workspace_bytes(int rows, int cols, int topk) {
    (void)rows; (void)cols; (void)topk;
    return 0;
}

dsaidx_status topk_select(const float* scores, int rows, int cols, int64_t row_stride,
                          const int32_t* row_len, int topk, int32_t* idx_out, float* val_out,
                          void* workspace, size_t workspace_bytes, void* stream) {
    (void)workspace; (void)workspace_bytes;
    g_err[0] = 0;
    if (!scores) return fail(DSAIDX_ERR_NULL, "scores is NULL");
    if (!idx_out) return fail(DSAIDX_ERR_NULL, "idx_out is NULL");
    if (rows < 1 || cols < 1 || topk < 1) return fail(DSAIDX_ERR_SHAPE, "rows=%d cols=%d topk=%d must be >= 1", rows, cols, topk);
    if (row_stride < cols) return fail(DSAIDX_ERR_SHAPE, "row_stride=%lld < cols=%d", (long long)row_stride, cols);
    if (topk > kMaxTopk) return fail(DSAIDX_ERR_UNSUPPORTED, "topk=%d > %d", topk, kMaxTopk);
    if (cols > kMaxSelectCols) return fail(DSAIDX_ERR_UNSUPPORTED, "cols=%d > %d", cols, kMaxSelectCols);
    dsaidx::SelectArgs a{};
    a.scores = scores;
    a.row_stride = row_stride;
    a.cols = cols;
    a.row_len = row_len;
    a.causal_L = 0;
    a.hist = nullptr;
    a.topk = topk;
    a.idx_out = idx_out;
    a.val_out = val_out;
    hipError_t e = dsaidx::launch_topk_select(a, rows, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "topk_select");
    return DSAIDX_OK;
}

size_t indexer_prefill_workspace_bytes(int B, int L, int H, int D, int topk, int qk_dtype, int want_scores) {
    (void)topk;
    if (B < 1 || L < 1) return 0;
    if (prefill_is_fused(qk_dtype, H, D)) return dsaidx::prefill_fused_workspace_bytes(B, L, qk_dtype);
    if (want_scores) return 0;
    return (size_t)B * (size_t)L * (size_t)L * sizeof(float);
}

}  // extern "C"

// Scratch of indexer_prefill_noalloc, the entry point that allocates nothing:
// one copy of this array per device, held until the process ends.  Host code
// never uses the array's name as a device address (in host code it is only
// a stand-in); the device address comes from hipGetSymbolAddress, taken once
// per device with that device current.
static constexpr size_t kNoAllocScratchBytes = (size_t)32 << 20;
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

namespace {

dsaidx::PerDevice<void*> g_scratch_ptr;

// Workspace of one prefill call: the caller's (checked against `need`), or,
// for the entry point that allocates nothing, this device's scratch array.
dsaidx_status prefill_workspace(bool noalloc, void* workspace, size_t workspace_bytes, size_t need, void** out) {
    if (noalloc) {
        if (need > kNoAllocScratchBytes)
            return fail(DSAIDX_ERR_UNSUPPORTED,
                        "this call needs %zu bytes of scratch; indexer_prefill_noalloc holds %zu (call "
                        "indexer_prefill with a workspace instead)", need, kNoAllocScratchBytes);
        const hipError_t e =
            g_scratch_ptr.get([](int, void** p) { return hipGetSymbolAddress(p, HIP_SYMBOL(scratch)); }, out);
        if (e != hipSuccess) return hip_fail(e, "indexer_prefill_noalloc (scratch address)");
        return DSAIDX_OK;
    }
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSAIDX_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need > 0 && !aligned16(workspace)) return fail(DSAIDX_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    *out = workspace;
    return DSAIDX_OK;
}

dsaidx_status prefill_run(const void* q, const float* q_scale, const void* k, const float* k_scale,
                          int qk_dtype, const float* w, int B, int L, int H, int D, int topk,
                          int32_t* topk_idx, float* topk_score, float* scores,
                          void* workspace, size_t workspace_bytes, void* stream, bool noalloc) {
    if (!q) return fail(DSAIDX_ERR_NULL, "q is NULL");
    if (!k) return fail(DSAIDX_ERR_NULL, "k is NULL");
    if (!w) return fail(DSAIDX_ERR_NULL, "w is NULL");
    if (!topk_idx) return fail(DSAIDX_ERR_NULL, "topk_idx is NULL");
    if (qk_dtype != DSAIDX_F32 && qk_dtype != DSAIDX_BF16 && qk_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "qk_dtype=%d", qk_dtype);
    if (qk_dtype == DSAIDX_FP8_E4M3) {
        if (!q_scale) return fail(DSAIDX_ERR_NULL, "q_scale is NULL for fp8 inputs");
        if (!k_scale) return fail(DSAIDX_ERR_NULL, "k_scale is NULL for fp8 inputs");
    } else if (q_scale || k_scale) {
        return fail(DSAIDX_ERR_SHAPE, "q_scale/k_scale must be NULL unless qk_dtype is FP8");
    }
    if (B < 1 || L < 1 || H < 1 || D < 1 || topk < 1)
        return fail(DSAIDX_ERR_SHAPE, "B=%d L=%d H=%d D=%d topk=%d must be >= 1", B, L, H, D, topk);
    if (L > kMaxL) return fail(DSAIDX_ERR_UNSUPPORTED, "L=%d > %d", L, kMaxL);
    if (H % 4 != 0 || H > 64) return fail(DSAIDX_ERR_UNSUPPORTED, "H=%d (multiple of 4 in [4, 64])", H);
    if (D != 32 && D != 64 && D != 128) return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d (32, 64 or 128)", D);
    if (topk > kMaxTopk) return fail(DSAIDX_ERR_UNSUPPORTED, "topk=%d > %d", topk, kMaxTopk);
    if (!aligned16(q) || !aligned16(k)) return fail(DSAIDX_ERR_UNSUPPORTED, "q and k must be 16-byte aligned");
    if ((size_t)B * (size_t)L > (size_t)0x7FFFFFFF) return fail(DSAIDX_ERR_UNSUPPORTED, "B*L too large");

    dsaidx::PrefillArgs a{};
    a.q = q;
    a.q_scale = q_scale;
    a.k = k;
    a.k_scale = k_scale;
    a.w = w;
    a.B = B;
    a.L = L;
    a.H = H;
    a.D = D;
    a.topk = topk;
    a.inv_sqrt_d = 1.0f / sqrtf((float)D);
    a.idx_out = topk_idx;
    a.val_out = topk_score;
    a.scores = scores;
    hipStream_t st = (hipStream_t)stream;

    const size_t need = indexer_prefill_workspace_bytes(B, L, H, D, topk, qk_dtype, scores ? 1 : 0);
    void* ws = nullptr;
    const dsaidx_status wst = prefill_workspace(noalloc, workspace, workspace_bytes, need, &ws);
    if (wst != DSAIDX_OK) return wst;
    if (prefill_is_fused(qk_dtype, H, D)) {
        a.workspace = ws;
        hipError_t e = dsaidx::launch_prefill_fused(a, qk_dtype, st);
        if (e != hipSuccess) return hip_fail(e, "indexer_prefill (fused)");
        return DSAIDX_OK;
    }
    float* mat = scores ? scores : reinterpret_cast<float*>(ws);
    hipError_t e = dsaidx::launch_prefill_scores_generic(a, qk_dtype, mat, st);
    if (e != hipSuccess) return hip_fail(e, "indexer_prefill (scores)");
    dsaidx::SelectArgs s{};
    s.scores = mat;
    s.row_stride = L;
    s.cols = L;
    s.row_len = nullptr;
    s.causal_L = L;
    s.hist = nullptr;
    s.topk = topk;
    s.idx_out = topk_idx;
    s.val_out = topk_score;
    e = dsaidx::launch_topk_select(s, B * L, st);
    if (e != hipSuccess) return hip_fail(e, "indexer_prefill (select)");
    return DSAIDX_OK;
}

}  // namespace

extern "C" {

dsaidx_status indexer_prefill(const void* q, const float* q_scale, const void* k, const float* k_scale,
                              int qk_dtype, const float* w, int B, int L, int H, int D, int topk,
                              int32_t* topk_idx, float* topk_score, float* scores,
                              void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = 0;
    return prefill_run(q, q_scale, k, k_scale, qk_dtype, w, B, L, H, D, topk, topk_idx, topk_score, scores,
                       workspace, workspace_bytes, stream, false);
}

size_t indexer_prefill_noalloc_scratch_bytes(void) { return kNoAllocScratchBytes; }

dsaidx_status indexer_prefill_noalloc(const void* q, const float* q_scale, const void* k, const float* k_scale,
                                      int qk_dtype, const float* w, int B, int L, int H, int D, int topk,
                                      int32_t* topk_idx, float* topk_score, float* scores, void* stream) {
    g_err[0] = 0;
    return prefill_run(q, q_scale, k, k_scale, qk_dtype, w, B, L, H, D, topk, topk_idx, topk_score, scores,
                       nullptr, 0, stream, true);
}

size_t indexer_prefill_chunk_paged_workspace_bytes(int B, int T, int max_kv_len, int q_dtype) {
    if (B < 1 || T < 1 || max_kv_len < 1) return 0;
    if (q_dtype == DSAIDX_BF16) return dsaidx::prefill_bf16_varlen_workspace_bytes(B, T, max_kv_len);
    return dsaidx::prefill_ws_workspace_bytes(B, max_kv_len, (T + 7) / 8 + B);
}

dsaidx_status indexer_prefill_chunk_paged(const void* q, const float* q_scale, int q_dtype, const float* w,
                                          const int32_t* cu_seqlens_q, const int32_t* q_start,
                                          const uint8_t* k_cache, const float* k_scale,
                                          const int32_t* block_table, int max_pages_per_seq, int num_pages,
                                          int B, int T, int max_kv_len, int H, int D, int page_size, int topk,
                                          int32_t* topk_idx, float* topk_score,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = 0;
    if (!q) return fail(DSAIDX_ERR_NULL, "q is NULL");
    if (!w) return fail(DSAIDX_ERR_NULL, "w is NULL");
    if (!cu_seqlens_q) return fail(DSAIDX_ERR_NULL, "cu_seqlens_q is NULL");
    if (!q_start) return fail(DSAIDX_ERR_NULL, "q_start is NULL");
    if (!k_cache) return fail(DSAIDX_ERR_NULL, "k_cache is NULL");
    if (!k_scale) return fail(DSAIDX_ERR_NULL, "k_scale is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!topk_idx) return fail(DSAIDX_ERR_NULL, "topk_idx is NULL");
    if (q_dtype != DSAIDX_F32 && q_dtype != DSAIDX_BF16 && q_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "q_dtype=%d", q_dtype);
    if (B < 1 || T < 1 || max_kv_len < 1 || H < 1 || D < 1 || page_size < 1 || topk < 1 || max_pages_per_seq < 1 ||
        num_pages < 1)
        return fail(DSAIDX_ERR_SHAPE, "B=%d T=%d max_kv_len=%d H=%d D=%d page_size=%d topk=%d max_pages_per_seq=%d "
                    "num_pages=%d", B, T, max_kv_len, H, D, page_size, topk, max_pages_per_seq, num_pages);
    if ((int64_t)max_kv_len > (int64_t)max_pages_per_seq * page_size)
        return fail(DSAIDX_ERR_SHAPE, "max_kv_len = %d > max_pages_per_seq * page_size = %lld", max_kv_len,
                    (long long)max_pages_per_seq * page_size);
    if (q_dtype == DSAIDX_F32) return fail(DSAIDX_ERR_UNSUPPORTED, "chunk queries must be fp8 or bf16");
    if (q_dtype == DSAIDX_FP8_E4M3 && !q_scale) return fail(DSAIDX_ERR_NULL, "q_scale is NULL (fp8 queries)");
    if (q_dtype == DSAIDX_BF16 && q_scale)
        return fail(DSAIDX_ERR_UNSUPPORTED, "q_scale must be NULL for bf16 queries");
    if (H % 16 != 0 || H > 64) return fail(DSAIDX_ERR_UNSUPPORTED, "H=%d (16, 32, 48 or 64)", H);
    if (D != 128) return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d (128)", D);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if (topk > kMaxTopk) return fail(DSAIDX_ERR_UNSUPPORTED, "topk=%d > %d", topk, kMaxTopk);
    if (max_kv_len > kMaxL) return fail(DSAIDX_ERR_UNSUPPORTED, "max_kv_len=%d > %d", max_kv_len, kMaxL);
    if ((int64_t)T + 8 * (int64_t)B > (int64_t)0x7FFFFFFF) return fail(DSAIDX_ERR_UNSUPPORTED, "T too large");
    if (!aligned16(q) || !aligned16(k_cache)) return fail(DSAIDX_ERR_UNSUPPORTED, "q and k_cache must be 16-byte aligned");
    if (!aligned16(workspace)) return fail(DSAIDX_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    const size_t need = indexer_prefill_chunk_paged_workspace_bytes(B, T, max_kv_len, q_dtype);
    if (!workspace || workspace_bytes < need)
        return fail(DSAIDX_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    dsaidx::PrefillArgs a{};
    a.q = q;
    a.q_scale = q_scale;
    a.k = k_cache;
    a.k_scale = k_scale;
    a.w = w;
    a.B = B;
    a.L = 0;
    a.H = H;
    a.D = D;
    a.topk = topk;
    a.inv_sqrt_d = 1.0f / sqrtf((float)D);
    a.idx_out = topk_idx;
    a.val_out = topk_score;
    a.scores = nullptr;
    a.workspace = workspace;
    a.block_table = block_table;
    a.max_pages = max_pages_per_seq;
    a.cu_q = cu_seqlens_q;
    a.q_start = q_start;
    a.T = T;
    a.max_kv = max_kv_len;
    const hipError_t e = q_dtype == DSAIDX_BF16 ? dsaidx::launch_prefill_bf16_varlen(a, (hipStream_t)stream)
                                                : dsaidx::launch_prefill_ws_varlen(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "indexer_prefill_chunk_paged");
    return DSAIDX_OK;
}

size_t indexer_decode_paged_workspace_bytes(int B, int max_context_len, int H, int D, int topk) {
    (void)H; (void)D; (void)topk;
    if (B < 1 || max_context_len < 0) return 0;
    // candidate scores and positions: [B][stride] each; per-query counters
    // [B][kCtrlStride]; page prefix over queries [B+1].
    return (size_t)B * decode_score_stride(max_context_len) * 8u +
           (size_t)B * dsaidx::kCtrlStride * sizeof(uint32_t) +
           (size_t)(B + 1) * sizeof(int32_t);
}

dsaidx_status indexer_decode_paged(const void* q, int q_dtype, const float* w,
                                   const uint8_t* k_cache, const float* k_scale,
                                   const int32_t* block_table, int max_pages_per_seq,
                                   const int32_t* context_lens, int max_context_len,
                                   int B, int H, int D, int page_size, int num_pages, int topk,
                                   int32_t* topk_idx, float* topk_score,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = 0;
    if (!q) return fail(DSAIDX_ERR_NULL, "q is NULL");
    if (!w) return fail(DSAIDX_ERR_NULL, "w is NULL");
    if (!k_cache) return fail(DSAIDX_ERR_NULL, "k_cache is NULL");
    if (!k_scale) return fail(DSAIDX_ERR_NULL, "k_scale is NULL");
    if (!block_table) return fail(DSAIDX_ERR_NULL, "block_table is NULL");
    if (!context_lens) return fail(DSAIDX_ERR_NULL, "context_lens is NULL");
    if (!topk_idx) return fail(DSAIDX_ERR_NULL, "topk_idx is NULL");
    if (q_dtype != DSAIDX_F32 && q_dtype != DSAIDX_BF16 && q_dtype != DSAIDX_FP8_E4M3)
        return fail(DSAIDX_ERR_DTYPE, "q_dtype=%d", q_dtype);
    if (B < 1 || H < 1 || D < 1 || page_size < 1 || num_pages < 1 || max_pages_per_seq < 1 || topk < 1 ||
        max_context_len < 0)
        return fail(DSAIDX_ERR_SHAPE, "B=%d H=%d D=%d page_size=%d num_pages=%d max_pages_per_seq=%d topk=%d "
                    "max_context_len=%d", B, H, D, page_size, num_pages, max_pages_per_seq, topk, max_context_len);
    if ((int64_t)max_context_len > (int64_t)max_pages_per_seq * page_size)
        return fail(DSAIDX_ERR_SHAPE, "max_context_len=%d > max_pages_per_seq*page_size=%lld", max_context_len,
                    (long long)max_pages_per_seq * page_size);
    if (q_dtype != DSAIDX_BF16) return fail(DSAIDX_ERR_UNSUPPORTED, "decode queries must be bf16");
    if (H % 16 != 0 || H > 64) return fail(DSAIDX_ERR_UNSUPPORTED, "H=%d (16, 32, 48 or 64)", H);
    if (D != 128) return fail(DSAIDX_ERR_UNSUPPORTED, "D=%d (128)", D);
    if (page_size != 64) return fail(DSAIDX_ERR_UNSUPPORTED, "page_size=%d (64)", page_size);
    if (topk > kMaxTopk) return fail(DSAIDX_ERR_UNSUPPORTED, "topk=%d > %d", topk, kMaxTopk);
    if (max_context_len > kMaxSelectCols) return fail(DSAIDX_ERR_UNSUPPORTED, "max_context_len too large");
    if (!aligned16(q) || !aligned16(k_cache)) return fail(DSAIDX_ERR_UNSUPPORTED, "q and k_cache must be 16-byte aligned");
    if (!aligned16(workspace)) return fail(DSAIDX_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    const size_t need = indexer_decode_paged_workspace_bytes(B, max_context_len, H, D, topk);
    if (!workspace || workspace_bytes < need)
        return fail(DSAIDX_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);

    hipStream_t st = (hipStream_t)stream;
    const size_t stride = decode_score_stride(max_context_len);
    char* wp = reinterpret_cast<char*>(workspace);
    float* cand_score = reinterpret_cast<float*>(wp);
    int32_t* cand_pos = reinterpret_cast<int32_t*>(wp + (size_t)B * stride * 4);
    uint32_t* ctrl = reinterpret_cast<uint32_t*>(wp + (size_t)B * stride * 8);  // [B][kCtrlStride]
    int32_t* prefix = reinterpret_cast<int32_t*>(ctrl + (size_t)B * dsaidx::kCtrlStride);
    hipError_t e;
    // Exact selection over each query's candidates (every score that can
    // be selected is among them), run by the scan's final kernel.
    dsaidx::SelectArgs s{};
    s.scores = cand_score;
    s.row_stride = (int64_t)stride;
    s.cols = (int)(stride > 0 ? stride : 1);
    s.row_len = reinterpret_cast<const int32_t*>(ctrl + 1);
    s.counter_stride = dsaidx::kCtrlStride;
    s.level0_bin = nullptr;
    s.causal_L = 0;
    s.pos = cand_pos;
    s.hist = nullptr;
    s.pre_count = nullptr;
    s.total = context_lens;
    s.total_max = max_context_len;
    s.topk = topk;
    s.idx_out = topk_idx;
    s.val_out = topk_score;
    if (max_context_len > 0) {
        dsaidx::DecodeArgs d{};
        d.q = reinterpret_cast<const uint16_t*>(q);
        d.w = w;
        d.k_cache = k_cache;
        d.k_scale = k_scale;
        d.block_table = block_table;
        d.max_pages = max_pages_per_seq;
        d.context_lens = context_lens;
        d.max_ctx = max_context_len;
        d.B = B;
        d.topk = topk;
        d.inv_sqrt_d = 1.0f / sqrtf((float)D);
        d.ctrl = ctrl;
        d.prefix = prefix;
        d.cand_score = cand_score;
        d.cand_pos = cand_pos;
        d.cand_stride = (int64_t)stride;
        e = dsaidx::launch_decode_scan(d, s, H, st);
        if (e != hipSuccess) return hip_fail(e, "indexer_decode_paged (scan)");
    } else {
        e = dsaidx::launch_zero_u32(ctrl, (size_t)B * dsaidx::kCtrlStride, st);
        if (e != hipSuccess) return hip_fail(e, "indexer_decode_paged (clear)");
        e = dsaidx::launch_topk_select(s, B, st);
        if (e != hipSuccess) return hip_fail(e, "indexer_decode_paged (select)");
    }
    return DSAIDX_OK;
}

}  // extern "C"
