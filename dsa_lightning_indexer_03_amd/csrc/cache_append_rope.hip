// The layer's cache write: T new tokens' latent rows and index keys, rotated
// by their positions and appended to the two paged caches in one launch.
//
// The pages' data flow rotates the key path by position before it enters the
// indexer's FP8 cache ("Study MLA Indexer", the data-flow diagram and the
// notes on its two caches: both caches are written before the scoring
// decision).  A latent row is [c | r]: its last R columns r are rotated; an
// index key's first R columns are.  With angle entries cos, sin of the
// token's position, the pair (a, b) becomes
//     a' = a cos - b sin,   b' = b cos + a sin
// where pair i is columns (2i, 2i + 1) or (i, i + R/2) of the rotated part.
// bf16 rows are the fp32 results rounded once; fp8 rows (fp8_row.h) take
// their scale from the rotated row.
//
// Layout: one wave per token.  The token's 8-column pieces, latent row first,
// index key behind it, go to lanes 0, 1, ... and round again, so all of a
// token's loads are in flight at once; a piece whose partner columns lie in
// another piece loads that piece too (from L1).
#include "common.h"
#include "fp8_row.h"
#include "kernels.h"

namespace dsaidx {
namespace {

constexpr int kD = 128;
constexpr int kPage = 64;
constexpr int kThreads = 256;

template <int DT>  // 0 = f32, 1 = bf16
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
    if constexpr (DT == 1) {
        const v4i u = *reinterpret_cast<const v4i*>(reinterpret_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float((uint32_t)u[j] << 16);
            x[2 * j + 1] = __uint_as_float((uint32_t)u[j] & 0xFFFF0000u);
        }
    } else {
        const float* p = reinterpret_cast<const float*>(base) + at;
        const v4f lo = *reinterpret_cast<const v4f*>(p);
        const v4f hi = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = lo[j];
            x[4 + j] = hi[j];
        }
    }
}

// Columns c .. c + 7 of a rotated part of R columns; `base + at` is its column
// c in memory, cs the position's R/2 cosines and R/2 sines.
template <int DT>
__device__ __forceinline__ void rotate8(float (&x)[8], const void* base, int64_t at, int c, int R, bool pairs,
                                        const float* cs) {
    if (pairs) {
        const v4f co = *reinterpret_cast<const v4f*>(cs + c / 2);
        const v4f si = *reinterpret_cast<const v4f*>(cs + R / 2 + c / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = x[2 * j], q = x[2 * j + 1];
            x[2 * j] = p * co[j] - q * si[j];
            x[2 * j + 1] = q * co[j] + p * si[j];
        }
    } else {
        const bool upper = c >= R / 2;
        const int i = upper ? c - R / 2 : c;
        float o[8];
        load8<DT>(base, upper ? at - R / 2 : at + R / 2, o);
        float co[8], si[8];
        load8<0>(cs, i, co);
        load8<0>(cs, R / 2 + i, si);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = upper ? x[j] * co[j] + o[j] * si[j] : x[j] * co[j] - o[j] * si[j];
    }
}

__device__ __forceinline__ float wave_fmax(float m) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    return m;
}

template <int DT, int NP, bool FP8>  // NP: rounds of 64 pieces; FP8: the latent rows' type
__global__ void __launch_bounds__(kThreads)
cache_append_rope_kernel(AppendRopeArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 6;
    if (t >= a.T) return;
    const int b = a.seq_ids[t], p = a.positions[t];
    if (b < 0 || b >= a.B || p < 0 || p >= a.rope_len || p / kPage >= a.max_pages) return;
    const int page = a.block_table[(int64_t)b * a.max_pages + p / kPage];
    if (page < 0 || page >= a.num_pages) return;
    const int64_t row = (int64_t)page * kPage + p % kPage;
    const float* cs = a.cos_sin + (int64_t)p * a.R;
    const int n_kv = a.E / 8;
    const int n = n_kv + (a.index_k ? kD / 8 : 0);
    const int first = a.E - a.R;

    float x[NP][8];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int i = lane + 64 * s;
        if (i < n_kv) load8<DT>(a.kv, t * a.kv_stride + 8 * i, x[s]);
        else if (i < n) load8<DT>(a.index_k, t * a.index_stride + 8 * (i - n_kv), x[s]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) x[s][j] = 0.f;
    }
    float m_kv = 0.f, m_ix = 0.f;
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int i = lane + 64 * s, c = 8 * (i - n_kv);
        if (i < n_kv && 8 * i >= first)
            rotate8<DT>(x[s], a.kv, t * a.kv_stride + 8 * i, 8 * i - first, a.R, a.kv_pairs, cs);
        else if (i >= n_kv && i < n && c < a.R)
            rotate8<DT>(x[s], a.index_k, t * a.index_stride + c, c, a.R, a.index_pairs, cs);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[s][j]));
        if (i < n_kv) m_kv = fmaxf(m_kv, m);
        else m_ix = fmaxf(m_ix, m);
    }
    const float s_ix = a.index_k ? row_scale(wave_fmax(m_ix)) : 1.f;
    const float s_kv = FP8 ? row_scale(wave_fmax(m_kv)) : 1.f;
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int i = lane + 64 * s;
        if (i < n_kv) {
            if constexpr (FP8) {
                *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.latent) + row * a.E + 8 * i) =
                    quant8(x[s], s_kv);
            } else {
                v8bf y;
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = (__bf16)x[s][j];
                *reinterpret_cast<v8bf*>(reinterpret_cast<uint16_t*>(a.latent) + row * a.E + 8 * i) = y;
            }
        } else if (i < n) {
            *reinterpret_cast<uint2*>(a.k_cache + row * kD + 8 * (i - n_kv)) = quant8(x[s], s_ix);
        }
    }
    if (lane == 0) {
        if (FP8) a.latent_scale[row] = s_kv;
        if (a.index_k) a.k_scale[row] = s_ix;
    }
}

template <int DT, int NP>
void launch(const AppendRopeArgs& a, bool fp8, unsigned blocks, hipStream_t stream) {
    if (fp8) hipLaunchKernelGGL((cache_append_rope_kernel<DT, NP, true>), dim3(blocks), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((cache_append_rope_kernel<DT, NP, false>), dim3(blocks), dim3(kThreads), 0, stream, a);
}

template <int DT>
void launch(const AppendRopeArgs& a, bool fp8, hipStream_t stream) {
    const unsigned blocks = (unsigned)(((int64_t)a.T * 64 + kThreads - 1) / kThreads);
    const int pieces = a.E / 8 + (a.index_k ? kD / 8 : 0);
    if (pieces <= 64) launch<DT, 1>(a, fp8, blocks, stream);
    else if (pieces <= 128) launch<DT, 2>(a, fp8, blocks, stream);
    else launch<DT, 3>(a, fp8, blocks, stream);
}

}  // namespace

hipError_t launch_cache_append_rope(const AppendRopeArgs& a, bool f32, bool fp8, hipStream_t stream) {
    if (a.T <= 0) return hipSuccess;
    if (f32) launch<0>(a, fp8, stream);
    else launch<1>(a, fp8, stream);
    return hipGetLastError();
}

}  // namespace dsaidx
