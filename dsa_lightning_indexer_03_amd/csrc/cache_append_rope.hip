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
// their scale from the rotated row.  A NaN stays one in a latent row of either
// type, so that attention over the row shows it; index keys are stored as
// kcache_append stores them, without NaN codes, which no score may meet.
//
// Layout: one wave per token.  Its 8-column pieces, latent row first, index key
// behind it, go to lanes 0, 1, ... and round again; a piece whose partner
// columns lie in another piece loads that piece too (from L1).  The rows' loads
// stand before the checks, so that they do not wait for the chain position ->
// page -> place; a token without a place takes position 0's angles, if it has
// none of its own, and stores nothing.
//
// Bound by HBM with many tokens: 32768 tokens of 576 + 128 columns, bf16 rows
// (94 MB with the angles): 27 us, 3.5 TB/s, from inputs that no cache holds (a
// 1 GiB copy: 5.2), 21 us where the inputs are still in one; two tokens a wave in
// full rounds of lanes took 24 there.  fp8 rows (75 MB): 27 and 23 us, bound by
// vector instructions, 487 a token, most of them the exact quotients: 50 more
// took 1.6 us longer.  One token: 2.5 us, the launch.
#include "common.h"
#include "fp8_row.h"
#include "latent.h"

namespace dsaidx {
namespace {

constexpr int kD = 128;
constexpr int kPage = 64;
constexpr int kThreads = 256;

// Eight consecutive elements as they are stored.
template <int DT>  // 0 = f32, 1 = bf16
struct Piece {
    v4i u[DT == 1 ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const v4i* p = reinterpret_cast<const v4i*>(reinterpret_cast<const char*>(base) + at * (DT == 1 ? 2 : 4));
#pragma unroll
        for (int j = 0; j < (DT == 1 ? 1 : 2); ++j) u[j] = p[j];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < (DT == 1 ? 1 : 2); ++j) u[j] = v4i{0, 0, 0, 0};
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (DT == 1)
            return __uint_as_float(j % 2 ? (uint32_t)u[0][j / 2] & 0xFFFF0000u : (uint32_t)u[0][j / 2] << 16);
        else
            return __int_as_float(u[j / 4][j % 4]);
    }
};

// Maximum over the wave of values that are not negative (their order is that of their bits).
__device__ __forceinline__ float wave_max(float x) {
    uint32_t v = __float_as_uint(x);
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));  // row_shr:1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));  // row_shr:2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));  // row_shr:4
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));  // row_shr:8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));  // row_bcast:15
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));  // row_bcast:31
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1));
}

template <int DT, int NP, bool FP8>  // NP: rounds of 64 pieces; FP8: the latent rows' type
__global__ void __launch_bounds__(kThreads)
cache_append_rope_kernel(AppendRopeArgs a) {
    const int lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + uniform((int)threadIdx.x >> 6);
    if (t >= a.T) return;
    const int n_kv = a.E / 8;
    const int n = n_kv + (a.index_k ? kD / 8 : 0);

    // where the token goes
    const int b = a.seq_ids[t], p = a.positions[t];
    const bool known = b >= 0 && b < a.B && p >= 0 && p < a.rope_len && p / kPage < a.max_pages;
    const int page = a.block_table[known ? (int64_t)b * a.max_pages + p / kPage : 0];
    const bool ok = known && page >= 0 && page < a.num_pages;
    const int64_t row = (int64_t)page * kPage + p % kPage;
    const float* cs = a.cos_sin + (known ? (int64_t)p * a.R : 0);

    // this lane's pieces and, for pairs a half apart, their partners
    Piece<DT> x[NP], o[NP];
    int col[NP];       // first column in the rotated part, or -1
    bool index[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int j = lane + 64 * s;
        x[s].zero();
        o[s].zero();
        col[s] = -1;
        index[s] = j >= n_kv;
        if (j < n) {
            const void* base = index[s] ? a.index_k : a.kv;
            const int c = index[s] ? 8 * (j - n_kv) : 8 * j - (a.E - a.R);
            const int64_t at = t * (index[s] ? a.index_stride : a.kv_stride) + 8 * (index[s] ? j - n_kv : j);
            x[s].load(base, at);
            if (c >= 0 && c < a.R) {
                col[s] = c;
                if (!(index[s] ? a.index_pairs : a.kv_pairs)) o[s].load(base, c < a.R / 2 ? at + a.R / 2 : at - a.R / 2);
            }
        }
    }

    float y[NP][8], m_kv = 0.f, m_ix = 0.f;
#pragma unroll
    for (int s = 0; s < NP; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[s][j] = x[s].get(j);
        if (col[s] >= 0) {
            if (index[s] ? a.index_pairs : a.kv_pairs) {
                const v4f co = *reinterpret_cast<const v4f*>(cs + col[s] / 2);
                const v4f si = *reinterpret_cast<const v4f*>(cs + a.R / 2 + col[s] / 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = y[s][2 * j], q = y[s][2 * j + 1];
                    y[s][2 * j] = p * co[j] - q * si[j];
                    y[s][2 * j + 1] = q * co[j] + p * si[j];
                }
            } else {
                const bool upper = col[s] >= a.R / 2;
                const float* c0 = cs + (upper ? col[s] - a.R / 2 : col[s]);
                Piece<0> co, si;
                co.load(c0, 0);
                si.load(c0, a.R / 2);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[s][j] = upper ? y[s][j] * co.get(j) + o[s].get(j) * si.get(j)
                                    : y[s][j] * co.get(j) - o[s].get(j) * si.get(j);
            }
        }
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[s][j]));
        m_kv = fmaxf(m_kv, index[s] ? 0.f : m);
        m_ix = fmaxf(m_ix, index[s] ? m : 0.f);
    }
    const float s_ix = a.index_k ? row_scale(wave_max(m_ix)) : 1.f;
    const float s_kv = FP8 ? row_scale(wave_max(m_kv)) : 1.f;
    if (!ok) return;
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int j = lane + 64 * s;
        if (j >= n) continue;
        if (index[s]) {
            *reinterpret_cast<uint2*>(a.k_cache + row * kD + 8 * (j - n_kv)) = quant8<false>(y[s], s_ix);
        } else if constexpr (FP8) {
            *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.latent) + row * a.E + 8 * j) =
                quant8<true>(y[s], s_kv);
        } else {
            v8bf b;
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = (__bf16)y[s][e];
            *reinterpret_cast<v8bf*>(reinterpret_cast<uint16_t*>(a.latent) + row * a.E + 8 * j) = b;
        }
    }
    if (lane == 0) {
        if (FP8) a.latent_scale[row] = s_kv;
        if (a.index_k) a.k_scale[row] = s_ix;
    }
}

template <int DT, int NP>
void launch(const AppendRopeArgs& a, bool fp8, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.T + kThreads / 64 - 1) / (kThreads / 64)));
    if (fp8) hipLaunchKernelGGL((cache_append_rope_kernel<DT, NP, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((cache_append_rope_kernel<DT, NP, false>), grid, dim3(kThreads), 0, stream, a);
}

template <int DT>
void launch(const AppendRopeArgs& a, bool fp8, hipStream_t stream) {
    const int pieces = a.E / 8 + (a.index_k ? kD / 8 : 0);
    if (pieces <= 64) launch<DT, 1>(a, fp8, stream);
    else if (pieces <= 128) launch<DT, 2>(a, fp8, stream);
    else launch<DT, 3>(a, fp8, stream);
}

}  // namespace

hipError_t launch_cache_append_rope(const AppendRopeArgs& a, bool f32, bool fp8, hipStream_t stream) {
    if (a.T <= 0) return hipSuccess;
    if (f32) launch<0>(a, fp8, stream);
    else launch<1>(a, fp8, stream);
    return hipGetLastError();
}

}  // namespace dsaidx
