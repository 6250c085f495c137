// The write of the paged key and value caches: T new tokens' G key rows, rotated
// by their positions, and G value rows, appended to both caches in one launch.
//
// "Study MLA Indexer", the data-flow diagram and the notes on its two caches: a
// cache is written before the attention that reads it.  With angle entries
// cos, sin of the token's position, the pair (a, b) of a key's first R columns
// becomes
//     a' = a cos - b sin,   b' = b cos + a sin
// where pair i is columns (2i, 2i + 1) or (i, i + R/2).  bf16 rows are the fp32
// results rounded once; fp8 rows (fp8_row.h) take their scale from the rotated
// row.  A NaN stays one in a row of either type.
//
// Layout: D/8 lanes hold a token's key and value of one head, 8 columns of each; a
// wave holds 4 or 8 heads, those of a token one after another.  A lane whose
// partner columns lie in another piece loads that piece too (from L1).  The rows'
// loads stand before the checks, so that they do not wait for the chain position
// -> page -> place; a row without a place takes position 0's angles and stores
// nothing.
//
// Bound by HBM with many tokens: 32768 tokens of 8 heads of 128 columns, bf16 (280
// MB), 53 us, 5.3 TB/s, a 1 GiB copy's rate; 76 with keys and values by different
// threads, 54 and 55 with two and four heads to a thread.  fp8 rows (215 MB): 47 us.
// One token: 2.5 us, the launch.
#include "common.h"
#include "fp8_row.h"
#include "kv.h"

namespace dsaidx {
namespace {

constexpr int kPage = 64;
constexpr int kThreads = 256;

// Eight consecutive elements as they are stored.
template <bool F32>
struct Piece {
    v4i u[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const v4i* p = reinterpret_cast<const v4i*>(reinterpret_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < (F32 ? 2 : 1); ++j) u[j] = p[j];
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (F32) return __int_as_float(u[j / 4][j % 4]);
        return __uint_as_float(j % 2 ? (uint32_t)u[0][j / 2] & 0xFFFF0000u : (uint32_t)u[0][j / 2] << 16);
    }
};

// Maximum over the N lanes of a row of values that are not negative (their order is that of their bits).
template <int N>
__device__ __forceinline__ float row_max(float x) {
    uint32_t v = __float_as_uint(x);
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // lane ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // mirrored in 8 lanes
    if constexpr (N == 16)
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // mirrored in 16
    return __uint_as_float(v);
}

template <int D, bool F32, bool FP8>
__global__ void __launch_bounds__(kThreads)
kv_append_rope_kernel(KvAppendArgs a) {
    constexpr int N = D / 8;   // lanes of a row
    const uint32_t r = (blockIdx.x * kThreads + threadIdx.x) / N;
    const int col = 8 * (int)(threadIdx.x % N);
    if (r >= (uint32_t)a.T * (uint32_t)a.G) return;
    const int t = (int)(r / (uint32_t)a.G), g = (int)(r % (uint32_t)a.G);
    const bool turned = col < a.R;
    const int across = a.pairs ? 0 : col < a.R / 2 ? a.R / 2 : -a.R / 2;   // where a column's partner is

    const int b = a.seq_ids[t], p = a.positions[t];
    Piece<F32> x[2], o;   // key and value; the key's partners
    const int64_t at = (int64_t)t * a.in[0].row + (int64_t)g * a.in[0].head + col;
    x[0].load(a.in[0].p, at);
    if (turned && across) o.load(a.in[0].p, at + across);
    x[1].load(a.in[1].p, (int64_t)t * a.in[1].row + (int64_t)g * a.in[1].head + col);
    // where the token goes
    const bool known = b >= 0 && b < a.B && p >= 0 && p < a.rope_len && p / kPage < a.max_pages;
    const int page = a.block_table[known ? (int64_t)b * a.max_pages + p / kPage : 0];
    float y[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[0][j] = x[0].get(j);
        y[1][j] = x[1].get(j);
    }
    if (turned) {
        const float* cs = a.cos_sin + (known ? (int64_t)p * a.R : 0);
        if (a.pairs) {
            const v4f co = *reinterpret_cast<const v4f*>(cs + col / 2);
            const v4f si = *reinterpret_cast<const v4f*>(cs + a.R / 2 + col / 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = y[0][2 * j], w = y[0][2 * j + 1];
                y[0][2 * j] = u * co[j] - w * si[j];
                y[0][2 * j + 1] = w * co[j] + u * si[j];
            }
        } else {
            const float* c0 = cs + (across > 0 ? col : col - a.R / 2);
            Piece<true> co, si;
            co.load(c0, 0);
            si.load(c0, a.R / 2);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[0][j] = across < 0 ? y[0][j] * co.get(j) + o.get(j) * si.get(j)
                                     : y[0][j] * co.get(j) - o.get(j) * si.get(j);
        }
    }
    const bool ok = known && page >= 0 && page < a.num_pages;
    const int64_t row = ((int64_t)page * a.G + g) * kPage + p % kPage;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if constexpr (FP8) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[which][j]));
            const float s = row_scale(row_max<N>(m));
            if (ok) {
                *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.cache[which]) + row * D + col) =
                    quant8<true>(y[which], s);
                if (col == 0) a.scale[which][row] = s;
            }
        } else if (ok) {
            v8bf z;
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = (__bf16)y[which][j];
            *reinterpret_cast<v8bf*>(reinterpret_cast<uint16_t*>(a.cache[which]) + row * D + col) = z;
        }
    }
}

template <int D, bool F32>
void launch(const KvAppendArgs& a, bool fp8, hipStream_t stream) {
    const int64_t threads = (int64_t)a.T * a.G * (D / 8);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
    if (fp8) hipLaunchKernelGGL((kv_append_rope_kernel<D, F32, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((kv_append_rope_kernel<D, F32, false>), grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_kv_append_rope(const KvAppendArgs& a, int D, bool f32, bool fp8, hipStream_t stream) {
    if (a.T <= 0) return hipSuccess;
    if (D == 64) f32 ? launch<64, true>(a, fp8, stream) : launch<64, false>(a, fp8, stream);
    else f32 ? launch<128, true>(a, fp8, stream) : launch<128, false>(a, fp8, stream);
    return hipGetLastError();
}

}  // namespace dsaidx
