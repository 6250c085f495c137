// Attention over the paged latent cache: every head of a query reads the same
// E-wide rows, whose first V columns are the values.
//
//   S[h, j] = scale * q[h] . c[j],  P = softmax_j S,  out[h] = sum_j P[h, j] c[j][:V]
//   lse[h] = log sum_j exp S[h, j]       (no key: out = 0, lse = -inf)
//
// The keys of query t are the rows at its selected positions (topk), or the
// rows of a prefix that the whole batch shares followed by the sequence's own
// (shared).
//
// Layout: one wave per query and head.  Lane l holds columns 8l .. 8l+7 of
// the query and of the sum, and column V + l of the query when E > V; the dot
// product is a wave sum, the softmax is kept as a running maximum and sum.
#include "common.h"
#include "kernels.h"

namespace dsaidx {
namespace {

constexpr int kPage = 64;
constexpr int kThreads = 256;
constexpr int kV = 512;

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

template <bool FP8>
__device__ __forceinline__ void load_row(const LatentArgs& a, int64_t row, int lane, float (&x)[8], float& r) {
    r = 0.f;
    if constexpr (FP8) {
        const uint8_t* p = reinterpret_cast<const uint8_t*>(a.cache) + row * a.E;
        const float s = a.cache_scale[row];
        const uint2 u = *reinterpret_cast<const uint2*>(p + 8 * lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)(j ? u.y : u.x), false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)(j ? u.y : u.x), true);
            x[4 * j] = lo[0] * s;
            x[4 * j + 1] = lo[1] * s;
            x[4 * j + 2] = hi[0] * s;
            x[4 * j + 3] = hi[1] * s;
        }
        if (a.E > kV) r = __builtin_amdgcn_cvt_f32_fp8((int)p[kV + lane], 0) * s;
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(a.cache) + row * a.E;
        const v4i u = *reinterpret_cast<const v4i*>(p + 8 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo((uint32_t)u[j]);
            x[2 * j + 1] = bf16_hi((uint32_t)u[j]);
        }
        if (a.E > kV) r = bf16_lo(p[kV + lane]);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads)
latent_attention_kernel(LatentArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 6;
    if (w >= (int64_t)a.T * a.H) return;
    const int t = (int)(w / a.H);
    const uint16_t* qp = a.q + w * a.E;
    float q[8], qr = 0.f;
    {
        const v4i u = *reinterpret_cast<const v4i*>(qp + 8 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q[2 * j] = bf16_lo((uint32_t)u[j]);
            q[2 * j + 1] = bf16_hi((uint32_t)u[j]);
        }
        if (a.E > kV) qr = bf16_lo(qp[kV + lane]);
    }
    float m = -__builtin_inff(), l = 0.f, o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.f;

    auto key = [&](int64_t row) {
        float x[8], r;
        load_row<FP8>(a, row, lane, x, r);
        float d = qr * r;
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fmaf(q[j], x[j], d);
#pragma unroll
        for (int i = 32; i >= 1; i >>= 1) d += __shfl_xor(d, i, kWave);
        d *= a.scale_log2;
        if (d == -__builtin_inff()) return;
        const float m2 = fmaxf(m, d);
        const float f = exp2f(m - m2), p = exp2f(d - m2);
        m = m2;
        l = l * f + p;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = o[j] * f + p * x[j];
    };
    auto paged = [&](const int32_t* table, int n) {
        for (int j = 0; j < n; ++j) {
            const int page = table[j / kPage];
            if (page >= 0 && page < a.num_pages) key((int64_t)page * kPage + j % kPage);
        }
    };
    if (a.idx) {
        const int b = a.seq_ids ? a.seq_ids[t] : t;
        if (b >= 0 && b < a.B) {
            const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
            for (int j = 0; j < a.K; ++j) {
                const int s = a.idx[(int64_t)t * a.K + j];
                if (s < 0 || s / kPage >= a.max_pages) continue;
                const int page = table[s / kPage];
                if (page >= 0 && page < a.num_pages) key((int64_t)page * kPage + s % kPage);
            }
        }
    } else {
        paged(a.prefix_table, a.prefix_len);
        paged(a.block_table + (int64_t)t * a.max_pages, min(max(a.context_lens[t], 0), a.max_ctx));
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    v8bf y;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (__bf16)(o[j] * inv);
    *reinterpret_cast<v8bf*>(a.out + w * kV + 8 * lane) = y;
    if (a.lse && lane == 0) a.lse[w] = l > 0.f ? (m + log2f(l)) * 0.693147180559945f : -__builtin_inff();
}

}  // namespace

size_t latent_topk_workspace_bytes(int T, int H, int E, int K) { return 0; }
size_t latent_shared_workspace_bytes(int B, int H, int E, int prefix_len, int max_ctx) { return 0; }

hipError_t launch_latent_attention(const LatentArgs& a, bool fp8, hipStream_t stream) {
    const int64_t blocks = ((int64_t)a.T * a.H * 64 + kThreads - 1) / kThreads;
    if (fp8) hipLaunchKernelGGL(latent_attention_kernel<true>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(latent_attention_kernel<false>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dsaidx
