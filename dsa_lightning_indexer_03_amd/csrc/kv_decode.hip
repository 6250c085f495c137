// Attention of one new token per sequence over paged key and value caches with
// G heads of their own: query head h reads key/value head h / (H / G).
//
//   S[j] = scale * q . k[j],  out = sum_j softmax_j(S) v[j],  lse = log sum_j exp S[j]
//
// over every position of the sequence, or over the positions listed for it (the
// indexer's selection: "Study MLA Indexer", the data-flow diagram's last step).
// No position: out = 0, lse = -inf.
//
// One workgroup takes up to 64 query heads of one key/value head and a run of
// positions.  Its four waves (one where contexts are short and many) walk the run
// 32 positions at a time, each on its own with two tiles in LDS: the next one's
// rows are copied while this one is computed, the page ids and entries of the next
// two are loads in flight, and no wave waits for another before the end.  Tiles
// without a row are passed over.  Products are
//   S^T (32 keys x 16 heads) = K Q^T, the queries in registers;
//   O^T (D columns x 16 heads) += V^T P^T.
// The first one leaves a lane with head lane % 16 and keys 4g .. 4g+3 (g = lane /
// 16) of each 16 keys, which is the second one's operand when its 32 keys are
// counted as 4g .. 4g+3 of two blocks: P never leaves its registers, and the
// values are read transposed in that order.  Sums are fp32, P's sum before any
// rounding.  The exponent's reference moves when a score passes it by 2^kSlack.
//
// The second product takes its operands in bf16, and P enters it in two terms, the
// leading bits and the rest, so that an output is off by 2^-15 of sum P |v| beside its
// own rounding, where one term leaves up to 2^-8.  One and two, us: 64 contexts of
// 4096 to 32768 824 and 825, one of 4096 10.5 and 10.5, of 100 4.8 and 4.9; 64 heads
// over one, 64 of 2048, 28.0 and 29.9; fp8, one of 131072 59.2 and 60.0, 37 of up to
// 6000 with 64 columns 19.8 and 21.5.
//
// fp8 rows stay codes in LDS and are widened as operands.  A key's scale
// multiplies its score, a value's its probability, in units of the wave's first
// value scale, so that rows of one scale bring no rounding of it.
//
// The runs of a sequence are joined by a second kernel from fp32 sums.
//
// Bound by HBM: 64 contexts of 4096 to 32768 positions, 8 heads of 128 columns, bf16
// (4.87 GB, read once by the counters): 825 us, 5.9 TB/s, where reading pages alone
// reaches 6.1 to 6.3; 2048 selected of 64 contexts (537 MB): 98 us, 5.5 (fp8, 277 MB:
// 69 to 76 us, 3.6 to 4.0); one context of 131072, fp8 (277 MB): 58 to 62 us with its
// join.  A wave's next tile is in flight, 64 KB a CU in all: a round takes its share of
// the bandwidth with the card full, 0.75 to 1 us of latency with little work (run_cost).
// Products and softmax take up to a tenth of the matrix cores' cycles.
#include "device_once.h"
#include "kv.h"
#include "tile_copy.h"

namespace dsaidx {
namespace {

constexpr int kPage = 64;
constexpr int kKeys = 32;      // positions of a wave's tile
constexpr int kJoinThreads = 256;
constexpr int kMaxRuns = 512;  // runs of a sequence

// The two terms of a probability in the second product: its leading bits, bf16 in the
// upper half of the first word, and what they leave.  Of a bf16 row the first is less
// than the probability, so that the second is not 0, which would make NaN of an
// infinite value (0 stays 0).  An fp8 row's codes are finite, but its scale may be
// infinite, and with it the first term; the second is then a number, 2^127 (it is below
// 2^121 of any finite one), not the NaN of inf - inf.
template <bool FP8>
__device__ __forceinline__ uint32_t leading(float p) {
    return FP8 ? __float_as_uint(p) : __builtin_elementwise_sub_sat(__float_as_uint(p), 1u);
}
template <bool FP8>
__device__ __forceinline__ float left(float p, uint32_t lead) {
    const float rest = p - __uint_as_float(lead & 0xFFFF0000u);
    return FP8 ? fminf(rest, 0x1p127f) : rest;
}

// What an entry without a row is copied from.
static __device__ __align__(16) const unsigned char kZeros[256] = {};

struct KvPlan {
    int rows;     // query heads of a workgroup: 16, 32 or 64
    int hb;       // workgroups for the heads of one key/value head
    int waves;    // of a workgroup
    int run;      // positions of a run
    int slots;    // runs of a sequence
    float* part_o;      // [slots][B * H][D]
    float2* part_ml;    // [slots][B * H] (maximum, sum)
};

// A tile's rows lie one behind another in LDS, their 16-byte pieces permuted by
// the row's number.  The 64 banks serve 16 lanes of a 16-byte read at once (lanes
// 0-3, 12-15 and 20-27 are one such group, 4-11, 16-19 and 28-31 the next), 32
// lanes of an 8-byte one; with these permutations every operand read, straight
// or transposed, uses every bank once.
template <int RB, bool FP8>
__device__ __forceinline__ int permute(int r) {
    if constexpr (RB == 256) return (r & 3) << 2 | ((r >> 2) + 1 & 3);
    if constexpr (RB == 128 && !FP8) return ((r >> 1 ^ (r >> 3 & 1) << 1) & 3) << 1 | (r >> 3 & 1);
    if constexpr (RB == 128) return (r >> 1 & 3) | ((r >> 3 ^ r >> 4) & 1) << 2;
    return (r >> 2 & 1) | ((r >> 3 ^ r >> 4) & 1) << 1;
}

template <int D, int MT, bool FP8, int W>
struct Lds {
    static constexpr int RB = D * (FP8 ? 1 : 2);
    static constexpr int kRows = kKeys * RB;              // keys or values of a tile
    static constexpr int kTile = 2 * kRows + (FP8 ? 2 * kKeys * 4 : 0);
    static constexpr int kSumB = D * 4 + 16;              // a row of sums, padded
    static constexpr int kSums = 16 * MT * kSumB;         // a wave's sums
    static constexpr int kTiles = W * 2 * kTile;
    static constexpr int kMl = W * kSums;            // (maximum, sum) of each wave's rows
    static constexpr int kJoin = kMl + W * 16 * MT * 8;
    static constexpr int kBytes = kTiles > kJoin ? kTiles : kJoin;
    static_assert(kBytes <= 160 * 1024, "LDS budget");
};

template <int D, int MT, bool TOPK, bool FP8, int W>
__global__ void __launch_bounds__(64 * W, MT == 4 ? 1 : 2)
kv_decode_kernel(KvDecodeArgs a, KvPlan p) {
    extern __shared__ __align__(16) unsigned char smem[];
    using L = Lds<D, MT, FP8, W>;
    constexpr int kRound = kKeys * W, kThreads = 64 * W;
    constexpr int RB = L::RB, KS = D / 32, CT = D / 16;
    constexpr int PL = RB / 16, RPC = 64 / PL, NC = kKeys / RPC;   // lanes of a row; rows and number of copies
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int n = lane & 15, g4 = lane >> 4;
    const int R = a.H / a.G;
    const int per = a.B * a.G * p.hb;
    const int slot = (int)(blockIdx.x / (unsigned)per), rest = (int)(blockIdx.x % (unsigned)per);
    const int hb = rest % p.hb, g = rest / p.hb % a.G, b = rest / p.hb / a.G;
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    const int32_t* idx = TOPK ? a.idx + (int64_t)b * a.K : nullptr;
    const int first = slot * p.run, most = min((TOPK ? a.K : a.max_ctx) - first, p.run) + first;
    int c = first + kKeys * wave;
    // what the first two tiles need, loaded before the context's length is known: listed
    // positions, or page ids
    auto ahead = [&](int c) -> int {
        const int e = c + (lane & (kKeys - 1));
        if (e >= most) return -1;
        return TOPK ? idx[e] : table[e / kPage];
    };
    const int a0 = ahead(c), a1 = ahead(c + kRound);
    const int ctx = min(max(a.lens[b], 0), a.max_ctx);
    const int len = TOPK ? a.K : ctx;
    const int end = min(most, len);
    if (first >= len && p.slots > 1) return;
    const int h0 = g * R + hb * p.rows;          // first head
    const int rows = min(p.rows, R - hb * p.rows);

    // ---- queries: B operand of 16 heads x 32 columns ----
    v8bf Q[MT][KS];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const uint16_t* qp = a.q + ((int64_t)b * a.H + h0 + min(16 * mt + n, rows - 1)) * D + 8 * g4;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) Q[mt][ks] = *reinterpret_cast<const v8bf*>(qp + 32 * ks);
    }

    // ---- the wave's tiles: entries, page ids, rows ----
    auto entry = [&](int c) -> int {   // position of entry lane % 32 of the tile at c, -1: none
        const int e = c + (lane & (kKeys - 1));
        if (e >= end) return -1;
        if constexpr (!TOPK) return e;
        const int s = idx[e];
        return s < ctx ? s : -1;
    };
    auto page = [&](int s) -> int { return s >= 0 ? table[s / kPage] : -1; };
    auto resolve = [&](int s, int id) -> int {   // row of the pool, -1: none
        return s >= 0 && id >= 0 && id < a.num_pages ? (id * a.G + g) * kPage + (s & (kPage - 1)) : -1;
    };
    const uint32_t lds0 = lds_address(smem) + wave * 2 * L::kTile;
    auto stage = [&](int row, int buf) {
        const uint32_t lds = lds0 + buf * L::kTile;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int r = i * RPC + lane / PL;
            const int mine = __builtin_amdgcn_ds_bpermute(4 * r, row);
            const uint32_t c = 16 * (lane % PL ^ permute<RB, FP8>(r));
            const int64_t off = (int64_t)max(mine, 0) * RB;
            copy_to_lds((mine >= 0 ? reinterpret_cast<const unsigned char*>(a.cache[0]) + off : kZeros) + c,
                        lds + i * 1024);
            copy_to_lds((mine >= 0 ? reinterpret_cast<const unsigned char*>(a.cache[1]) + off : kZeros) + c,
                        lds + L::kRows + i * 1024);
        }
        if constexpr (FP8)
            copy4_to_lds(row >= 0 ? reinterpret_cast<const unsigned char*>(a.scale[lane >> 5] + row) : kZeros,
                         lds + 2 * L::kRows);
    };

    v4f O[MT][CT];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -3.402823466e38f;   // the lowest finite: any score but -inf moves it
        l[mt] = 0.f;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) O[mt][ct] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    if (a.scale_log2 < 0.f)   // the products then take the scale's magnitude
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                v4i u = __builtin_bit_cast(v4i, Q[mt][ks]);
                u ^= (int)0x80008000;
                Q[mt][ks] = __builtin_bit_cast(v8bf, u);
            }
    // (never 0: a score of -inf, an entry without a row, has to stay one)
    const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);

    float unit = 1.f, inv_unit = 1.f;
    if (c < end) {
        const int s0 = TOPK ? (a0 < ctx ? a0 : -1) : entry(c);
        int s1 = TOPK ? (a1 < ctx ? a1 : -1) : entry(c + kRound), s2 = entry(c + 2 * kRound);
        int row = resolve(s0, TOPK ? page(s0) : a0);
        int page1 = TOPK ? page(s1) : a1;
        if constexpr (FP8) {
            const uint64_t some = wave_ballot(row >= 0);
            if (some) {
                const float u = fabsf(a.scale[1][__builtin_amdgcn_readlane(row, __builtin_ctzll(some))]);
                if (u >= 0x1p-40f && u <= 0x1p40f) unit = u;
                inv_unit = 1.f / unit;
            }
        }
        if (wave_ballot(row >= 0)) stage(row, 0);
        int buf = 0;
        for (; c < end; c += kRound, buf ^= 1) {
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the tile, and the loads behind it
            asm volatile("" ::: "memory");
            const uint32_t here = (uint32_t)wave_ballot(row >= 0);
            row = resolve(s1, page1);
            page1 = page(s2);
            s1 = s2;
            s2 = entry(c + 3 * kRound);
            if (wave_ballot(row >= 0)) stage(row, buf ^ 1);
            if (here == 0) continue;   // (no row: nothing was copied)
            const unsigned char* kt = smem + wave * 2 * L::kTile + buf * L::kTile;
            const unsigned char* vt = kt + L::kRows;
            // ---- scores ----
            v4f S[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) S[mt][0] = S[mt][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int r = 16 * kk + n;
                    v8bf k;
                    if constexpr (FP8)
                        k = __builtin_bit_cast(v8bf, widen8(*reinterpret_cast<const uint2*>(
                                kt + r * RB + 16 * ((2 * ks + (g4 >> 1)) ^ permute<RB, FP8>(r)) + 8 * (g4 & 1))));
                    else
                        k = *reinterpret_cast<const v8bf*>(kt + r * RB + 16 * ((4 * ks + g4) ^ permute<RB, FP8>(r)));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        S[mt][kk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, Q[mt][ks], S[mt][kk], 0, 0, 0);
                }
            // ---- softmax ----
            v4f vs[2];
            if constexpr (FP8) {
                const unsigned char* st = kt + 2 * L::kRows + 16 * g4;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const v4f by = *reinterpret_cast<const v4f*>(st + 64 * kk);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) S[mt][kk] *= by;
                    vs[kk] = *reinterpret_cast<const v4f*>(st + 128 + 64 * kk) * inv_unit;
                }
            }
            v8bf P[MT], rest[MT];   // probabilities; what their leading bits leave
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float top = -__builtin_inff();
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    S[mt][kk] = scaled_scores(S[mt][kk], scale);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!(here >> (16 * kk + 4 * g4 + i) & 1)) S[mt][kk][i] = -__builtin_inff();
                        top = fmaxf(top, S[mt][kk][i]);
                    }
                }
                if (wave_ballot(top > m[mt] + kSlack)) {
                    // a head's reference moves to these keys' maximum where that is so far above it (the
                    // heads beside it keep theirs: no head's result depends on another's)
                    top = fmaxf(top, __shfl_xor(top, 16, kWave));
                    top = fmaxf(top, __shfl_xor(top, 32, kWave));
                    const float to = top > m[mt] + kSlack ? top : m[mt];
                    const float f = __builtin_amdgcn_exp2f(m[mt] - to);
                    m[mt] = to;
                    l[mt] *= f;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) O[mt][ct] *= f;
                }
                v4i u, w;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    float pr[4];
                    uint32_t lead[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pr[i] = __builtin_amdgcn_exp2f(S[mt][kk][i] - m[mt]);
                        l[mt] += pr[i];
                        if constexpr (FP8) pr[i] *= vs[kk][i];
                        lead[i] = leading<FP8>(pr[i]);
                        pr[i] = left<FP8>(pr[i], lead[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        u[2 * kk + i] = (int)__builtin_amdgcn_perm(lead[2 * i + 1], lead[2 * i], 0x07060302u);   // upper halves
                        w[2 * kk + i] = (int)pack_bf16(pr[2 * i], pr[2 * i + 1]);
                    }
                }
                P[mt] = __builtin_bit_cast(v8bf, u);
                rest[mt] = __builtin_bit_cast(v8bf, w);
            }
            // ---- values: A operand of 16 columns x 32 keys ----
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                v8bf w;
                if constexpr (FP8) {
                    const int j = n >> 1, r = (j & 4) * 4 + 4 * g4 + (j & 3);
                    const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (lds_v2i*)(vt + r * RB + 16 * (ct ^ permute<RB, FP8>(r)) + 8 * (n & 1)));
                    w = __builtin_bit_cast(v8bf, widen8(uint2{(uint32_t)x[0], (uint32_t)x[1]}));
                } else {
                    const int r = 4 * g4 + (n >> 2), q = 2 * ct + (n >> 1 & 1);
                    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_v4s*)(vt + r * RB + 16 * (q ^ permute<RB, FP8>(r)) + 8 * (n & 1)));
                    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_v4s*)(vt + (r + 16) * RB + 16 * (q ^ permute<RB, FP8>(r + 16)) + 8 * (n & 1)));
                    w = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    O[mt][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, rest[mt], O[mt][ct], 0, 0, 0);
                    O[mt][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, P[mt], O[mt][ct], 0, 0, 0);
                }
            }
        }
    }

    // ---- join the waves' sums, write ----
    tile_barrier();
    float2* ml = reinterpret_cast<float2*>(smem + L::kMl);   // [wave][row]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16, kWave);
        l[mt] += __shfl_xor(l[mt], 32, kWave);
        if (g4 == 0) ml[wave * 16 * MT + 16 * mt + n] = float2{m[mt], l[mt]};
    }
    tile_barrier();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float to = m[mt];
#pragma unroll
        for (int w = 0; w < W; ++w) to = fmaxf(to, ml[w * 16 * MT + 16 * mt + n].x);
        const float f = __builtin_amdgcn_exp2f(m[mt] - to) * unit;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            *reinterpret_cast<v4f*>(smem + wave * L::kSums + (16 * mt + n) * L::kSumB + 64 * ct + 16 * g4) =
                O[mt][ct] * f;
    }
    tile_barrier();
    const int64_t out0 = (int64_t)b * a.H + h0;
    for (int i = (int)threadIdx.x; i < rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), col = 4 * (i % (D / 4));
        float to = ml[r].x, sum = 0.f;
#pragma unroll
        for (int w = 1; w < W; ++w) to = fmaxf(to, ml[w * 16 * MT + r].x);
        v4f o = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 x = ml[w * 16 * MT + r];
            sum += x.y * __builtin_amdgcn_exp2f(x.x - to);
            o += *reinterpret_cast<const v4f*>(smem + w * L::kSums + r * L::kSumB + 4 * col);
        }
        if (p.slots == 1) {
            o = sum == 0.f ? v4f{0.f, 0.f, 0.f, 0.f} : o * (1.f / sum);
            *reinterpret_cast<uint2*>(a.out + (out0 + r) * D + col) =
                uint2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
            if (a.lse && col == 0)
                a.lse[out0 + r] = sum == 0.f ? -__builtin_inff() : (to + log2f(sum)) * 0.693147180559945f;
        } else {
            const int64_t at = (int64_t)slot * ((int64_t)a.B * a.H) + out0 + r;
            *reinterpret_cast<v4f*>(p.part_o + at * D + col) = o;
            if (col == 0) p.part_ml[at] = float2{to, sum};
        }
    }
}

// One workgroup a row: its threads weigh the runs, then a lane takes 4 columns of
// every run that is its wave part's, four runs' loads in flight (one context of
// 131072, 16 heads over one: both kernels 20.5 us, with one load at a time 24.7).
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
kv_join_kernel(KvDecodeArgs a, KvPlan p) {
    constexpr int N = D / 4, kParts = kJoinThreads / N;   // lanes of a run's row, runs at once
    __shared__ float weights[kMaxRuns];
    __shared__ float red[2][(kJoinThreads / 64)];
    __shared__ v4f sums[kParts][N];
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int64_t row = blockIdx.x, rows = (int64_t)a.B * a.H;
    const int b = (int)(row / a.H);
    const int len = a.idx ? a.K : min(max(a.lens[b], 0), a.max_ctx);
    const int runs = min((len + p.run - 1) / p.run, p.slots);
    const int part = (int)threadIdx.x / N, col = 4 * ((int)threadIdx.x % N);
    const float* at = p.part_o + row * D + col;
    float2 ml[kMaxRuns / kJoinThreads];
    float to = -3.402823466e38f;
#pragma unroll
    for (int i = 0; i < kMaxRuns / kJoinThreads; ++i) {
        const int s = i * kJoinThreads + (int)threadIdx.x;
        ml[i] = s < runs ? p.part_ml[s * rows + row] : float2{-3.402823466e38f, 0.f};
        to = fmaxf(to, ml[i].x);
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) to = fmaxf(to, __shfl_xor(to, d, kWave));
    if (lane == 0) red[0][wave] = to;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < (kJoinThreads / 64); ++w) to = fmaxf(to, red[0][w]);
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxRuns / kJoinThreads; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[i].x - to);
        l += ml[i].y * f;
        weights[i * kJoinThreads + (int)threadIdx.x] = f;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) l += __shfl_xor(l, d, kWave);
    if (lane == 0) red[1][wave] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < (kJoinThreads / 64); ++w) l += red[1][w];
    v4f o = v4f{0.f, 0.f, 0.f, 0.f};
    const int64_t step = kParts * rows * D;
    at += part * rows * D;
    int s = part;
    for (; s + 3 * kParts < runs; s += 4 * kParts, at += 4 * step) {
        v4f x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const v4f*>(at + i * step);
#pragma unroll
        for (int i = 0; i < 4; ++i) o += x[i] * weights[s + i * kParts];
    }
    for (; s < runs; s += kParts, at += step) o += *reinterpret_cast<const v4f*>(at) * weights[s];
    sums[part][threadIdx.x % N] = o;
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int i = 1; i < kParts; ++i) o += sums[i][threadIdx.x];
    o = l == 0.f ? v4f{0.f, 0.f, 0.f, 0.f} : o * (1.f / l);
    *reinterpret_cast<uint2*>(a.out + row * D + col) = uint2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    if (a.lse && col == 0) a.lse[row] = l == 0.f ? -__builtin_inff() : (to + log2f(l)) * 0.693147180559945f;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Workgroups that the card holds at once.
template <int D, int W>
int held_by_lds(int rows, bool fp8) {
    const int lds = rows == 16   ? (fp8 ? Lds<D, 1, true, W>::kBytes : Lds<D, 1, false, W>::kBytes)
                    : rows == 32 ? (fp8 ? Lds<D, 2, true, W>::kBytes : Lds<D, 2, false, W>::kBytes)
                                 : (fp8 ? Lds<D, 4, true, W>::kBytes : Lds<D, 4, false, W>::kBytes);
    return 160 * 1024 / lds;
}
int held(int D, int rows, bool fp8, int waves) {
    const int by_lds = D == 64 ? (waves == 1 ? held_by_lds<64, 1>(rows, fp8) : held_by_lds<64, 4>(rows, fp8))
                               : (waves == 1 ? held_by_lds<128, 1>(rows, fp8) : held_by_lds<128, 4>(rows, fp8));
    const int by_registers = (rows == 64 ? 8 : 16) / waves;
    return 256 * (by_lds < by_registers ? by_lds : by_registers);
}

// Microseconds of runs of `run` rounds (32 positions a wave), by what was measured: 3
// until a workgroup's first tile and for its join of the waves; a round its bytes'
// share of 5.9 TB/s or, with part of the card, 0.75 (fp8: 1) and 0.6 of that; 2.5 for
// the second kernel and 0.03 a run.  8 heads of 128 columns, bf16, in runs of 1, 4, 8,
// 16, 32 and 128 rounds of four waves: one context of 32768 44.3, 29.4, 27.3, 30.5,
// 48.5 and 164 us; 8 of 8192 86, 58.5, 55.0, 52.6, 58.8 and 92.6; 64 of 4096 to 32768
// 1608, 983, 862, 831, 825 and 867.  One wave a workgroup and four: 128 contexts of 64
// 9.7 and 17.7, of 300 30.7 and 38.0, of 1024 102 and 105; fp8, 512, 34.2 and 30.1,
// 1024, 64.5 and 56.9.
double run_cost(int64_t blocks, int64_t rounds, int64_t run, int held, int round_bytes, bool fp8) {
    const int64_t slots = ceil_div(rounds, run), wgs = blocks * slots, at_once = wgs < held ? wgs : held;
    const double share = 1e-6 * round_bytes * (double)at_once / 5.9, part = (fp8 ? 1. : 0.75) + 0.6 * share;
    const double round = share > part ? share : part;
    return ceil_div(wgs, held) * (3. + round * (double)(run < rounds ? run : rounds)) + (slots > 1 ? 2.5 + 0.03 * slots : 0.);
}

KvPlan make_plan(int B, int H, int G, int D, int max_ctx, int K, bool fp8) {
    const int R = H / G;
    KvPlan p{};
    p.rows = R <= 16 ? 16 : R <= 32 ? 32 : 64;
    p.hb = ceil_div(R, p.rows);
    const int64_t len = K > 0 ? K : max_ctx, blocks = (int64_t)B * G * p.hb;
    p.waves = 4;
    int64_t run = 32;   // runs of up to 32 rounds keep contexts of different lengths even
    double best = 1e300;
    const int64_t rounds4 = ceil_div(len, kKeys * 4);
    for (const int r : {32, 24, 16, 12, 8, 6, 4, 3, 2, 1}) {
        const double us = run_cost(blocks, rounds4, r, held(D, p.rows, fp8, 4), kKeys * 4 * 2 * D * (fp8 ? 1 : 2), fp8);
        if (us < best) {
            best = us;
            run = r;
        }
    }
    // short contexts, each with one wave for all of it
    if (len <= (fp8 ? 512 : 1024)) {
        const int64_t rounds1 = len > 0 ? ceil_div(len, kKeys) : 1;
        if (run_cost(blocks, rounds1, rounds1, held(D, p.rows, fp8, 1), kKeys * 2 * D * (fp8 ? 1 : 2), fp8) < best) {
            p.waves = 1;
            run = rounds1;
        }
    }
    const int64_t rounds = ceil_div(len, kKeys * p.waves);
    // (a launch holds less than 2^32 threads: B * H is at most 2^23, so one run a sequence fits)
    while (run < rounds && (ceil_div(rounds, run) > kMaxRuns || ceil_div(rounds, run) * blocks >= (int64_t)1 << 24))
        run *= 2;
    p.run = (int)(run * kKeys * p.waves);
    p.slots = len > 0 ? ceil_div(len, p.run) : 1;
    return p;
}

template <int D, int MT, bool TOPK, bool FP8, int W>
hipError_t run(const KvDecodeArgs& a, const KvPlan& p, hipStream_t stream) {
    static PerDevice<int> once;
    constexpr int lds = Lds<D, MT, FP8, W>::kBytes;
    const hipError_t e = set_lds_limit(once, (const void*)kv_decode_kernel<D, MT, TOPK, FP8, W>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((kv_decode_kernel<D, MT, TOPK, FP8, W>), dim3((unsigned)(p.slots * a.B * a.G * p.hb)),
                       dim3(64 * W), lds, stream, a, p);
    return hipGetLastError();
}

template <int D, int MT, int W>
hipError_t run(const KvDecodeArgs& a, const KvPlan& p, bool fp8, hipStream_t stream) {
    if (a.idx) return fp8 ? run<D, MT, true, true, W>(a, p, stream) : run<D, MT, true, false, W>(a, p, stream);
    return fp8 ? run<D, MT, false, true, W>(a, p, stream) : run<D, MT, false, false, W>(a, p, stream);
}

template <int D, int W>
hipError_t run(const KvDecodeArgs& a, const KvPlan& p, bool fp8, hipStream_t stream) {
    return p.rows == 16   ? run<D, 1, W>(a, p, fp8, stream)
           : p.rows == 32 ? run<D, 2, W>(a, p, fp8, stream)
                          : run<D, 4, W>(a, p, fp8, stream);
}

template <int D>
hipError_t run(const KvDecodeArgs& a, const KvPlan& p, bool fp8, hipStream_t stream) {
    const hipError_t e = p.waves == 1 ? run<D, 1>(a, p, fp8, stream) : run<D, 4>(a, p, fp8, stream);
    if (e != hipSuccess || p.slots == 1) return e;
    hipLaunchKernelGGL(kv_join_kernel<D>, dim3((unsigned)(a.B * a.H)), dim3(kJoinThreads), 0, stream, a, p);
    return hipGetLastError();
}

}  // namespace

// The caller's workspace holds the sums, then the (maximum, sum) pairs.
size_t kv_decode_workspace_bytes(int B, int H, int G, int D, int max_ctx, int K, bool fp8) {
    const KvPlan p = make_plan(B, H, G, D, max_ctx, K, fp8);
    return p.slots == 1 ? 0 : (size_t)p.slots * B * H * (D + 2) * sizeof(float);
}

hipError_t launch_kv_decode(const KvDecodeArgs& a, int D, bool fp8, hipStream_t stream) {
    KvPlan p = make_plan(a.B, a.H, a.G, D, a.max_ctx, a.idx ? a.K : 0, fp8);
    p.part_o = reinterpret_cast<float*>(a.workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)p.slots * a.B * a.H * D);
    return D == 64 ? run<64>(a, p, fp8, stream) : run<128>(a, p, fp8, stream);
}

}  // namespace dsaidx
