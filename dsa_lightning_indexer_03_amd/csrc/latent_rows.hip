// Attention over the paged latent cache for blocks of many query rows: 64 or
// 128 of one query's heads, or of the batch's rows stacked against a shared
// prefix (the formulas: latent_attention.hip).
//
// One workgroup of eight waves shares each staged 64-key tile; a wave owns 16
// query rows and carries them alone through both products:
//   S^T (64 keys x 16 rows) = K Q^T, its queries in registers;
//   O^T (512 columns x 16 rows) += V^T P^T.
// The first product leaves a lane with row lane % 16 and keys 4g .. 4g+3
// (g = lane / 16) of each 16-key block, which is the second one's operand
// when its 32 keys are counted as 4g .. 4g+3 of two blocks: P never leaves its
// registers, and the values are read transposed in that order.  So waves meet
// only where a tile is handed over, and the two waves of a SIMD fill each
// other's pauses.  The exponent's reference moves when a score of the wave's
// rows passes it by 2^kSlack.  With 64 rows the waves form two groups of four,
// each with half of every tile's keys, joined through LDS at the end.
//
// fp8 rows are staged as codes two tiles ahead.  Beside the products of one half
// tile, 32 keys, the next half is widened to bf16 in the other of two buffers,
// once for all rows: in registers every wave would widen every operand.  The
// rows' scales multiply the scores and P.  With 64 rows four waves compute and
// the other four copy and widen.
//
// Bound by the matrix cores and, behind them, LDS reads: a tile of 128 rows
// needs 4352 cycles of the first (a SIMD) and, at the measured rates of the two
// kinds of reads, 5200 of the second.  1000 queries of 128 heads, 2048 selected
// rows of 576 (571 GFLOP): 552 us a call, calls in a row (1.03 PFLOP/s); 64
// queries of 128 heads on a prefix of 32751 (588 GFLOP): 526 us (1.12), where a
// bf16 matrix product of 8192 cubed reached 1.09 to 1.28: at these rates the
// power limit sets the clock, by card and by run (542 and 515 us on another card,
// medians of 593 and 552 in a profile's bursts; with zeros for data the second
// takes 449).  fp8 rows: 587 and 557 us.
#include "device_once.h"
#include "latent_common.h"

namespace dsaidx {
namespace {

constexpr int kThreads = 512;
constexpr int kAhead = 3;   // operand reads in flight
constexpr int kLds = 2 * kTileB;
static_assert(4 * 32 * 64 * 16 + 4 * 64 * 8 <= kLds, "the join of two key groups fits the tiles' place");
// fp8: two half tiles, two tiles of codes (512 bytes a row, then 64 of rotary
// columns a row), the scales of four tiles
constexpr int kHalfB = kTileB / 2;
constexpr int kCodesAt = 2 * kHalfB;
constexpr int kCodesB = kTile * (kV + 64);
constexpr int kScaleAt = kCodesAt + 2 * kCodesB;
constexpr int kLds8 = kScaleAt + 4 * kTile * 4;
static_assert(kLds <= 160 * 1024 && kLds8 <= 160 * 1024, "LDS budget");

template <int KD, int KG, bool TOPK, bool FP8>
__global__ void __launch_bounds__(kThreads, 2)
latent_rows_kernel(LatentArgs a, LatentPlan p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int E = 32 * KD;
    constexpr int RB = FP8 ? E : 2 * E;
    constexpr int RG = 8 / KG;            // row groups of 16
    constexpr bool kMovers = FP8 && KG == 2;    // the second four waves move data for the first
    constexpr int kMainParts = FP8 && KG == 1 ? 4 : 8, kParts = kMainParts + (KD > 16);  // copies of a tile that a wave makes
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int n = lane & 15, g = lane >> 4;
    const int rg = wave % RG, kg = wave / RG;
    LatentKeys<TOPK> keys;
    if (!keys.start(a, p)) return;
    const int nrows = keys.nrows, t1 = keys.t1;
    const bool active = 16 * rg < nrows && !(kMovers && kg == 1);
    const bool mover = !kMovers || kg == 1;

    // ---- queries: B operand of 16 rows x 32 columns ----
    v8bf Q[KD];
    {
        const uint16_t* qp = a.q + (int64_t)(keys.r0 + min(16 * rg + n, nrows - 1)) * E + 8 * g;
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) Q[ks] = *reinterpret_cast<const v8bf*>(qp + 32 * ks);
    }

    // The lane, made anew for every phase: what follows from it, kept longer,
    // would cost registers that the queries and sums need (or spill, and a reload
    // waits for every copy in flight).
    int ln = lane;
    auto renew = [&]() { asm volatile("" : "+v"(ln)); };
    // x of another lane
    auto from_lane = [](int x, int i) { return __builtin_amdgcn_ds_bpermute(4 * i, x); };
    auto across = [&](float x, int d) { return __int_as_float(from_lane(__float_as_int(x), ln ^ d)); };

    // ---- copies: rows kb .. of a tile; fp8: their codes two rows at a time, the rotary
    //      columns of 16 rows by each of four waves, the scales by one ----
    const int kb = kMovers ? 16 * (wave & 3) : 8 * wave;
    const uint32_t lds0 = lds_address(smem);
    int rope_row = -1;   // bf16: the row whose rotary columns this lane copies a piece of
    auto spread = [&]() {
        if constexpr (KD > 16 && !FP8) rope_row = __shfl(keys.row, kb + (lane >> 3));
    };
    auto stage = [&](int buf, int i) {
        if constexpr (FP8) {
            const uint32_t lds = lds0 + kCodesAt + buf * kCodesB;
            if (i < kMainParts) {
                const int mine = from_lane(keys.row, kb + 2 * i + (ln >> 5));
                copy_to_lds(row_address<RB>(a.cache, mine) + 16 * (ln & 31), lds + (kb + 2 * i) * kV);
            } else if (kMovers || wave < 4) {
                const int r = 16 * (wave & 3), mine = from_lane(keys.row, r + (ln >> 2));
                copy_to_lds(row_address<RB>(a.cache, mine) + kV + 16 * (ln & 3), lds + kTile * kV + r * 64);
            }
        } else {
            const uint32_t lds = lds0 + buf * kTileB;
            if (i < 8) {
                copy_to_lds(row_address<RB>(a.cache, __builtin_amdgcn_readlane(keys.row, kb + i)), 16 * lane,
                            lds + (kb + i) * kRowB);
            } else {
                const int piece = (lane & 7) ^ ((kb / 2 + (lane >> 4)) & 7);
                copy_to_lds(row_address<RB>(a.cache, rope_row) + 2 * kV + 16 * piece, lds + kMainB + kb * 128);
            }
        }
    };
    auto stage_scales = [&](int at) {   // a tile's place among four
        if constexpr (FP8)
            if (wave == 4)
                copy4_to_lds(row_address<4>(a.cache_scale, keys.row), lds0 + kScaleAt + at * kTile * 4);
    };

    LatentAhead ahead;
    int t = keys.seek(keys.t0, ahead);
    int t_next = t;
    // the first tile with a row behind t_next, from what is ahead of it
    auto advance = [&]() {
        ++t_next;
        keys.resolve(t_next < t1 ? keys.entry_of(t_next, ahead.s2) : -1, ahead.page2);
        if (keys.mask == 0 && t_next < t1) {
            t_next = keys.seek(t_next + 1, ahead);
        } else {
            ahead.s2 = ahead.s3;
            ahead.page2 = keys.page(ahead.s2, t_next + 1);
            ahead.s3 = keys.entry(t_next + 2);
        }
        spread();
    };
    uint64_t here = keys.mask;
    const float shift = FP8 ? scale_shift(keys, a.cache_scale) : 0.f;
    spread();
    if (mover) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) stage(0, i);
        stage_scales(0);
    }
    int buf = 0;
    advance();

    if (a.scale_log2 < 0.f)   // the products then take the scale's magnitude
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            v4i u = __builtin_bit_cast(v4i, Q[ks]);
            u ^= (int)0x80008000;
            Q[ks] = __builtin_bit_cast(v8bf, u);
        }
    // (never 0: a score of -inf, an entry without a row, has to stay one)
    const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);

    v4f O[32];
#pragma unroll
    for (int ct = 0; ct < 32; ++ct) O[ct] = v4f{0.f, 0.f, 0.f, 0.f};
    // the reference starts below every score that is not -inf, so that a row's first one moves it
    float m = -3.402823466e38f, l = 0.f;

    // 32 keys, the rows at `tile` and their rotary columns at `rope`, through both
    // products; `live` says which have a row, `by` are their scales; between the steps
    // of each product the calls of beside_k and beside_v
    auto half = [&](const unsigned char* tile, const unsigned char* rope, uint32_t live, const unsigned char* by,
                    auto beside_k, auto beside_v) __attribute__((always_inline)) {
        // ---- scores ----
        renew();
        const unsigned char* kp = tile + (ln & 15) * kRowB + 16 * (ln >> 4);
        const unsigned char* kr = rope + (ln & 15) * 128;
        auto read_k = [&](int f) {   // step f: columns 32 (f / 2) .., keys 16 (f % 2) ..
            const int ks = f / 2, kt = f % 2;
            return *reinterpret_cast<const v8bf*>(
                ks < 16 ? kp + 16 * kt * kRowB + 64 * ks
                        : kr + 16 * kt * 128 + 16 * ((4 * (ks - 16) + (ln >> 4)) ^ ((ln >> 1) & 7)));
        };
        v4f S[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
        v8bf K[kAhead];
#pragma unroll
        for (int f = 0; f < kAhead; ++f) K[f] = read_k(f);
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const int f = 2 * ks + kt;
                S[kt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(K[f % kAhead], Q[ks], S[kt], 0, 0, 0);
                if (f + kAhead < 2 * KD) K[f % kAhead] = read_k(f + kAhead);
            }
            beside_k(ks);
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- softmax ----
        renew();
        v4f by4[2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            if constexpr (FP8) {
                by4[kt] = *reinterpret_cast<const v4f*>(by + 64 * kt + 16 * (ln >> 4));
                S[kt] *= by4[kt];
            }
            S[kt] = scaled_scores(S[kt], scale);
        }
        if (live != ~0u) {
            const uint32_t mine = live >> (4 * (ln >> 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[0][i] = mine >> i & 1 ? S[0][i] : -__builtin_inff();
                S[1][i] = mine >> (16 + i) & 1 ? S[1][i] : -__builtin_inff();
            }
        }
        float top = fmaxf(S[0][0], S[1][0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) top = fmaxf(top, fmaxf(S[0][i], S[1][i]));
        if (wave_ballot(top > m + (kSlack - shift))) {
            // the reference moves to these keys' maximum where that is above it
            top = fmaxf(top, across(top, 16));
            top = fmaxf(top, across(top, 32));
            const float to = fmaxf(m, top + shift);
            const float f = __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int ct = 0; ct < 32; ++ct) O[ct] *= f;
        }
        v4i u;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            float pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pr[i] = __builtin_amdgcn_exp2f(S[kt][i] - m);
                l += pr[i];
                if constexpr (FP8) pr[i] *= by4[kt][i];
            }
            u[2 * kt] = (int)pack_bf16(pr[0], pr[1]);
            u[2 * kt + 1] = (int)pack_bf16(pr[2], pr[3]);
        }
        const v8bf P = __builtin_bit_cast(v8bf, u);
        // ---- values ----
        const unsigned char* vp = tile + (4 * (ln >> 4) + (ln >> 2 & 3)) * kRowB + 8 * (ln & 3);
        auto read_v = [&](int ct) {
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(vp + 32 * ct));
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(vp + 32 * ct + 16 * kRowB));
            return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        v8bf W[kAhead];
#pragma unroll
        for (int f = 0; f < kAhead; ++f) W[f] = read_v(f);
#pragma unroll
        for (int ct = 0; ct < 32; ++ct) {
            if (ct % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            O[ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(W[ct % kAhead], P, O[ct], 0, 0, 0);
            if (ct + kAhead < 32) W[ct % kAhead] = read_v(ct + kAhead);
            if (ct == 8) beside_v();
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // fp8: rows r4 .. r4+3 of half hb of the codes in buffer `from`, to bf16 in half buffer hb.
    // Steps 0 .. 17, a row at a time: read, and written three steps later.
    uint2 codes{0, 0}, rope_codes{0, 0};
    auto widen = [&](int from, int hb, int r4, int step) {
        const int r = 32 * hb + r4;
        const unsigned char* in = smem + kCodesAt + from * kCodesB;
        unsigned char* out = smem + hb * kHalfB;
        if (step < 16 && step % 4 == 0)
            codes = *reinterpret_cast<const uint2*>(in + (r + step / 4) * kV + 8 * ln);
        if (step < 16 && step % 4 == 3)
            *reinterpret_cast<v4i*>(out + (r4 + step / 4) * kRowB + 16 * ln) = widen8(codes);
        if constexpr (KD > 16) {   // (both halves of the wave the same)
            const int row = r4 + (ln >> 3 & 3);
            if (step == 14)
                rope_codes = *reinterpret_cast<const uint2*>(in + kTile * kV + (32 * hb + row) * 64 + 8 * (ln & 7));
            if (step == 17)
                *reinterpret_cast<v4i*>(out + 32 * kRowB + row * 128 + 16 * ((ln & 7) ^ ((row >> 1) & 7))) =
                    widen8(rope_codes);
        }
    };
    auto widen_all = [&](int from, int hb) {   // this wave's rows, at once
#pragma unroll
        for (int j = 0; j < (kMovers ? 2 : 1); ++j)
#pragma unroll
            for (int step = 0; step < 18; ++step) widen(from, hb, kMovers ? 8 * (wave & 3) + 4 * j : 4 * wave, step);
    };

    int at = 0;   // fp8: the place of this tile's scales
    if constexpr (FP8) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the first tile
        tile_barrier();
        if (mover) {
            widen_all(0, 0);
#pragma unroll
            for (int i = 0; i < kParts; ++i) stage(1, i);
            stage_scales(1);
        }
    }

    while (t < t1) {
        if constexpr (!FP8) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the tile
        tile_barrier();
        // loads for the tiles behind the next one
        const int page3 = keys.page(ahead.s3, t_next + 2);
        const int s4 = keys.entry(t_next + 3);
        const int t_now = t_next;
        const uint64_t next = keys.mask;
        // the rows of the tile behind the next one
        auto resolve = [&]() {
            keys.resolve(t_now + 1 < t1 ? keys.entry_of(t_now + 1, ahead.s2) : -1, ahead.page2);
            spread();
        };
        auto step = [&]() {
            t_next = t_now + 1;
            ahead = LatentAhead{ahead.s3, page3, s4};
            if (keys.mask == 0 && t_next < t1) {
                t_next = keys.seek(t_next + 1, ahead);
                spread();
            }
        };
        if constexpr (FP8) {
            const unsigned char* by = smem + kScaleAt + at * kTile * 4;
            auto first = [&](int ks) {
                if constexpr (!kMovers) widen(buf, 1, 4 * wave, ks);
            };
            if (active) {
                half(smem, smem + 32 * kRowB, (uint32_t)here, by, first, resolve);
            } else {
                if (mover) widen_all(buf, 1);
                resolve();
            }
            step();
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the next tile
            tile_barrier();
            auto second = [&](int ks) {   // behind the last tile: zeros
                if constexpr (!kMovers) {
                    widen(buf ^ 1, 0, 4 * wave, ks);
                    if (ks % 4 == 1 && ks / 4 < kParts) stage(buf, ks / 4);
                    if (ks == 2) stage_scales((at + 2) & 3);
                }
            };
            if (active) {
                half(smem + kHalfB, smem + kHalfB + 32 * kRowB, (uint32_t)(here >> 32), by + 128, second, [] {});
            } else if (mover) {
#pragma unroll
                for (int i = 0; i < kParts; ++i) stage(buf, i);
                stage_scales((at + 2) & 3);
                widen_all(buf ^ 1, 0);
            }
            at = (at + 1) & 3;
        } else {
            const unsigned char* tile = smem + buf * kTileB;
            if (active) {
                auto copies = [&](int ks) {   // behind the last tile: zeros
                    if (ks % 2 == 0 && ks / 2 < kParts) stage(buf ^ 1, ks / 2);
                };
                if constexpr (KG == 2) {
                    half(tile + 32 * kg * kRowB, tile + kMainB + 32 * kg * 128, (uint32_t)(here >> (32 * kg)), nullptr,
                         copies, resolve);
                } else {
                    half(tile, tile + kMainB, (uint32_t)here, nullptr, copies, [] {});
                    half(tile + 32 * kRowB, tile + kMainB + 32 * 128, (uint32_t)(here >> 32), nullptr, [](int) {},
                         resolve);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kParts; ++i) stage(buf ^ 1, i);
                resolve();
            }
            step();
        }
        here = next;
        buf ^= 1;
        t = t_now;
    }

    // ---- join the key groups, write ----
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no copy may still be in flight
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
    if constexpr (kMovers) {
        if (kg == 1) return;
    } else if constexpr (KG == 2) {
        v4f* there = reinterpret_cast<v4f*>(smem) + rg * 32 * 64 + lane;
        float2* ml = reinterpret_cast<float2*>(smem + 4 * 32 * 64 * 16) + rg * 64 + lane;
        tile_barrier();
        if (kg == 1) {
#pragma unroll
            for (int ct = 0; ct < 32; ++ct) there[64 * ct] = O[ct];
            *ml = float2{m, l};
        }
        tile_barrier();
        if (kg == 1) return;
        const float2 b = *ml;
        const float to = fmaxf(m, b.x);
        const float f = __builtin_amdgcn_exp2f(m - to), fb = __builtin_amdgcn_exp2f(b.x - to);
        m = to;
        l = l * f + b.y * fb;
#pragma unroll
        for (int ct = 0; ct < 32; ++ct) O[ct] = O[ct] * f + there[64 * ct] * fb;
    }
    if (16 * rg + n >= nrows) return;
    const int64_t r = keys.r0 + 16 * rg + n;
    if (p.slots == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* out = a.out + r * kV + 4 * g;
#pragma unroll
        for (int ct = 0; ct < 32; ++ct) {
            const v4f o = O[ct] * inv;
            *reinterpret_cast<uint2*>(out + 16 * ct) = uint2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
        }
        if (a.lse && g == 0) a.lse[r] = l == 0.f ? -__builtin_inff() : (m + log2f(l)) * 0.693147180559945f;
    } else {
        const int64_t at = (int64_t)keys.slot * (a.T * a.H) + r;
        if (l != 0.f) {   // (NaN too)
            float* out = p.part_o + at * kV + 4 * g;
#pragma unroll
            for (int ct = 0; ct < 32; ++ct) *reinterpret_cast<v4f*>(out + 16 * ct) = O[ct];
        }
        if (g == 0) p.part_ml[at] = float2{m, l};
    }
}

template <int KD, int KG, bool TOPK, bool FP8>
hipError_t run(const LatentArgs& a, const LatentPlan& p, hipStream_t stream) {
    static PerDevice<int> once;
    constexpr int lds = FP8 ? kLds8 : kLds;
    const hipError_t e = set_lds_limit(once, (const void*)latent_rows_kernel<KD, KG, TOPK, FP8>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((latent_rows_kernel<KD, KG, TOPK, FP8>), dim3((unsigned)(p.n_prefix + p.n_own)), dim3(kThreads),
                       lds, stream, a, p);
    return hipGetLastError();
}

template <int KD, int KG>
hipError_t run(const LatentArgs& a, const LatentPlan& p, bool fp8, hipStream_t stream) {
    if (a.idx) return fp8 ? run<KD, KG, true, true>(a, p, stream) : run<KD, KG, true, false>(a, p, stream);
    return fp8 ? run<KD, KG, false, true>(a, p, stream) : run<KD, KG, false, false>(a, p, stream);
}

template <int KD>
hipError_t run(const LatentArgs& a, const LatentPlan& p, bool fp8, hipStream_t stream) {
    return p.rows == 64 ? run<KD, 2>(a, p, fp8, stream) : run<KD, 1>(a, p, fp8, stream);
}

}  // namespace

hipError_t launch_latent_rows(const LatentArgs& a, const LatentPlan& p, bool fp8, hipStream_t stream) {
    return a.E == 576 ? run<18>(a, p, fp8, stream) : run<16>(a, p, fp8, stream);
}

}  // namespace dsaidx
