// Attention over the paged latent cache: every head of a query reads the same
// E-wide rows, whose first V columns are the values.
//
//   S[h, j] = scale * q[h] . c[j],  P = softmax_j S,  out[h] = sum_j P[h, j] c[j][:V]
//   lse[h] = log sum_j exp S[h, j]       (no key: out = 0, lse = -inf)
//
// The keys of query t are the rows at its selected positions (topk), or the
// rows of a prefix that the whole batch shares followed by the sequence's own
// (shared).  "Study MLA Indexer", the data-flow diagram's last step; "Lightning
// Indexer explained", section 1.
//
// Here: blocks of 16 or 32 query rows (larger ones: latent_rows.hip), the
// choice of block and split, and the join.  One workgroup takes a block (a
// query's heads, or the stacked heads of several queries for the shared prefix)
// and a run of 64-key tiles.  A tile is staged once in LDS and serves both
// products; with four waves, for 16 rows:
//   S^T (16 keys x rows) = K Q^T: wave w has keys 16w .. 16w+15, the queries
//     sit in its registers;
//   O^T (128 columns x rows) += V^T P^T: wave w has columns 128w .. 128w+127,
//     the probabilities of all 64 keys come through LDS as bf16, the values
//     are read transposed from the same tile.
// Eight waves, for 32 rows, take 16 keys and 16 rows each, and 64 columns: 229
// us for 1000 queries of 32 heads, 2048 selected, where four took 239.  Both
// products leave a lane with one query row (lane % 16 of each 16-row block), so
// the softmax's factors are per lane.  The exponent's reference m is common to
// the waves and only moves when a score exceeds it by more than kSlack
// (base 2): a flag in LDS, read behind the barrier that the exchange of P needs
// anyway, sends all waves through a second pass that takes the tile's maximum,
// rescales and rewrites P.  Sums are fp32; P is rounded to bf16, because the
// matrix cores take both operands of the second product in the values' type: an
// output is off by at most 2^-8 of sum P |c| for that, beside its own rounding
// (2.0e-3 rms of the outputs where the rounding alone is 1.7e-3; a second
// operand with the rest of P would double that product).  P's sum is taken before
// the rounding, so that lse does not have it.
// When the rows alone do not fill the GPU the key tiles are split over
// workgroups, whose fp32 partial sums a second kernel joins by their maxima.
//
// With few rows a tile is bound by its bytes: 64 queries of 16 heads, 2048 rows
// of 1152 bytes each, take 31 us and the join 5, 4.9 TB/s of distinct rows (a
// 1 GiB copy reaches 5.2 read and written).  1000 queries of 16 heads on 4
// sequences take 214 us, 11 TB/s of rows from the caches; most of a tile's 1.7
// us is the wait for its copies.  With one query it is latency: 32 workgroups
// of one tile take 8 us, four dependent loads and the launch, and the join 4.
#include "device_once.h"
#include "latent_common.h"

namespace dsaidx {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 2048;   // from here on a wave joins a row

// LDS: two tiles, P (its rows padded like a bf16 tile's), the exchange of
// maxima and sums, the rows' fp8 scales, flags.  The queries pass through the
// second tile's place and what lies behind it.
//
// An fp8 tile holds the codes, two rows of 512 bytes and 16 bytes of padding at
// a time; odd rows have the halves of each 256 bytes swapped.  There a wave's 16
// keys are every second row of 32, so that both an operand read (16 rows) and a
// transposed one (16 rows) use every bank once.  Then 64 bytes a row of rotary
// columns, their 16-byte pieces permuted within the row.
constexpr int kPRowB = 2 * kTile + 32;
constexpr int kPairB = 2 * kV + 16;
template <int KD, int MT, bool FP8>
struct Lds {
    static constexpr int kMain = FP8 ? kTile / 2 * kPairB : kMainB;                // a tile's value columns,
    static constexpr int kRope = KD > 16 ? (FP8 ? kTile * 64 : kRopeB) : 0;        // and rotary columns
    static constexpr int kRopeAt = 2 * kMain;
    static constexpr int kP = kRopeAt + 2 * kRope;
    static constexpr int kRed = kP + MT * 16 * kPRowB;     // [4][16 MT] floats
    static constexpr int kScale = kRed + 4 * 16 * MT * 4;  // [2][64] floats
    static constexpr int kFlag = kScale + (FP8 ? 512 : 0); // [2]
    static constexpr int kUsed = kFlag + 16;
    // queries: 16 MT padded rows, in the second tile's place or, too large for
    // it, behind both; their rotary columns behind them
    static constexpr int kQ = FP8 ? kP : kMain;
    static constexpr int kQRope = kQ + MT * 16 * kRowB;
    static constexpr int kQEnd = kQRope + (KD > 16 ? MT * 16 * 128 : 0);
    static constexpr int kBytes = kUsed > kQEnd ? kUsed : kQEnd;
    static_assert(kBytes <= 160 * 1024, "LDS budget");
};

// An operand as it is read: eight bf16, or eight codes that are widened for use.
template <bool FP8>
struct Operand {
    v8bf x;
    __device__ __forceinline__ v8bf get() const { return x; }
};
template <>
struct Operand<true> {
    v2i x;
    __device__ __forceinline__ v8bf get() const {
        return __builtin_bit_cast(v8bf, widen8(uint2{(uint32_t)x[0], (uint32_t)x[1]}));
    }
};

// Four waves for 16 rows, eight for 32.
constexpr int waves_of(int mt) { return 4 * mt; }

template <int KD, int MT, bool TOPK, bool FP8>
__global__ void __launch_bounds__(64 * waves_of(MT), MT)
latent_attention_kernel(LatentArgs a, LatentPlan p) {
    extern __shared__ __align__(16) unsigned char smem[];
    using L = Lds<KD, MT, FP8>;
    constexpr int E = 32 * KD;
    constexpr int RB = FP8 ? E : 2 * E;   // bytes of a cached row
    constexpr int NW = waves_of(MT);
    constexpr int CT = 32 / NW;           // 16-column blocks of the values that a wave computes
    constexpr int kAhead = 3;             // operand reads in flight
    constexpr int KB = kTile / NW;        // rows of a tile that a wave copies
    constexpr int kMainParts = FP8 ? KB / 2 : KB, kParts = kMainParts + (KD == 16 ? 0 : FP8 ? 1 : KB / 8);
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int n = lane & 15, g = lane >> 4;
    const int kq = wave & 3, mq = wave >> 2;   // whose 16 keys' and 16 rows' scores this wave computes
    const int total = a.T * a.H;
    LatentKeys<TOPK> keys;
    if (!keys.start(a, p)) return;
    const int nrows = keys.nrows, t1 = keys.t1;
    const int kb = KB * wave;   // the rows of a tile that this wave copies
    const uint32_t lds0 = lds_address(smem);

    // ---- queries: copied to LDS, read as operands below ----
    {
        const uint16_t* q = a.q + (int64_t)keys.r0 * E;
#pragma unroll
        for (int i = 0; i < 16 * MT / NW; ++i) {
            const int r = 16 * MT / NW * wave + i;
            copy_to_lds(q + (int64_t)min(r, nrows - 1) * E, 16 * lane, lds0 + L::kQ + r * kRowB);
        }
        if constexpr (KD > 16)
            if (wave < 2 * MT) {
                const int r = 8 * wave + (lane >> 3);
                copy_to_lds(q + (int64_t)min(r, nrows - 1) * E + kV + 8 * ((lane & 7) ^ ((r >> 1) & 7)),
                            lds0 + L::kQRope + 8 * wave * 128);
            }
    }

    // ---- copies: rows kb .. kb + KB - 1 of a tile ----
    // bf16: parts a row each, then the rotary columns of 8 rows each; fp8: parts
    // of two rows each, then the rotary columns of 16 (by four waves).  A lane of a
    // part that covers several rows needs its own row: part_row, found one part
    // ahead.
    auto part_row = [&](int i) -> int {
        if constexpr (FP8)
            return __shfl(keys.row, i < kMainParts ? kb + 2 * i + (lane >> 5) : 16 * kq + (lane >> 2));
        return i < kMainParts ? -1 : __shfl(keys.row, kb + 8 * (i - kMainParts) + (lane >> 3));
    };
    uint64_t src = 0;   // bf16: addresses of the next tile's rows
    auto address = [&]() {
        if constexpr (!FP8) src = (uint64_t)row_address<RB>(a.cache, keys.row);
    };
    auto rope_piece = [&](int r) { return 16 * ((lane & 7) ^ ((r >> 1) & 7)); };
    auto stage = [&](int buf, int i, int mine) {
        const uint32_t lds = lds0 + buf * L::kMain, rope = lds0 + L::kRopeAt + buf * L::kRope;
        if constexpr (FP8) {
            if (i < kMainParts) {
                copy_to_lds(row_address<RB>(a.cache, mine) + 16 * ((lane & 31) ^ (lane >> 5) * 8),
                            lds + (kb / 2 + i) * kPairB);
            } else if (NW == 4 || wave < 4) {
                const int r = 16 * kq + (lane >> 2);
                copy_to_lds(row_address<RB>(a.cache, mine) + kV + 16 * ((lane & 3) ^ ((r >> 2) & 3)),
                            rope + 16 * kq * 64);
            }
        } else if (i < kMainParts) {
            copy_to_lds(lane_pointer(src, kb + i), 16 * lane, lds + (kb + i) * kRowB);
        } else {
            const int r = kb + 8 * (i - kMainParts);
            copy_to_lds(row_address<RB>(a.cache, mine) + 2 * kV + rope_piece(r + (lane >> 3)), rope + r * 128);
        }
    };
    float kscale = 0.f;   // fp8: scale of the next tile's entry `lane`
    auto load_scale = [&]() {
        if constexpr (FP8) kscale = keys.row >= 0 ? a.cache_scale[keys.row] : 0.f;
    };
    auto store_scale = [&](int buf) {
        if constexpr (FP8)
            if (wave == 0)   // in the order of the waves' keys
                reinterpret_cast<float*>(smem + L::kScale)[64 * buf + (lane & 32) + 16 * (lane & 1) + (lane >> 1 & 15)] =
                    kscale;
    };

    LatentAhead ahead;
    int t = keys.seek(keys.t0, ahead);
    uint64_t here = keys.mask;   // the entries of the tile that is computed
    const float shift = FP8 ? scale_shift(keys, a.cache_scale) : 0.f;
    address();
#pragma unroll
    for (int i = 0; i < kParts; ++i) stage(0, i, part_row(i));
    load_scale();
    int t_next = t + 1, buf = 0;
    // the tile behind t, from what is ahead of it
    keys.resolve(t_next < t1 ? keys.entry_of(t_next, ahead.s2) : -1, ahead.page2);
    if (keys.mask == 0 && t_next < t1) {
        t_next = keys.seek(t_next + 1, ahead);
    } else {
        ahead.s2 = ahead.s3;
        ahead.page2 = keys.page(ahead.s2, t_next + 1);
        ahead.s3 = keys.entry(t_next + 2);
    }
    address();
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): queries and first tile
    tile_barrier();
    // B operand of 16 rows x 32 columns: row n, columns 8g .. 8g+7 of each 32
    v8bf Q[KD];
    auto read_q = [&](int mt, int ks) {
        const int r = 16 * mt + n;
        v8bf q = *reinterpret_cast<const v8bf*>(
            smem + (ks < 16 ? L::kQ + r * kRowB + 16 * g + 64 * ks
                            : L::kQRope + r * 128 + 16 * ((4 * (ks - 16) + g) ^ ((n >> 1) & 7))));
        if (a.scale_log2 < 0.f) {   // the products then take the scale's magnitude
            v4i u = __builtin_bit_cast(v4i, q);
            u ^= (int)0x80008000;
            q = __builtin_bit_cast(v8bf, u);
        }
        return q;
    };
#pragma unroll
    for (int ks = 0; ks < KD; ++ks) Q[ks] = read_q(mq, ks);
    // (never 0: a score of -inf, an entry without a row, has to stay one)
    const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
    tile_barrier();
    int* flag = reinterpret_cast<int*>(smem + L::kFlag);   // [buf]
    float* red = reinterpret_cast<float*>(smem + L::kRed);
    if (threadIdx.x < 2) flag[threadIdx.x] = 0;
    store_scale(0);

    v4f O[CT][MT];
    float m[MT], l = 0.f;   // all rows' references; the sums of the rows and keys whose scores are this wave's
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -3.402823466e38f;   // the lowest finite: any score but -inf moves it
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) O[ct][mt] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    // The lane, made anew for every tile and phase: what follows from it, kept
    // longer, would cost registers that the queries and sums need.
    int ln = lane;
    auto renew = [&]() { asm volatile("" : "+v"(ln)); };
    // A operand of the scores: this wave's 16 keys, 32 columns of step ks
    auto read_k = [&](int buf, int ks) {
        const unsigned char *tile = smem + buf * L::kMain, *rope = smem + L::kRopeAt + buf * L::kRope;
        Operand<FP8> k;
        const int n = ln & 15, g = ln >> 4;
        if constexpr (FP8) {
            const int odd = kq & 1, q = 16 * (kq >> 1) + n;   // row 2q + odd
            k.x = *reinterpret_cast<const v2i*>(
                ks < 16 ? tile + q * kPairB + kV * odd + 8 * g + (ks & 4 ? -128 : 128) * odd + 32 * ks
                        : rope + (2 * q + odd) * 64 + 16 * ((2 * (ks - 16) + (g >> 1)) ^ ((n >> 1) & 3)) +
                              8 * (g & 1));
        } else {
            k.x = *reinterpret_cast<const v8bf*>(
                ks < 16 ? tile + (16 * kq + n) * kRowB + 16 * g + 64 * ks
                        : rope + (16 * kq + n) * 128 + 16 * ((4 * (ks - 16) + g) ^ ((n >> 1) & 7)));
        }
        return k;
    };
    // A operand of the values: 16 columns of this wave's 16 CT, keys 4g .. 4g+3
    // of two 16-key blocks; step i: columns 16 (i % CT) .., keys 32 (i / CT) ..
    auto read_v = [&](int buf, int i) {
        const unsigned char* tile = smem + buf * L::kMain;
        Operand<FP8> w;
        const int n = ln & 15, g = ln >> 4;
        if constexpr (FP8) {
            const int j = n >> 1, odd = j >> 2, q = 16 * (i / CT) + 4 * g + (j & 3);
            const unsigned char* at =
                tile + q * kPairB + kV * odd + ((16 * CT * wave) ^ (128 * odd)) + 16 * (i % CT) + 8 * (n & 1);
            w.x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)at);
        } else {
            const unsigned char* at =
                tile + (32 * (i / CT) + 4 * g + (n >> 2)) * kRowB + 8 * (n & 3) + 32 * CT * wave + 32 * (i % CT);
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 16 * kRowB));
            w.x = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return w;
    };
    Operand<FP8> K[kAhead], W[kAhead];
    v8bf P[MT];
    v4f S;
    float sum = 0.f, ks4[4] = {1.f, 1.f, 1.f, 1.f};
    auto read_p = [&](int kk) {
        const int n = ln & 15, g = ln >> 4;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            P[mt] = *reinterpret_cast<const v8bf*>(smem + L::kP + (16 * mt + n) * kPRowB + 16 * (4 * kk + g));
    };
    auto own_m = [&]() { return MT == 1 || mq == 0 ? m[0] : m[MT - 1]; };
    auto write_p = [&]() {
        const int n = ln & 15, g = ln >> 4;
        const float ref = own_m();
        float pr[4];
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            pr[e] = __builtin_amdgcn_exp2f(S[e] - ref);
            sum += pr[e];
            if constexpr (FP8) pr[e] *= ks4[e];
        }
        // P[row][key]: 16-byte piece 4(kq/2) + g holds the keys 4g .. 4g+3 of the key blocks
        // 2(kq/2) and 2(kq/2) + 1
        *reinterpret_cast<uint2*>(smem + L::kP + (16 * mq + n) * kPRowB + 16 * (4 * (kq >> 1) + g) + 8 * (kq & 1)) =
            uint2{pack_bf16(pr[0], pr[1]), pack_bf16(pr[2], pr[3])};
    };
    auto highest = [&]() { return fmaxf(fmaxf(S[0], S[1]), fmaxf(S[2], S[3])); };
    // The rows' references move to the tile's maxima where those are above them.
    auto rebase = [&]() {
        float top = highest();
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        if (g == 0) red[kq * 16 * MT + 16 * mq + n] = top + shift;
        tile_barrier();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float v = m[mt];
#pragma unroll
            for (int w = 0; w < 4; ++w) v = fmaxf(v, red[w * 16 * MT + 16 * mt + n]);
            const float f = __builtin_amdgcn_exp2f(m[mt] - v);
            m[mt] = v;
            if (mt == mq) l *= f;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) O[ct][mt] *= f;
        }
        write_p();
        tile_barrier();
        read_p(0);
    };

    tile_barrier();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) K[i] = read_k(0, i);
    while (t < t1) {
        renew();
        // loads for the tiles behind the next one
        const int page3 = keys.page(ahead.s3, t_next + 2);
        const int s4 = keys.entry(t_next + 3);
        load_scale();
        const int t_now = t_next;
        const uint64_t next = keys.mask;
        int mine = part_row(0);
        S = v4f{0.f, 0.f, 0.f, 0.f};

        // ---- scores: S^T, keys 4g .. 4g+3 of this wave's 16, row n of each block; beside
        //      them the next tile's copies (behind the last tile: zeros that nobody reads) ----
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            __builtin_amdgcn_sched_barrier(0);
            const v8bf k = K[ks % kAhead].get();
            S = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, Q[ks], S, 0, 0, 0);
            if (ks + kAhead < KD) K[ks % kAhead] = read_k(buf, ks + kAhead);
            if ((ks + 1) * kParts / KD > ks * kParts / KD) {
                const int i = ks * kParts / KD, row = mine;
                if (i + 1 < kParts) mine = part_row(i + 1);
                stage(buf ^ 1, i, row);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- softmax against the rows' references ----
        if constexpr (FP8) {
            const v4f s4 = *reinterpret_cast<const v4f*>(smem + L::kScale + 256 * buf + 4 * (16 * kq + 4 * (ln >> 4)));
#pragma unroll
            for (int e = 0; e < 4; ++e) ks4[e] = s4[e];
            S *= s4;
        }
        S = scaled_scores(S, scale);
        if (here != ~0ull) {
            const uint32_t mine = FP8 ? (uint32_t)(here >> (32 * (kq >> 1) + (kq & 1))) >> (8 * (ln >> 4))
                                      : (uint32_t)(here >> (16 * kq)) >> (4 * (ln >> 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) S[e] = mine >> (FP8 ? 2 * e : e) & 1 ? S[e] : -__builtin_inff();
        }
        const bool rise = highest() > own_m() + (kSlack - shift);
        write_p();
        if (wave_ballot(rise) && lane == 0) flag[buf] = 1;
        if (threadIdx.x == 0) flag[buf ^ 1] = 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) W[i] = read_v(buf, i);
        tile_barrier();
        const int risen = flag[buf];
        read_p(0);
        if (uniform(risen)) rebase();
        l += sum;

        // ---- O^T += V^T P^T; beside it the rows of the tile behind the next one, and the
        //      hand-over: every wave has read its last operands, and the next tile is there ----
#pragma unroll
        for (int i = 0; i < 2 * CT; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            const v8bf w = W[i % kAhead].get();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                O[i % CT][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, P[mt], O[i % CT][mt], 0, 0, 0);
            if (i == CT - 1) read_p(1);
            if (i + kAhead < 2 * CT) W[i % kAhead] = read_v(buf, i + kAhead);
            if (i == 1) {
                keys.resolve(t_now + 1 < t1 ? keys.entry_of(t_now + 1, ahead.s2) : -1, ahead.page2);
                address();
            }
            if (i == 2 * CT - kAhead) {
                __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
                store_scale(buf ^ 1);
                tile_barrier();
            }
            if (i >= 2 * CT - kAhead) K[i - (2 * CT - kAhead)] = read_k(buf ^ 1, i - (2 * CT - kAhead));
        }
        __builtin_amdgcn_sched_barrier(0);
        here = next;
        buf ^= 1;
        t = t_now;
        t_next = t_now + 1;
        ahead = LatentAhead{ahead.s3, page3, s4};
        if (keys.mask == 0 && t_next < t1) {
            t_next = keys.seek(t_next + 1, ahead);
            address();
        }
    }

    // ---- join the waves' sums, write ----
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no copy may still be in flight
    tile_barrier();
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
    if (g == 0) red[kq * 16 * MT + 16 * mq + n] = l;
    tile_barrier();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) x += red[w * 16 * MT + 16 * mt + n];
        if (16 * mt + n >= nrows) continue;
        const int64_t r = keys.r0 + 16 * mt + n;
        if (p.slots == 1) {
            const float inv = x == 0.f ? 0.f : 1.f / x;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const v4f o = O[ct][mt] * inv;
                *reinterpret_cast<uint2*>(a.out + r * kV + 16 * CT * wave + 16 * ct + 4 * g) =
                    uint2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
            }
            if (a.lse && wave == 0 && g == 0)
                a.lse[r] = x == 0.f ? -__builtin_inff() : (m[mt] + log2f(x)) * 0.693147180559945f;
        } else {
            const int64_t at = (int64_t)keys.slot * total + r;
            if (x != 0.f)   // (NaN too)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    *reinterpret_cast<v4f*>(p.part_o + at * kV + 16 * CT * wave + 16 * ct + 4 * g) = O[ct][mt];
            if (wave == 0 && g == 0) p.part_ml[at] = float2{m[mt], x};
        }
    }
}

// Joins the slots' partial results, W waves to a row: each takes every W-th
// slot, 8 columns a lane, and the waves' sums meet in LDS.  Slots are at most
// 64, one per lane for the weights.  Bound by reading the partial sums; with
// few rows by latency, so a wave has four slots in flight.  8192 rows of 4
// slots (67 MB): 13.0 us with one wave a row, 19.7 with four; 16 rows of 32
// slots: 6.6 and 3.9; 1320 rows of 13 slots (36 MB): 7.5 and 6.9.
template <int W>
__global__ void __launch_bounds__(kJoinThreads)
latent_join_kernel(LatentArgs a, LatentPlan p) {
    __shared__ float sums[W == 1 ? 1 : 4][kV];
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int total = a.T * a.H;
    const int64_t r = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (W == 1 && r >= total) return;
    const float2 ml = lane < p.slots ? p.part_ml[(int64_t)lane * total + r] : float2{0.f, 0.f};
    const bool some = ml.y != 0.f;
    float top = some ? ml.x : -__builtin_inff();
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    const float w = some ? __builtin_amdgcn_exp2f(ml.x - top) : 0.f;
    float l = w * ml.y;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) l += __shfl_xor(l, d, kWave);
    const uint64_t filled = wave_ballot(some);
    const int any = filled ? __builtin_ctzll(filled) : 0;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.f;
    if (filled)
        for (int s0 = W == 1 ? 0 : wave; s0 < p.slots; s0 += 4 * W) {
            v4f x[4], y[4];
            float f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {   // a slot that holds nothing was not written: another's place, weight 0
                const int s = s0 + W * u < p.slots ? s0 + W * u : any;
                const bool ok = s0 + W * u < p.slots && filled >> s & 1;
                f[u] = ok ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), s)) : 0.f;
                const float* at = p.part_o + ((int64_t)(ok ? s : any) * total + r) * kV + 8 * lane;
                x[u] = *reinterpret_cast<const v4f*>(at);
                y[u] = *reinterpret_cast<const v4f*>(at + 4);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[j] += f[u] * x[u][j];
                    o[4 + j] += f[u] * y[u][j];
                }
        }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    if constexpr (W == 1) {
        v4i out;
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = (int)pack_bf16(o[2 * j] * inv, o[2 * j + 1] * inv);
        *reinterpret_cast<v4i*>(a.out + r * kV + 8 * lane) = out;
        if (a.lse && lane == 0) a.lse[r] = l != 0.f ? (top + log2f(l)) * 0.693147180559945f : -__builtin_inff();
    } else {
        *reinterpret_cast<v4f*>(&sums[wave][8 * lane]) = v4f{o[0], o[1], o[2], o[3]};
        *reinterpret_cast<v4f*>(&sums[wave][8 * lane + 4]) = v4f{o[4], o[5], o[6], o[7]};
        __syncthreads();
        const int c = 2 * threadIdx.x;
        v2bf out;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            out[j] = (__bf16)(((sums[0][c + j] + sums[1][c + j]) + (sums[2][c + j] + sums[3][c + j])) * inv);
        *reinterpret_cast<v2bf*>(a.out + r * kV + c) = out;
        if (a.lse && threadIdx.x == 0) a.lse[r] = l != 0.f ? (top + log2f(l)) * 0.693147180559945f : -__builtin_inff();
    }
}

constexpr int kCUs = 256;
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
int pad8(int n) { return (n + 7) / 8 * 8; }

// Query rows of a workgroup: the smallest block that holds all of them, at
// most 128.  1000 queries, 2048 selected rows of 576 (bf16 / fp8), in us a call,
// calls in a row:
//   32 heads: blocks of 16: 422 / 427, of 32: 229 / 242, of 64: 272 / 344
//   64 heads: of 32: 493 / 516, of 64: 319 / 397, of 128: 377 / 457
//   128 heads: of 64: 622 / 787, of 128: 542 / 589 (on another card 552 / 587)
int block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// Time of a 64-key tile in a block of that many rows, on a busy GPU and not
// bound by memory.
double tile_us(int rows) { return rows == 16 ? 1.4 : rows == 32 ? 1.9 : rows == 64 ? 2.6 : 4.2; }

// Threads of a workgroup (launch_latent_attention), and of the largest launch.
int plan_threads(int rows) { return rows == 16 ? 64 * waves_of(1) : 512; }
constexpr int64_t kMaxThreads = (1ll << 32) - 1;

// Splits of the key tiles that finish first, in us (p.rows and the tile counts
// are given); 1e30 where every one passes a launch's threads.  A workgroup takes 5 and its tiles, own ones longer the more CUs
// stream 74 KB (fp8: 37) a tile of their own; the GPU runs one workgroup per
// CU, prefix parts first; joining takes 4 and reads and writes every slot's
// sums.  A run of own tiles takes as long as one of the prefix.  64 queries of
// 16 heads, 2048 selected: 2 splits 45.6 us, 4 (chosen) 36.
// Counts tried: each up to 8, then steps of a seventh to a quarter.  The times are
// rough, and a finer list gives the rule more near-ties to lose: with 20 counts 64
// queries of 16 heads on a prefix of 32768 took 30 parts for 28, 109 us for 91.
double split(int64_t blocks_p, int tiles_p, int64_t blocks_o, int tiles_o, int64_t rows, int H, bool fp8,
             LatentPlan& p) {
    static const int kSplits[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32};
    const double tile = tile_us(p.rows), tile_o = tile_us(block_rows(H < p.rows ? H : p.rows));
    const int tiles = tiles_p > 0 ? tiles_p : tiles_o;
    double best = 1e30;
    for (int n : kSplits) {
        if (n > 1 && n > tiles) break;
        const int len = ceil_div(tiles, n);
        const int sp = tiles_p > 0 ? ceil_div(tiles_p, len) : 0;
        int lo = tiles_p > 0 ? (int)(len * tile / tile_o) : len;
        if (lo > tiles_o) lo = tiles_o;
        if (lo < ceil_div(tiles_o, 32)) lo = ceil_div(tiles_o, 32);
        const int so = tiles_o > 0 ? ceil_div(tiles_o, lo) : 0;
        const int64_t np = blocks_p * sp, no = blocks_o * so;
        if ((np + no + 14) * plan_threads(p.rows) > kMaxThreads) continue;   // (14: both rounded up to 8s)
        const double full = (fp8 ? 1.8 : 3.6) - tile_o;   // more per tile with every CU streaming
        const double cp = 5 + tile * len, co = 5 + (tile_o + (full > 0 ? full : 0) * (double)(no < kCUs ? no : kCUs) / kCUs) * lo;
        // whole rounds of prefix parts; the rest of them beside the own parts
        const int64_t rest = np % kCUs;
        int64_t k = no / kCUs;   // own parts one after another on a CU
        auto room = [&](int64_t k) {
            const int64_t behind = k * co > cp ? (int64_t)((k * co - cp) / co) : 0;
            return (kCUs - rest) * k + rest * behind;
        };
        while (room(k) < no) ++k;
        double us = k * co;
        if (rest > 0 && us < cp) us = cp;
        us += (double)(np / kCUs) * cp;
        const int slots = sp + so;
        if (slots > 1) us += 4 + 1e-3 * (double)rows * slots;
        if (us < best) {
            best = us;
            p.sp = sp;
            p.so = so;
            p.lp = len;
            p.lo = lo;
        }
    }
    return best;
}

LatentPlan make_plan(int T, int H, bool topk, int K, int prefix_len, int max_ctx, bool fp8) {
    const int tiles_p = topk ? 0 : ceil_div(prefix_len, kTile);
    const int tiles_o = ceil_div(topk ? K : max_ctx, kTile);
    const int64_t rows = (int64_t)T * H;
    // every query walks all its keys (none: one workgroup a row block writes that)
    LatentPlan p{};
    p.rows = block_rows(H);
    p.hb = ceil_div(H, p.rows);
    p.joint = tiles_p > 0;
    const int all = tiles_p + tiles_o;
    // (in one part it is T workgroups, which fit a launch for all T * H <= 2^23)
    const double us = split(0, 0, (int64_t)T * p.hb, all > 0 ? all : 1, rows, H, fp8, p);
    if (tiles_p > 0) {   // or the prefix is walked once for the stacked rows
        LatentPlan s{};
        s.rows = block_rows(rows);
        s.hb = ceil_div(H, s.rows);
        s.rb = ceil_div(rows, s.rows);
        if (split(s.rb, tiles_p, tiles_o > 0 ? (int64_t)T * s.hb : 0, tiles_o, rows, H, fp8, s) < us) p = s;
    }
    p.n_prefix = pad8(p.rb * p.sp);
    p.n_own = pad8(T * p.hb * p.so);
    p.slots = p.sp + p.so;
    return p;
}

size_t plan_bytes(const LatentPlan& p, int T, int H) {
    return p.slots == 1 ? 0 : (size_t)p.slots * T * H * (kV + 2) * sizeof(float);
}

template <int KD, int MT, bool TOPK, bool FP8>
hipError_t run(const LatentArgs& a, const LatentPlan& p, hipStream_t stream) {
    static PerDevice<int> once;
    constexpr int lds = Lds<KD, MT, FP8>::kBytes;
    const hipError_t e = set_lds_limit(once, (const void*)latent_attention_kernel<KD, MT, TOPK, FP8>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((latent_attention_kernel<KD, MT, TOPK, FP8>), dim3((unsigned)(p.n_prefix + p.n_own)),
                       dim3(64 * waves_of(MT)), lds, stream, a, p);
    return hipGetLastError();
}

template <int KD, int MT>
hipError_t run(const LatentArgs& a, const LatentPlan& p, bool fp8, hipStream_t stream) {
    if (a.idx) return fp8 ? run<KD, MT, true, true>(a, p, stream) : run<KD, MT, true, false>(a, p, stream);
    return fp8 ? run<KD, MT, false, true>(a, p, stream) : run<KD, MT, false, false>(a, p, stream);
}

template <int KD>
hipError_t run(const LatentArgs& a, const LatentPlan& p, bool fp8, hipStream_t stream) {
    return p.rows == 16 ? run<KD, 1>(a, p, fp8, stream) : run<KD, 2>(a, p, fp8, stream);
}

}  // namespace

// The caller's workspace holds the partial sums, then the (maximum, sum) pairs.
size_t latent_topk_workspace_bytes(int T, int H, int K, bool fp8) {
    return plan_bytes(make_plan(T, H, true, K, 0, 0, fp8), T, H);
}
size_t latent_shared_workspace_bytes(int B, int H, int prefix_len, int max_ctx, bool fp8) {
    return plan_bytes(make_plan(B, H, false, 0, prefix_len, max_ctx, fp8), B, H);
}

hipError_t launch_latent_attention(const LatentArgs& a, bool fp8, hipStream_t stream) {
    LatentPlan p = make_plan(a.T, a.H, a.idx != nullptr, a.K, a.prefix_len, a.max_ctx, fp8);
    p.part_o = reinterpret_cast<float*>(a.workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)p.slots * a.T * a.H * kV);
    hipError_t e = p.rows >= 64 ? launch_latent_rows(a, p, fp8, stream) : a.E == 576 ? run<18>(a, p, fp8, stream) : run<16>(a, p, fp8, stream);
    if (e != hipSuccess || p.slots == 1) return e;
    const int rows = a.T * a.H;
    if (rows >= kJoinRows)
        hipLaunchKernelGGL(latent_join_kernel<1>, dim3((unsigned)ceil_div(rows, 4)), dim3(kJoinThreads), 0, stream, a, p);
    else
        hipLaunchKernelGGL(latent_join_kernel<4>, dim3((unsigned)rows), dim3(kJoinThreads), 0, stream, a, p);
    return hipGetLastError();
}

}  // namespace dsaidx
