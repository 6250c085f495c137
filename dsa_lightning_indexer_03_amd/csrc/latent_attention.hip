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
// One workgroup of four waves takes a block of up to 16*MT query rows (a
// query's heads, or the stacked heads of several queries for the shared
// prefix) and a run of 64-key tiles.  A tile is staged once in LDS and serves
// both products:
//   S^T (16 keys x rows) = K Q^T: wave w has keys 16w .. 16w+15, the queries
//     sit in its registers;
//   O^T (128 columns x rows) += V^T P^T: wave w has columns 128w .. 128w+127,
//     the probabilities of all 64 keys come through LDS as bf16, the values
//     are read transposed from the same tile.
// Both leave a lane with one query row (lane % 16 of each 16-row block), so
// the softmax's factors are per lane.  The exponent's reference m is common to
// the four waves and only moves when a score exceeds it by more than
// 2^kSlack (base 2): a flag in LDS, read behind the barrier that the exchange of P needs
// anyway, sends all waves through a second pass that takes the tile's maximum,
// rescales and rewrites P.  Sums are fp32; P is rounded to bf16 (the second
// product's operand; its sum is taken before the rounding).
// When the rows alone do not fill the GPU the key tiles are split over
// workgroups, whose fp32 partial sums a second kernel joins by their maxima.
#include "common.h"
#include "device_once.h"
#include "kernels.h"

namespace dsaidx {
namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kPage = 64;
constexpr int kTile = 64;      // keys of a tile
constexpr int kThreads = 256;
constexpr int kV = 512;
constexpr float kSlack = 16.f;
constexpr int kAhead = 3;      // operand reads in flight

// LDS: two tiles, P, the exchange of maxima and sums, flags.  The 64 banks
// serve 16 lanes of a 16-byte read at once (lanes 0-3, 12-15 and 20-27 are one
// such group, 4-11, 16-19 and 28-31 the next), 32 lanes of an 8-byte one.  A
// tile's row is its 512 value columns padded by 32 bytes: consecutive rows
// start 8 banks apart, and both an operand read (16 rows, lane groups 16 bytes
// apart) and a transposed one (8 rows of 32 bytes) use every bank once: 235
// bytes a clock and CU against 127 with a padding of 16.  P's rows are padded
// alike.  The rotary columns lie behind, 128 bytes a row, their 16-byte pieces
// permuted within the row.
constexpr int kRowB = 2 * kV + 32;
constexpr int kPRowB = 2 * kTile + 32;
constexpr int kMainB = kTile * kRowB;
constexpr int kRopeB = kTile * 128;
constexpr int kTileB = kMainB + kRopeB;
constexpr int kPOff = 2 * kTileB;
__host__ __device__ constexpr int p_bytes(int mt) { return mt * 16 * kPRowB; }
__host__ __device__ constexpr int red_off(int mt) { return kPOff + p_bytes(mt); }   // [4][16 mt] floats
__host__ __device__ constexpr int scale_off(int mt) { return red_off(mt) + 4 * 16 * mt * 4; }  // [2][64] floats
__host__ __device__ constexpr int flag_off(int mt) { return scale_off(mt) + 512; }
__host__ __device__ constexpr int lds_bytes(int mt) { return flag_off(mt) + 16; }
static_assert(lds_bytes(4) <= 160 * 1024, "LDS budget");

// What an entry without a row is copied from.
__device__ __align__(16) const unsigned char kZeroRow[1152] = {};

struct Plan {
    int n_prefix, n_own;   // workgroups of each part (multiples of 8)
    int rb;                // prefix: row blocks of all T * H rows
    int sp, lp;            // prefix: splits, tiles of a split
    int hb;                // own rows or selection: row blocks of one query's H rows
    int so, lo;            //   splits, tiles of a split
    int slots;             // partial results per row (1: written directly)
    float* part_o;         // [slots][T * H][V]
    float2* part_ml;       // [slots][T * H] (maximum, sum)
};

__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 16 bytes per lane from base + off (off per lane) straight to LDS byte
// address lds + 16 * lane.  Written as asm so that later LDS reads of the
// other tile do not wait for it; it has no register result, and the kernel
// waits for vmcnt itself before the tile is read.  The base often comes from a
// lane read: the scalar move in between makes it safe to address with at once,
// and is the wait state that M0 needs.
__device__ __forceinline__ void copy_to_lds(const void* base, uint32_t off, uint32_t lds) {
    uint64_t b;
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
                 : "=&s"(b) : "s"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void copy_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}

// Eight E4M3 codes -> eight bf16 (exact).
__device__ __forceinline__ v4i widen8(uint2 c) {
    return v4i{(int)fp8x2_to_bf16x2<false>((int)c.x), (int)fp8x2_to_bf16x2<true>((int)c.x),
               (int)fp8x2_to_bf16x2<false>((int)c.y), (int)fp8x2_to_bf16x2<true>((int)c.y)};
}

template <int KD, int MT, bool TOPK, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
latent_attention_kernel(LatentArgs a, Plan p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int E = 32 * KD;
    constexpr int RB = FP8 ? E : 2 * E;   // bytes of a cached row
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int n = lane & 15, g = lane >> 4;
    const int total = a.T * a.H;

    // ---- which rows, which keys ----
    // Workgroups go to the 8 XCDs in turn; the ones that read the same keys
    // follow each other on one XCD.
    int r0, nrows, t0, t1, slot, len;
    const int32_t* table;
    const int32_t* idx = nullptr;
    {
        const int id = blockIdx.x;
        if (!TOPK && id < p.n_prefix) {
            const int w = (id & 7) * (p.n_prefix >> 3) + (id >> 3);
            slot = w / p.rb;
            if (slot >= p.sp) return;
            r0 = (w % p.rb) * 16 * MT;
            nrows = min(16 * MT, total - r0);
            len = a.prefix_len;
            table = a.prefix_table;
            t0 = slot * p.lp;
            t1 = min(t0 + p.lp, (len + kTile - 1) / kTile);
        } else {
            const int id2 = id - p.n_prefix;
            const int w = (id2 & 7) * (p.n_own >> 3) + (id2 >> 3);
            const int q = w / (p.hb * p.so), s = w / p.hb % p.so, h = w % p.hb * 16 * MT;
            if (q >= a.T) return;
            r0 = q * a.H + h;
            nrows = min(16 * MT, a.H - h);
            slot = p.sp + s;
            t0 = s * p.lo;
            if constexpr (TOPK) {
                const int b = a.seq_ids ? a.seq_ids[q] : q;
                const bool ok = b >= 0 && b < a.B;
                table = a.block_table + (int64_t)(ok ? b : 0) * a.max_pages;
                idx = a.idx + (int64_t)q * a.K;
                len = ok ? a.K : 0;
            } else {
                table = a.block_table + (int64_t)q * a.max_pages;
                len = min(max(a.context_lens[q], 0), a.max_ctx);
            }
            t1 = min(t0 + p.lo, (len + kTile - 1) / kTile);
        }
    }

    // ---- queries: copied to the second tile's place in a tile's layout ----
    const int kb = 16 * wave;   // this wave's rows of a tile
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
    {
        const uint16_t* q = a.q + (int64_t)r0 * E;
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i) {
            const int r = 4 * MT * wave + i;
            copy_to_lds(q + (int64_t)min(r, nrows - 1) * E, 16 * lane, lds0 + kTileB + r * kRowB);
        }
        if constexpr (KD > 16)
#pragma unroll
            for (int j = 0; j < (MT + 1) / 2; ++j) {
                const int r8 = 8 * (wave + 4 * j);
                if (r8 < 16 * MT) {
                    const int r = r8 + (lane >> 3);
                    copy_to_lds(q + (int64_t)min(r, nrows - 1) * E + kV + 8 * ((lane & 7) ^ ((r >> 1) & 7)),
                                lds0 + kTileB + kMainB + r8 * 128);
                }
            }
    }
    v4f O[8][MT];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -__builtin_inff();
        l[mt] = 0.f;
#pragma unroll
        for (int ct = 0; ct < 8; ++ct) O[ct][mt] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    int* flag = reinterpret_cast<int*>(smem + flag_off(MT));
    float* red = reinterpret_cast<float*>(smem + red_off(MT));
    if (threadIdx.x < 2) flag[threadIdx.x] = 0;

    // ---- the rows of a tile: lane i holds entry i's row of the pool ----
    auto entry = [&](int t) -> int {   // position (topk) of entry `lane`, -1: none
        const int j = t * kTile + lane;
        if constexpr (TOPK) return j < len ? idx[j] : -1;
        return j < len ? j : -1;
    };
    auto page_of = [&](int s) -> int {
        return s >= 0 && s / kPage < a.max_pages ? table[s / kPage] : -1;
    };
    int zero;   // keeps the loads of page ids among the vector loads
    asm volatile("v_mov_b32 %0, 0" : "=v"(zero));
    auto page_of_tile = [&](int s, int t) -> int {
        if constexpr (TOPK) return page_of(s);
        return t < t1 ? table[t + zero] : -1;
    };
    auto live = [&](int s, int page) { return s >= 0 && page >= 0 && page < a.num_pages; };

    // While a tile is computed the next one is copied, the addresses of the one
    // behind it are made, and page ids and entries of the next two are loads in
    // flight.  An entry without a row takes a row of zeros: its probability is
    // zero, and zero its values must be.
    int row = 0;                      // the next tile: rows,
    uint64_t mask = 0;                // which entries have one,
    uint64_t src = 0;                 // their addresses,
    uint64_t rope_src[2] = {0, 0};    // and this lane's pieces of the rotary columns
    int s2, page2, s3;                // entries and page ids of the tile behind it, entries of the next
    auto address = [&](int r) {
        return r >= 0 ? (uint64_t)a.cache + (uint64_t)(uint32_t)r * RB : (uint64_t)kZeroRow;
    };
    auto resolve = [&](int s, int page) {
        const bool ok = live(s, page);
        mask = wave_ballot(ok);
        row = ok ? page * kPage + (s & (kPage - 1)) : -1;
        src = address(row);
        if constexpr (KD > 16)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = kb + 8 * j + (lane >> 3);
                rope_src[j] = address(__shfl(row, r)) + (RB / E) * (kV + 8 * ((lane & 7) ^ ((r >> 1) & 7)));
            }
    };
    // First tile at or behind t with an entry, resolved, and the loads behind it.
    auto seek = [&](int t) -> int {
        for (; t < t1; ++t) {
            const int s = entry(t);
            resolve(s, page_of_tile(s, t));
            if (mask) break;
        }
        if (t >= t1) {
            resolve(-1, -1);
            return t1;
        }
        s2 = entry(t + 1);
        s3 = entry(t + 2);
        page2 = page_of_tile(s2, t + 1);
        return t;
    };

    uint2 main8[FP8 ? 16 : 1], rope8[FP8 ? 2 : 1];
    float kscale = 0.f;
    // Part i of a tile's copy: row kb + i, then (i = 16, 17) 8 rows' rotary columns.
    auto stage = [&](int buf, int i) {
        const uint32_t lds = lds0 + buf * kTileB;
        if (i < 16) {
            const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)src, kb + i);
            const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(src >> 32), kb + i);
            const unsigned char* from = reinterpret_cast<const unsigned char*>((uint64_t)hi << 32 | lo);
            if constexpr (FP8) main8[i] = *reinterpret_cast<const uint2*>(from + 8 * lane);
            else copy_to_lds(from, 16 * lane, lds + (kb + i) * kRowB);
        } else {
            if constexpr (FP8) rope8[i - 16] = *reinterpret_cast<const uint2*>(rope_src[i - 16]);
            else
                copy_to_lds(reinterpret_cast<const void*>(rope_src[i - 16]),
                            lds + kMainB + (kb + 8 * (i - 16)) * 128);
        }
    };
    // fp8 rows: widened on their way into the tile
    auto stage_store = [&](int buf) {
        if constexpr (FP8) {
            unsigned char* dst = smem + buf * kTileB;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                *reinterpret_cast<v4i*>(dst + (kb + r) * kRowB + 16 * lane) = widen8(main8[r]);
            if constexpr (KD > 16)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<v4i*>(dst + kMainB + (kb + 8 * j) * 128 + 16 * lane) = widen8(rope8[j]);
            if ((lane >> 4) == wave) reinterpret_cast<float*>(smem + scale_off(MT))[64 * buf + lane] = kscale;
        }
    };

    int t = seek(t0);
    uint64_t here = mask;   // the entries of the tile that is computed
    auto stage_scale = [&]() {
        if constexpr (FP8) kscale = row >= 0 ? a.cache_scale[row] : 0.f;
    };
#pragma unroll
    for (int i = 0; i < KD; ++i) stage(0, i);
    stage_scale();
    stage_store(0);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    lds_barrier();
    // B operand of 16 rows x 32 columns: row n, columns 8g .. 8g+7 of each 32
    v8bf Q[MT][KD];
    auto operand = [&](const unsigned char* tile, int r, int ks) {   // row r: r % 16 == n
        return *reinterpret_cast<const v8bf*>(
            tile + (ks < 16 ? r * kRowB + 16 * g + 64 * ks
                            : kMainB + r * 128 + 16 * ((4 * (ks - 16) + g) ^ ((n >> 1) & 7))));
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            v8bf q = operand(smem + kTileB, 16 * mt + n, ks);
            if (a.scale_log2 < 0.f) {   // the products then take the scale's magnitude
                v4i u = __builtin_bit_cast(v4i, q);
                u ^= (int)0x80008000;
                q = __builtin_bit_cast(v8bf, u);
            }
            Q[mt][ks] = q;
        }
    // 64 rows' queries fill most of the accumulation registers, which an
    // operand may be read from as well
    if constexpr (MT == 4)
#pragma unroll
        for (int i = 0; i < MT * KD && i < 60; ++i) asm volatile("" : "+a"(Q[i / KD][i % KD]));
    // (never 0: a score of -inf, an entry without a row, has to stay one)
    const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);

    int t_next = t1, buf = 0;
    if (t < t1) {
        if (t + 1 < t1) {
            resolve(s2, page2);
            if (mask == 0) {
                t_next = seek(t + 2);
            } else {
                t_next = t + 1;
                s2 = s3;
                page2 = page_of_tile(s2, t + 2);
                s3 = entry(t + 3);
            }
        } else {
            resolve(-1, -1);
        }
    }
    while (t < t1) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the tile
        lds_barrier();
        const uint32_t live4 = (uint32_t)(here >> (kb + 4 * g)) & 15u;
        // loads for the tiles behind the next one
        const int page3 = page_of_tile(s3, t_next + 2);
        const int s4 = entry(t_next + 3);
        stage_scale();

        const unsigned char* tile = smem + buf * kTileB;
        // ---- scores: S^T, keys 4g .. 4g+3 of this wave's 16, row n of each block ----
        v4f S[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) S[mt] = v4f{0.f, 0.f, 0.f, 0.f};
        {
            v8bf K[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) K[i] = operand(tile, kb + n, i);
#pragma unroll
            for (int ks = 0; ks < KD; ++ks) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    S[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(K[ks % kAhead], Q[mt][ks], S[mt], 0, 0, 0);
                if (ks + kAhead < KD) K[ks % kAhead] = operand(tile, kb + n, ks + kAhead);
                stage(buf ^ 1, ks);   // behind the last tile: zeros that nobody reads
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // ---- softmax against the common reference ----
        float ks4[4] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (FP8) {
            const v4f s4 = *reinterpret_cast<const v4f*>(smem + scale_off(MT) + 256 * buf + 4 * (kb + 4 * g));
#pragma unroll
            for (int i = 0; i < 4; ++i) ks4[i] = s4[i];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[mt][i] *= ks4[i];
        }
        if (here != ~0ull)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[mt][i] = live4 >> i & 1 ? S[mt][i] : -__builtin_inff();
        float top[MT], sum[MT];
        bool rise = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            top[mt] = scale * fmaxf(fmaxf(S[mt][0], S[mt][1]), fmaxf(S[mt][2], S[mt][3]));
            rise |= top[mt] > m[mt] + kSlack;
        }
        auto write_p = [&]() {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float ref = m[mt] == -__builtin_inff() ? 0.f : m[mt];
                float pr[4];
                sum[mt] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pr[i] = __builtin_amdgcn_exp2f(fmaf(S[mt][i], scale, -ref));
                    sum[mt] += pr[i];
                    if (FP8) pr[i] *= ks4[i];
                }
                // P[row][key]: 16-byte piece 4(w/2) + g holds the keys 4g .. 4g+3 of waves
                // 2(w/2) and 2(w/2) + 1
                const v2bf lo = v2bf{(__bf16)pr[0], (__bf16)pr[1]}, hi = v2bf{(__bf16)pr[2], (__bf16)pr[3]};
                *reinterpret_cast<uint2*>(smem + kPOff + (16 * mt + n) * kPRowB + 16 * (4 * (wave >> 1) + g) +
                                          8 * (wave & 1)) =
                    uint2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
            }
        };
        write_p();
        if (wave_ballot(rise) && lane == 0) flag[buf] = 1;
        if (threadIdx.x == 0) flag[buf ^ 1] = 0;
        // the values: columns 16ct .. 16ct+15 of keys 4g .. 4g+3 of two 16-key groups; step i: ct = i / 2, kk = i % 2
        const unsigned char* vp = tile + (4 * g + (n >> 2)) * kRowB + 8 * (n & 3) + 256 * wave;
        auto read_v = [&](int i) {
            const unsigned char* at = vp + 32 * (i >> 1) + 32 * (i & 1) * kRowB;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 16 * kRowB));
            return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        v8bf P[MT][2], W[kAhead];
        auto read_p = [&]() {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    P[mt][kk] = *reinterpret_cast<const v8bf*>(smem + kPOff + (16 * mt + n) * kPRowB +
                                                               16 * (4 * kk + g));
        };
        lds_barrier();
        const int risen = flag[buf];
        read_p();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) W[i] = read_v(i);
        if (uniform(risen)) {
            // the reference moves to the tile's maximum where that is above it
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x = top[mt];
                x = fmaxf(x, __shfl_xor(x, 16, kWave));
                x = fmaxf(x, __shfl_xor(x, 32, kWave));
                if (g == 0) red[wave * 16 * MT + 16 * mt + n] = x;
            }
            lds_barrier();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x = m[mt];
#pragma unroll
                for (int w = 0; w < 4; ++w) x = fmaxf(x, red[w * 16 * MT + 16 * mt + n]);
                const float f = m[mt] == x ? 1.f : __builtin_amdgcn_exp2f(m[mt] - x);
                m[mt] = x;
                l[mt] *= f;
#pragma unroll
                for (int ct = 0; ct < 8; ++ct) O[ct][mt] *= f;
            }
            write_p();
            lds_barrier();
            read_p();
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) l[mt] += sum[mt];

        // ---- O^T += V^T P^T; beside it, the addresses of the tile behind the next one ----
        const int t_now = t_next;
        here = mask;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                O[i >> 1][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(W[i % kAhead], P[mt][i & 1], O[i >> 1][mt], 0, 0, 0);
            if (i + kAhead < 16) W[i % kAhead] = read_v(i + kAhead);
            if (i == 2) {
                if (t_now + 1 >= t1) s2 = -1;
                resolve(s2, page2);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        stage_store(buf ^ 1);
        buf ^= 1;
        t = t_now;
        t_next = t_now + 1;
        s2 = s3;
        page2 = page3;
        s3 = s4;
        if (mask == 0 && t_next < t1) t_next = seek(t_next + 1);
    }

    // ---- join the waves' sums, write ----
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no copy may still be in flight
    lds_barrier();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x = l[mt];
        x += __shfl_xor(x, 16, kWave);
        x += __shfl_xor(x, 32, kWave);
        if (g == 0) red[wave * 16 * MT + 16 * mt + n] = x;
    }
    lds_barrier();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) x += red[w * 16 * MT + 16 * mt + n];
        if (16 * mt + n >= nrows) continue;
        const int64_t r = r0 + 16 * mt + n;
        if (p.slots == 1) {
            const float inv = x > 0.f ? 1.f / x : 0.f;
#pragma unroll
            for (int ct = 0; ct < 8; ++ct) {
                const v4f o = O[ct][mt] * inv;
                const v2bf lo = v2bf{(__bf16)o[0], (__bf16)o[1]}, hi = v2bf{(__bf16)o[2], (__bf16)o[3]};
                *reinterpret_cast<uint2*>(a.out + r * kV + 128 * wave + 16 * ct + 4 * g) =
                    uint2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
            }
            if (a.lse && wave == 0 && g == 0)
                a.lse[r] = x > 0.f ? (m[mt] + log2f(x)) * 0.693147180559945f : -__builtin_inff();
        } else {
            const int64_t at = (int64_t)slot * total + r;
            if (x != 0.f)   // (NaN too)
#pragma unroll
                for (int ct = 0; ct < 8; ++ct)
                    *reinterpret_cast<v4f*>(p.part_o + at * kV + 128 * wave + 16 * ct + 4 * g) = O[ct][mt];
            if (wave == 0 && g == 0) p.part_ml[at] = float2{m[mt], x};
        }
    }
}

// Joins the slots' partial results of a row: one workgroup per row, a wave
// takes every fourth slot (8 columns a lane), the waves' sums meet in LDS.
// Slots are at most 64, one per lane for the weights.  Bound by reading the
// partial sums; with few rows by latency, so a wave has four slots in flight.
__global__ void __launch_bounds__(kThreads)
latent_join_kernel(LatentArgs a, Plan p) {
    __shared__ float sums[4][kV];
    const int wave = uniform((int)threadIdx.x >> 6), lane = lane_id();
    const int total = a.T * a.H;
    const int64_t r = blockIdx.x;
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
        for (int s0 = wave; s0 < p.slots; s0 += 16) {
            v4f x[4], y[4];
            float f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {   // a slot that holds nothing was not written: another's place, weight 0
                const int s = s0 + 4 * u < p.slots ? s0 + 4 * u : any;
                const bool ok = s0 + 4 * u < p.slots && filled >> s & 1;
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
    *reinterpret_cast<v4f*>(&sums[wave][8 * lane]) = v4f{o[0], o[1], o[2], o[3]};
    *reinterpret_cast<v4f*>(&sums[wave][8 * lane + 4]) = v4f{o[4], o[5], o[6], o[7]};
    __syncthreads();
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int c = 2 * threadIdx.x;
    v2bf out;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        out[j] = (__bf16)(((sums[0][c + j] + sums[1][c + j]) + (sums[2][c + j] + sums[3][c + j])) * inv);
    *reinterpret_cast<v2bf*>(a.out + r * kV + c) = out;
    if (a.lse && threadIdx.x == 0) a.lse[r] = l != 0.f ? (top + log2f(l)) * 0.693147180559945f : -__builtin_inff();
}

constexpr int kCUs = 256;
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
int pad8(int n) { return (n + 7) / 8 * 8; }

// Row blocks of 64 where the rows fill them; fp8 tiles pass through registers,
// which leaves room for 32.
int blocks_of_16(int64_t rows, bool fp8) { return rows <= 16 ? 1 : rows <= 32 || fp8 ? 2 : 4; }

// Splits that finish first, in us: a workgroup takes 5 and 1.4 a tile, the GPU
// runs one per CU, prefix parts first; joining takes 4 and reads and writes
// every slot's sums.  A run of own tiles is as long as one of the prefix.
void split(int tiles_p, int64_t blocks_o, int tiles_o, int64_t rows, Plan& p) {
    static const int kSplits[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32};
    const int tiles = tiles_p > 0 ? tiles_p : tiles_o;
    double best = 1e30;
    for (int n : kSplits) {
        if (n > tiles) break;
        const int len = ceil_div(tiles, n);
        const int sp = tiles_p > 0 ? ceil_div(tiles_p, len) : 0;
        int lo = tiles_p > 0 ? (len < tiles_o ? len : tiles_o) : len;
        if (lo < ceil_div(tiles_o, 32)) lo = ceil_div(tiles_o, 32);
        const int so = tiles_o > 0 ? ceil_div(tiles_o, lo) : 0;
        const int64_t np = tiles_p > 0 ? (int64_t)p.rb * sp : 0, no = blocks_o * so;
        const double cp = 5 + 1.4 * len, co = 5 + 1.4 * lo;
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
}

Plan make_plan(int T, int H, bool topk, int K, int prefix_len, int max_ctx, bool fp8, int* mt) {
    Plan p{};
    const int tiles_p = topk ? 0 : ceil_div(prefix_len, kTile);
    int tiles_o = ceil_div(topk ? K : max_ctx, kTile);
    if (tiles_p + tiles_o == 0) tiles_o = 1;   // nothing to see: one workgroup a row block writes that
    *mt = blocks_of_16(tiles_p > 0 ? (int64_t)T * H : H, fp8);
    p.rb = ceil_div((int64_t)T * H, 16 * *mt);
    p.hb = ceil_div(H, 16 * *mt);
    split(tiles_p, tiles_o ? (int64_t)T * p.hb : 0, tiles_o, (int64_t)T * H, p);
    p.n_prefix = pad8(p.rb * p.sp);
    p.n_own = pad8(T * p.hb * p.so);
    p.slots = p.sp + p.so;
    return p;
}

size_t plan_bytes(const Plan& p, int T, int H) {
    return p.slots == 1 ? 0 : (size_t)p.slots * T * H * (kV + 2) * sizeof(float);
}

template <int KD, int MT, bool TOPK, bool FP8>
hipError_t run(const LatentArgs& a, const Plan& p, hipStream_t stream) {
    static PerDevice<int> once;
    const hipError_t e = set_lds_limit(once, (const void*)latent_attention_kernel<KD, MT, TOPK, FP8>, lds_bytes(MT));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((latent_attention_kernel<KD, MT, TOPK, FP8>), dim3((unsigned)(p.n_prefix + p.n_own)),
                       dim3(kThreads), lds_bytes(MT), stream, a, p);
    return hipGetLastError();
}

template <int KD, int MT, bool TOPK>
hipError_t run(const LatentArgs& a, const Plan& p, bool fp8, hipStream_t stream) {
    if constexpr (MT <= 2)
        if (fp8) return run<KD, MT, TOPK, true>(a, p, stream);
    return run<KD, MT, TOPK, false>(a, p, stream);
}

template <int KD, int MT>
hipError_t run(const LatentArgs& a, const Plan& p, bool fp8, hipStream_t stream) {
    return a.idx ? run<KD, MT, true>(a, p, fp8, stream) : run<KD, MT, false>(a, p, fp8, stream);
}

template <int KD>
hipError_t run(const LatentArgs& a, const Plan& p, int mt, bool fp8, hipStream_t stream) {
    return mt == 1 ? run<KD, 1>(a, p, fp8, stream) : mt == 2 ? run<KD, 2>(a, p, fp8, stream)
                                                             : run<KD, 4>(a, p, fp8, stream);
}

}  // namespace

// The caller's workspace holds the partial sums, then the (maximum, sum) pairs.
size_t latent_topk_workspace_bytes(int T, int H, int K, bool fp8) {
    int mt;
    return plan_bytes(make_plan(T, H, true, K, 0, 0, fp8, &mt), T, H);
}
size_t latent_shared_workspace_bytes(int B, int H, int prefix_len, int max_ctx, bool fp8) {
    int mt;
    return plan_bytes(make_plan(B, H, false, 0, prefix_len, max_ctx, fp8, &mt), B, H);
}

hipError_t launch_latent_attention(const LatentArgs& a, bool fp8, hipStream_t stream) {
    int mt;
    Plan p = make_plan(a.T, a.H, a.idx != nullptr, a.K, a.prefix_len, a.max_ctx, fp8, &mt);
    p.part_o = reinterpret_cast<float*>(a.workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)p.slots * a.T * a.H * kV);
    hipError_t e = a.E == 576 ? run<18>(a, p, mt, fp8, stream) : run<16>(a, p, mt, fp8, stream);
    if (e != hipSuccess || p.slots == 1) return e;
    hipLaunchKernelGGL(latent_join_kernel, dim3((unsigned)(a.T * a.H)), dim3(kThreads), 0, stream, a, p);
    return hipGetLastError();
}

}  // namespace dsaidx
