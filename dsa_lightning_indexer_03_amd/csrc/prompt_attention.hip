// Causal attention over whole prompts: packed sequences of different lengths,
// H query heads over G key/value heads (query head h reads head h / (H / G)).
//
//   S[i, j] = scale * q[i] . k[j]  for the rows j <= i of i's sequence
//   out[i] = sum_j softmax_j(S) v[j],  lse[i] = log sum_j exp S[i, j]
//
// The attention of prompts that are too short for a selection ("Study MLA
// Indexer", the last of the "three whys": dense attention where the prompt has
// no more rows than the selection takes).
//
// One workgroup takes a head and a block of query rows, 32 to a wave, which
// carries them alone through both products:
//   S^T (64 keys x 32 rows) = K Q^T, its queries in registers;
//   O^T (V columns x 32 rows) += V^T P^T.
// The first product leaves a lane with row lane % 32 and keys 4h .. 4h+3 of
// every eight (h = lane / 32), which is the second one's operand when its 16
// keys are counted as 4h .. 4h+3 of two eights: P never leaves its registers,
// and the values are read transposed in that order.  The softmax's factors are
// per lane; the exponent's reference moves when a score passes it by 2^kSlack.
// Sums are fp32; P is rounded to bf16, because the matrix cores take both
// operands of the second product in one type: an output is off by at most 2^-8
// of sum P |v| for that, beside its own rounding.  P's sum is taken before the
// rounding, so that lse does not have it.
//
// Tiles of 64 keys and values are copied to LDS while the tile before is
// computed.  A wave walks its keys from its own rows down to the first: the one
// tile that the causal mask cuts comes first, while the sums are still zero.
// There, and only there, a masked row can meet a value that is not finite, as 0
// times it in the product; the sums then are not finite either, and that tile's
// values are taken again with such elements apart.
#include <utility>

#include "device_once.h"
#include "kv.h"
#include "tile_copy.h"

namespace dsaidx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kTile = 64;       // keys of a tile
constexpr int kWaves = 4;       // waves that share a tile's rows of queries
constexpr int kRows = 32 * kWaves;
constexpr float kFar = 0x1p30f; // references of this size are taken off rounded scores

// A tile's rows lie one behind another in LDS, their 16-byte pieces permuted
// within each 8 (or 16, where a row has a multiple of that) by the row's number.
// The 64 banks serve 16 lanes of a 16-byte read at once (rows of 16 different
// numbers mod 16), 32 lanes of an 8-byte one (64 bytes of four consecutive rows):
// with this permutation both use every bank once.
template <int P>
__device__ __forceinline__ int permute(int row) {
    return P % 16 == 0 ? (row & 3) << 2 | (row >> 2 & 3) : (row >> 1 & 1) << 2 | (row >> 2 & 3);
}

template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* lds_pointer(uint32_t at) {
    return (__attribute__((address_space(3))) T*)(uintptr_t)at;
}
template <typename T>
__device__ __forceinline__ T lds_read(uint32_t at) {
    return *lds_pointer<T>(at);
}

// A wave's copies of a tile of rows of P pieces: N of 1024 bytes, kStep rows each
// kBase.  A lane's place in its source row is found once for kBase
// copies; the next ones are a number of rows on, and permuted by one bit more.
template <int P, int N>
struct Copies {
    static constexpr int kBase = P == 24 ? 3 : 1, kStep = P == 16 ? 4 : 8;
    static constexpr int kBit = P == 16 ? 16 : 32, kTurns = P == 16 ? 4 : 2;
    static_assert(N % kBase == 0, "whole steps");
    int row[kBase];       // of the tile
    uint32_t piece[kBase];
    int64_t stride;       // bytes
    uint32_t first;       // byte of the tile in LDS
    __device__ __forceinline__ Copies(int wave, int lane, int64_t row_stride) {
        stride = 2 * row_stride;
        first = (uint32_t)(wave * N * 1024);
#pragma unroll
        for (int i = 0; i < kBase; ++i) {
            const int at = (wave * N + i) * 64 + lane;
            row[i] = at / P;
            piece[i] = 16u * (uint32_t)(at % P ^ permute<P>(at / P));
        }
    }
    __device__ __forceinline__ void tile(const uint16_t* src, uint32_t lds) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            copy_to_lds(reinterpret_cast<const char*>(src) + i / kBase * kStep * stride,
                        (piece[i % kBase] ^ (uint32_t)(i / kBase % kTurns * kBit)) + (uint32_t)row[i % kBase] * (uint32_t)stride,
                        lds + first + i * 1024);
    }
    // The same where row `last` is the last one: rows behind it are that row again.
    __device__ __forceinline__ void last_tile(const uint16_t* src, uint32_t lds, int last) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            copy_to_lds(src, (piece[i % kBase] ^ (uint32_t)(i / kBase % kTurns * kBit)) +
                                 (uint32_t)min(row[i % kBase] + i / kBase * kStep, last) * (uint32_t)stride,
                        lds + first + i * 1024);
    }
};

// Rows of a block of one sequence.
struct Block {
    int start, len;   // the sequence
    int r0;           // the block's first row in it
    bool pad;         // rows of no sequence, behind the last one
};

// Block `item` of all, false: there are fewer.  The rows behind the last
// sequence count as one more.  With few sequences the blocks come longest first
// (a block's work grows with its first row), so that the last ones to start are
// short; else sequence by sequence, which takes one pass over them.
__device__ __forceinline__ bool find_block(const PromptArgs& a, int item, Block& out) {
    const int lane = lane_id(), segments = a.B + 1;
    auto load = [&](int b, int& s, int& e) {
        s = e = 0;
        if (b < segments) {
            s = min(max(a.cu[b], 0), a.T);
            e = b < a.B ? min(max(a.cu[b + 1], s), a.T) : a.T;
        }
    };
    int s, e, level, found;
    if (segments <= kWave) {
        load(lane, s, e);
        const int n = (e - s + kRows - 1) / kRows;
        if (item >= (int)wave_sum((uint32_t)n)) return false;
        // largest level with more than `item` blocks at or above it
        int lo = 0, hi = (a.T + kRows - 1) / kRows;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int)wave_sum((uint32_t)max(n - mid, 0)) > item) lo = mid;
            else hi = mid;
        }
        level = lo;
        const int rank = item - (int)wave_sum((uint32_t)max(n - level - 1, 0));
        const uint64_t mask = wave_ballot(n > level);
        found = __builtin_ctzll(wave_ballot(n > level && lanes_below(mask) == rank));
        out.pad = found == a.B;
    } else {
        int base = 0, at = 0;
        uint32_t incl;
        for (;; at += kWave) {
            if (at >= segments) return false;
            load(at + lane, s, e);
            incl = wave_incl_scan((uint32_t)((e - s + kRows - 1) / kRows));
            const int all = __builtin_amdgcn_readlane((int)incl, kWave - 1);
            if (base + all > item) break;
            base += all;
        }
        found = __builtin_ctzll(wave_ballot(base + (int)incl > item));
        level = base + __builtin_amdgcn_readlane((int)incl, found) - 1 - item;
        out.pad = at + found == a.B;
    }
    out.start = __builtin_amdgcn_readlane(s, found);
    out.len = __builtin_amdgcn_readlane(e, found) - out.start;
    out.r0 = level * kRows;
    return true;
}

// bf16 pairs: 1.0 where an element is not finite and of that sign (NaN: of both).
__device__ __forceinline__ uint32_t not_finite(uint32_t x, uint32_t sign) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
        const uint32_t u = x >> i & 0xFFFFu;
        if ((u & 0x7FFFu) > 0x7F80u || u == (sign | 0x7F80u)) r |= 0x3F80u << i;
    }
    return r;
}
__device__ __forceinline__ uint32_t finite(uint32_t x) {
    if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
    if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
    return x;
}

// f(0), f(1), ..., f(N - 1) with numbers known while compiling
template <typename F, int... I>
__device__ __forceinline__ void steps(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void steps(F&& f) {
    steps(f, std::make_integer_sequence<int, N>{});
}

// The products of a turn, in order: scores of the next tile (half `a` of its keys,
// 16 columns b) between values of this one (16 keys a, 32 columns b).
struct Step {
    bool values;
    int a, b;
};
template <int KS, int MT>
struct Turn {
    static constexpr int kSteps = 2 * KS + 4 * MT;
    static constexpr Step step(int f) {
        if (f < KS) return {false, 0, f};
        f -= KS;
        for (int s = 0; s < 2; ++s) {
            if (f < MT) return {true, s, f};
            f -= MT;
            if (f < KS / 2) return {false, 1, s * (KS / 2) + f};
            f -= KS / 2;
        }
        return {true, 2 + f / MT, f % MT};
    }
    // elements of a lane's 32 whose probabilities are made before step f: 8 (s + 1) of them
    // before the values of keys 16 s take the first
    static constexpr int made(int f) {
        constexpr int len[6] = {KS, MT, KS / 2, MT, KS / 2, MT}, el[6] = {12, 4, 4, 4, 4, 4};
        int n = 0;
        for (int i = 0; i < 6; ++i) {
            if (f <= len[i]) return n + el[i] * f / len[i];
            n += el[i];
            f -= len[i];
        }
        return n;
    }
};

template <int D, int V, int KG>
__global__ void __launch_bounds__(64 * kWaves * KG, 2)
prompt_attention_kernel(PromptArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int KP = D / 8, VP = V / 8;                       // 16-byte pieces of a row
    constexpr int kKeyB = kTile * D * 2, kTileB = kKeyB + kTile * V * 2;
    constexpr int KI = kKeyB / 1024 / kWaves, VI = kTile * V * 2 / 1024 / kWaves;  // copies of a wave
    constexpr int kAhead = D >= 128 ? 3 : 4;                    // operand reads in flight
    constexpr int KS = D / 16, MT = V / 32;                     // steps of the first product, blocks of the second
    const int wave = uniform((int)threadIdx.x >> 6) % kWaves, kg = KG == 1 ? 0 : uniform((int)threadIdx.x >> 6) / kWaves;
    const int lane = lane_id(), n = lane & 31, h = lane >> 5;
    constexpr int kThreads = 64 * kWaves * KG;

    // heads of one key/value head go to one XCD (workgroups go to the 8 in turn)
    const int j = (int)(blockIdx.x % (unsigned)a.H);
    const int head = a.H % 8 == 0 ? (j & 7) * (a.H >> 3) + (j >> 3) : j;
    Block blk;
    if (!find_block(a, (int)(blockIdx.x / (unsigned)a.H), blk)) return;
    const int rows = min(kRows, blk.len - blk.r0);
    const int64_t out_row = (int64_t)(blk.start + blk.r0) * a.H + head;   // of [T][H]
    if (blk.pad) {
        for (int i = (int)threadIdx.x; i < rows * VP; i += kThreads)
            *reinterpret_cast<v4i*>(a.out + (out_row + (int64_t)(i / VP) * a.H) * V + 8 * (i % VP)) = v4i{0, 0, 0, 0};
        if (a.lse)
            for (int i = (int)threadIdx.x; i < rows; i += kThreads)
                a.lse[out_row + (int64_t)i * a.H] = -__builtin_inff();
        return;
    }
    const int g = head / (a.H / a.G);
    const uint16_t* kbase = reinterpret_cast<const uint16_t*>(a.k.p) + blk.start * a.k.row + g * a.k.head;
    const uint16_t* vbase = reinterpret_cast<const uint16_t*>(a.v.p) + blk.start * a.v.row + g * a.v.head;

    const int r0 = blk.r0 + 32 * wave;   // this wave's first row in the sequence
    const bool active = 32 * wave < rows;
    // (never 0: a score of -inf has to stay one)
    const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);

    // ---- copies: a wave's part of a tile, 1024 bytes each; first of all the first keys and
    //      the wave's queries, the latter behind the first keys ----
    const uint32_t lds0 = lds_address(smem) + kg * 2 * kTileB;   // this key group's two slots
    const Copies<KP, KI> kc(wave, lane, a.k.row);
    const Copies<VP, VI> vc(wave, lane, a.v.row);
    const int t_mine = r0 / kTile;   // the tile that the mask cuts for this wave's rows
    const int t_first = (blk.r0 + rows - 1) / kTile;
    int t = t_first - kg + KG;       // (the loop below)
    if (t >= KG)
        kc.last_tile(kbase + (int64_t)kTile * (t - KG) * a.k.row, lds0, blk.len - 1 - kTile * (t - KG));
    v8bf Q[KS];   // B operand of 32 rows x 16 columns
    if (active) {
        static_assert(kWaves * 32 * 2 * D <= kTileB + kTile * V * 2, "the queries fit the first values' place and the second slot");
        const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q.p) + blk.start * a.q.row + head * a.q.head;
        const uint32_t at = lds0 + kKeyB + wave * (32 * 2 * D);
        const Copies<KP, D / 16> qc(0, lane, a.q.row);
        qc.last_tile(qp + (int64_t)r0 * a.q.row, at, min(31, blk.len - 1 - r0));
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        asm volatile("" ::: "memory");
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Q[ks] = lds_read<v8bf>(at + n * (2 * D) + 16 * ((2 * ks + h) ^ permute<KP>(n)));
            if (a.scale_log2 < 0.f) {   // the products then take the scale's magnitude
                v4i u = __builtin_bit_cast(v4i, Q[ks]);
                u ^= (int)0x80008000;
                Q[ks] = __builtin_bit_cast(v8bf, u);
            }
        }
    }

    v16f O[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[mt][i] = 0.f;
    // the reference starts below every score that is not -inf, so that a row's first one moves it
    float m = -3.402823466e38f, l = 0.f;
    bool far = false;
    v16f S0[2], S1[2];      // scores of this turn's tile and the next one's, in turn
    float top = 0.f;        // the highest of the next one's
    v4i P[4];               // probabilities of keys 16 s ..
    float by = 0.f, off = 0.f, sum = 0.f, even = 0.f;
    auto weigh = [&](const v16f (&S)[2], int e) {   // element e of a lane's 32
        const float x = __builtin_amdgcn_exp2f(fmaf(S[e / 16][e % 16], by, -off));
        sum += x;
        if (e % 2) P[e / 8][e % 8 / 2] = (int)pack_bf16(even, x);
        even = x;
    };

    // operand addresses in the first slot; a step's columns differ in bits of the permuted piece
    constexpr int KPX = KP % 16 == 0 ? 16 : 8;
    const uint32_t k_at = lds0 + n * (2 * D) + 16 * (h ^ permute<KP>(n));
    const int v_row = 4 * h + (lane >> 2 & 3);
    const uint32_t v_at = lds0 + kKeyB + v_row * (2 * V) +
                          16 * ((2 * (lane >> 4 & 1) + (lane >> 1 & 1)) ^ permute<VP>(v_row)) + 8 * (lane & 1);
    int slot = 0;
    auto read_k = [&](int kt, int ks) {   // A operand: 32 keys x 16 columns
        const int c = 2 * ks;
        return lds_read<v8bf>(((k_at + slot * kTileB) ^ (16 * (c % KPX))) + 16 * (c / KPX * KPX) + kt * (64 * D));
    };
    auto read_v = [&](int s, int mt) {    // A operand: 32 columns x 16 keys
        const uint32_t at = (v_at + slot * kTileB) ^ (64 * mt);
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_pointer<v4s>(at + s * (32 * V)));
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_pointer<v4s>((at ^ 32) + s * (32 * V) + 16 * V));
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto highest = [&](const v16f (&S)[2], int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i) top = fmaxf(top, S[i / 16][i % 16]);
    };
    using T = Turn<KS, MT>;
    auto read = [&](auto f) {
        constexpr Step st = T::step(decltype(f)::value);
        if constexpr (st.values) return read_v(st.a, st.b);
        else return read_k(st.a, st.b);
    };

    // A turn: the probabilities of the tile with scores S, its values, and the next tile's
    // scores N (behind the last tile: of keys that are none, for nothing).
    auto turn = [&](v16f (&S)[2], v16f (&N)[2], bool first) __attribute__((always_inline)) {
        v8bf F[kAhead];
        steps<kAhead>([&](auto f) { F[f] = read(f); });
        by = scale;
        off = m;
        sum = 0.f;
        if (first || far || wave_ballot(top * scale > m + kSlack)) {
            // a row's reference moves to these keys' maximum where that is so far above it (the
            // rows beside it keep theirs: no row's result depends on another's)
            float to = top * scale;
            to = fmaxf(to, __shfl_xor(to, 32, kWave));
            to = to > m + kSlack ? to : m;
            const float f = __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
            if (!first)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) O[mt] *= f;
            // rows with a reference that far off: scores are rounded before it is taken off them (left
            // whole in an fma, they would keep what it has not: 2 to that may be infinite)
            const bool here = fabsf(m) >= kFar;
            far = wave_ballot(here) != 0;
            by = here ? 1.f : scale;
            off = here ? 0.f : m;
            if (far) {
#pragma clang fp contract(off)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = S[kt][i] * scale;
                        S[kt][i] = here ? x - m : S[kt][i];
                    }
            }
        }
        top = -__builtin_inff();
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int i = 0; i < 16; ++i) N[kt][i] = 0.f;
        steps<T::kSteps>([&](auto step) {
            constexpr int f = decltype(step)::value, kLast = T::kSteps - MT;
            constexpr Step st = T::step(f);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (st.values)
                O[st.b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F[f % kAhead], __builtin_bit_cast(v8bf, P[st.a]),
                                                                  O[st.b], 0, 0, 0);
            else
                N[st.a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F[f % kAhead], Q[st.b], N[st.a], 0, 0, 0);
            if constexpr (f + kAhead < T::kSteps) F[f % kAhead] = read(std::integral_constant<int, f + kAhead>{});
            constexpr int e0 = T::made(f), e1 = T::made(f + 1);
            steps<e1 - e0>([&](auto e) { weigh(S, e0 + decltype(e)::value); });
            if constexpr (f >= kLast) highest(N, (f - kLast) * 32 / MT, (f - kLast + 1) * 32 / MT);
        });
        // (made here, beside the products, not where it is known that they are used)
        asm volatile("" : "+v"(sum), "+v"(top));
        __builtin_amdgcn_sched_barrier(0);
        l += sum;
    };

    // ---- the tiles of this key group, from t_first - kg down.  A slot holds the values of a
    //      turn's tile t and the keys of the next, t - KG; while a turn is taken the slot of the
    //      next one is copied.  Every wave meets the others once a turn, with or without work. ----
    auto stage = [&](int t, int slot) {
        const int last = blk.len - 1 - kTile * t;   // (only the last tile can pass the sequence's last row)
        if (t >= KG) kc.tile(kbase + (int64_t)kTile * (t - KG) * a.k.row, lds0 + slot * kTileB);
        if (t == t_first) vc.last_tile(vbase + (int64_t)kTile * t * a.v.row, lds0 + slot * kTileB + kKeyB, last);
        else if (t >= 0) vc.tile(vbase + (int64_t)kTile * t * a.v.row, lds0 + slot * kTileB + kKeyB);
    };
    auto next_turn = [&]() {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the slot
        tile_barrier();
        stage(t - KG, slot ^ 1);
    };
    auto done = [&]() {
        t -= KG;
        slot ^= 1;
    };
    while (t + kg >= 0 && (!active || t - KG > t_mine)) {
        next_turn();
        done();
    }
    if (t - KG >= 0 && active) {
        next_turn();
        {
            v8bf F[kAhead];
#pragma unroll
            for (int f = 0; f < kAhead; ++f) F[f] = read_k(f / KS, f % KS);
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int i = 0; i < 16; ++i) S0[kt][i] = 0.f;
#pragma unroll
            for (int f = 0; f < 2 * KS; ++f) {
                __builtin_amdgcn_sched_barrier(0);
                S0[f / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F[f % kAhead], Q[f % KS], S0[f / KS], 0, 0, 0);
                if (f + kAhead < 2 * KS) F[f % kAhead] = read_k((f + kAhead) / KS, (f + kAhead) % KS);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        done();
        const int mine = t == t_mine ? (r0 & (kTile - 1)) + n - 4 * h : kTile;
        top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (32 * (i / 16) + 8 * (i % 16 / 4) + i % 4 > mine) S0[i / 16][i % 16] = -__builtin_inff();
        highest(S0, 0, 32);
        next_turn();
        turn(S0, S1, true);
        if (t == t_mine) {
            float z = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i) z = fmaf(O[mt][i], 0.f, z);
            if (wave_ballot(z != z)) {
                // once more: finite elements as before, the others by which rows see them
                v8bf see[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    v4i u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * s + 8 * (i / 2) + 2 * (i % 2);
                        u[i] = (key <= mine ? 0x3F80 : 0) | (key + 1 <= mine ? 0x3F800000 : 0);
                    }
                    see[s] = __builtin_bit_cast(v8bf, u);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) weigh(S0, e);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    v16f up, down;
#pragma unroll
                    for (int i = 0; i < 16; ++i) O[mt][i] = up[i] = down[i] = 0.f;
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const v4i w = __builtin_bit_cast(v4i, read_v(s, mt));
                        v4i f, p, q;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[i] = (int)finite((uint32_t)w[i]);
                            p[i] = (int)not_finite((uint32_t)w[i], 0);
                            q[i] = (int)not_finite((uint32_t)w[i], 0x8000u);
                        }
                        O[mt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, f),
                                                                        __builtin_bit_cast(v8bf, P[s]), O[mt], 0, 0, 0);
                        up = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, p), see[s], up, 0, 0, 0);
                        down = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, q), see[s], down, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (up[i] > 0.f) O[mt][i] += __builtin_inff();
                        if (down[i] > 0.f) O[mt][i] -= __builtin_inff();
                    }
                }
            }
        }
        done();
        while (t >= 0) {
            next_turn();
            turn(S1, S0, false);
            done();
            if (t < 0) break;
            next_turn();
            turn(S0, S1, false);
            done();
        }
    }
    while (t + kg >= 0) {
        next_turn();
        done();
    }

    if constexpr (KG > 1) {   // ---- join the key groups ----
        v4f* there = reinterpret_cast<v4f*>(smem) + wave * (4 * MT * 64) + lane;
        float2* ml = reinterpret_cast<float2*>(smem + kWaves * MT * 4 * 64 * 16) + wave * 64 + lane;
        static_assert(KG == 2 && kWaves * 64 * (MT * 64 + 8) <= 4 * kTileB, "the sums fit the tiles' place");
        tile_barrier();
        if (kg == 1) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    there[(4 * mt + i) * 64] = v4f{O[mt][4 * i], O[mt][4 * i + 1], O[mt][4 * i + 2], O[mt][4 * i + 3]};
            *ml = float2{m, l};
        }
        tile_barrier();
        if (kg == 1) return;
        const float2 x = *ml;
        const float to = fmaxf(m, x.x);
        const float f = __builtin_amdgcn_exp2f(m - to), fx = __builtin_amdgcn_exp2f(x.x - to);
        m = to;
        l = l * f + x.y * fx;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 16; ++i) O[mt][i] = O[mt][i] * f + there[(4 * mt + i / 4) * 64][i % 4] * fx;
    }

    // ---- write: rows through LDS, so that a store takes whole ones ----
    l += __shfl_xor(l, 32, kWave);
    constexpr int kOutB = 2 * V + 16;
    unsigned char* rows_at = smem + wave * (KG > 1 ? MT * 4 * 64 * 16 : 32 * kOutB);
    static_assert(32 * kOutB <= MT * 4 * 64 * 16 && kWaves * 32 * kOutB <= 2 * kTileB, "the rows fit the sums' or tiles' place");
    if constexpr (KG == 1) tile_barrier();
    if (!active) return;
    const float inv = 1.f / l;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i)   // columns 4h .. 4h+3 of every eight of row n
            *reinterpret_cast<uint2*>(rows_at + n * kOutB + 64 * mt + 16 * i + 8 * h) =
                l == 0.f ? uint2{0, 0}
                         : uint2{pack_bf16(O[mt][4 * i] * inv, O[mt][4 * i + 1] * inv),
                                 pack_bf16(O[mt][4 * i + 2] * inv, O[mt][4 * i + 3] * inv)};
    const int64_t first_row = out_row + (int64_t)(32 * wave) * a.H;
#pragma unroll
    for (int i = 0; i < VP / 2; ++i) {
        const int r = i * (64 / VP) + lane / VP, c = lane % VP;
        const v4i x = *reinterpret_cast<const v4i*>(rows_at + r * kOutB + 16 * c);
        if (32 * wave + r < rows) *reinterpret_cast<v4i*>(a.out + (first_row + (int64_t)r * a.H) * V + 8 * c) = x;
    }
    if (a.lse && h == 0 && 32 * wave + n < rows)
        a.lse[first_row + (int64_t)n * a.H] = l == 0.f ? -__builtin_inff() : (m + log2f(l)) * 0.693147180559945f;
}

template <int D, int V, int KG>
hipError_t run(const PromptArgs& a, hipStream_t stream) {
    static PerDevice<int> once;
    constexpr int lds = KG * 2 * kTile * 2 * (D + V);
    const hipError_t e = set_lds_limit(once, (const void*)prompt_attention_kernel<D, V, KG>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((prompt_attention_kernel<D, V, KG>), dim3((unsigned)prompt_blocks(a.T, a.B, a.H)),
                       dim3(64 * kWaves * KG), lds, stream, a);
    return hipGetLastError();
}

// Two key groups where the blocks leave waves' places free and sequences are long
// enough: with up to 640 blocks (256 CUs hold 512 of one group) and more than 256
// rows a sequence.  Of 128 columns, one and two groups: 2048 rows of 16 heads (272
// blocks) 38.9 and 33.3 us, 8192 of 8 (528) 165 and 142, 2048 of 32 (576) 48.6 and
// 47.3, 8192 of 16 (1056) 269 and 272; 256 rows of 16 heads 10.1 and 10.2, 64 6.2
// and 7.5.
template <int D, int V>
hipError_t run(const PromptArgs& a, hipStream_t stream) {
    const bool two = prompt_blocks(a.T, a.B, a.H) <= 640 && (int64_t)a.T > 256 * (int64_t)a.B;
    return two ? run<D, V, 2>(a, stream) : run<D, V, 1>(a, stream);
}

}  // namespace

// At most floor(T / kRows) whole blocks and a rest of each of the B sequences and of the rows behind them.
int64_t prompt_blocks(int T, int B, int H) { return ((int64_t)T / kRows + B + 1) * H; }

hipError_t launch_prompt_attention(const PromptArgs& a, int D, hipStream_t stream) {
    if (a.T <= 0) return hipSuccess;
    return D == 64 ? run<64, 64>(a, stream) : D == 128 ? run<128, 128>(a, stream) : run<192, 128>(a, stream);
}

}  // namespace dsaidx
