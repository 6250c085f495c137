// Causal attention over whole prompts: packed sequences of different lengths,
// H query heads over G key/value heads (query head h reads head h / (H / G)).
//
//   S[i, j] = scale * q[i] . k[j]  for the rows j <= i of i's sequence
//   out[i] = sum_j softmax_j(S) v[j],  lse[i] = log sum_j exp S[i, j]
//
// The attention of prompts that are too short for a selection ("Study MLA
// Indexer": a prompt of no more rows than the selection takes is attended to
// densely).
//
// One workgroup takes a head and a block of query rows, 32 to a wave, which
// carries them through both products:
//   S^T (keys x 32 rows) = K Q^T, its queries in registers;
//   O^T (V columns x 32 rows) += V^T P^T.
// The first product leaves a lane with row lane % 32 and keys 4h .. 4h+3 of
// every eight (h = lane / 32), which is the second one's operand when its 16
// keys are counted as 4h .. 4h+3 of two eights: P never leaves its registers,
// and the values are read transposed in that order.  The softmax's factors are
// per lane; the exponent's reference moves when a score passes it by 2^kSlack.
// Sums are fp32; P is rounded to bf16, because the matrix cores take both
// operands of the second product in one type, and a second term for what the
// rounding leaves would be half as many matrix instructions again in a kernel
// that they bound: an output is off by at most 2^-8 of sum P |v| for that, beside
// its own rounding (2.1e-3 rms of the outputs where the rounding alone is 1.6e-3).
// P's sum is taken before the rounding, so that lse does not have it.
//
// A turn of a wave makes the probabilities of its keys, 64 or 32 of a tile, beside the
// next tile's scores, and takes these keys' values between those: matrix and
// vector instructions alternate, and each has about as many cycles as the other
// (32 rows of 128 columns: 1024 and 900).  Where blocks are few, two or four key
// groups of waves share a block's tiles and are joined through LDS (choice and
// figures: run).  Keys and values are copied to LDS by turns, a tile ahead.
//
// A wave walks its keys from its own rows down to the first: the one tile that
// the causal mask cuts comes first, while the sums are still zero.  There, and
// only there, a masked row can meet a value that is not finite, as 0 times it in
// the product; the sums then are not finite either, and that tile's values are
// taken again with such elements apart.
//
// Bound by the matrix cores and the power limit, which sets the clock: 32768 rows
// of 16 heads over 2, 128 columns (4.4 TFLOP): 3.67 to 4.05 ms on different cards, 1.09
// to 1.20 PFLOP/s, the matrix cores busy 71% of the cycles at about 1.7 GHz, where a
// bf16 matrix product of 8192 cubed reaches 1.37 in a row.  64 columns are bound by the
// vector instructions of the softmax, as many as for 128: 0.94 to 0.98 PFLOP/s; 192
// and 128 columns, 8192 rows of 16 heads: 1.04 to 1.09.  Short sequences by their
// first tiles' latency, the masked part and the end: 16 of 59 to 2331 rows, 16 heads
// of 192 and 128 columns with keys of their own (79 GFLOP, 252 MB), 113 to 126 us, 106
// where the caches hold the inputs; 32 of 512, 32 heads over 8 of 128 columns (70
// GFLOP, 335 MB) 119.  61 rows: 8 us, of which the launch, the first loads and the end
// are all but one.
#include <utility>

#include "device_once.h"
#include "kv.h"
#include "tile_copy.h"

namespace dsaidx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

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

// Block `item` of the launch, false: none.  The rows behind the last sequence
// count as one more.  With few sequences the blocks come longest first (a
// block's work grows with its first row), so that the last ones to start are
// short.  Else sequence b's blocks have the numbers from cu[b] / kRows + b on,
// which leaves room for all of them before the next one's, and b is found among
// 64 places at a time: sequences may be as many as rows.
template <int kRows>
__device__ __forceinline__ bool find_block(const PromptArgs& a, int item, Block& out) {
    const int lane = lane_id(), segments = a.B + 1;
    auto first_row = [&](int b) { return min(max(a.cu[b], 0), a.T); };
    int start, end, level;
    if (segments <= kWave) {
        int s = 0, e = 0;
        if (lane < segments) {
            s = first_row(lane);
            e = lane < a.B ? max(first_row(lane + 1), s) : a.T;
        }
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
        const int found = __builtin_ctzll(wave_ballot(n > level && lanes_below(mask) == rank));
        out.pad = found == a.B;
        start = __builtin_amdgcn_readlane(s, found);
        end = __builtin_amdgcn_readlane(e, found);
    } else {
        int b = 0, n = segments;
        while (n > 1) {
            const int step = (n + kWave - 1) / kWave, at = b + lane * step;
            const bool in = lane * step < n;
            const uint64_t upto = wave_ballot(in && first_row(in ? at : b) / kRows + at <= item);
            const int last = max(__builtin_popcountll(upto) - 1, 0) * step;
            b += last;
            n = min(step, n - last);
        }
        start = uniform(first_row(b));
        end = b < a.B ? max(uniform(first_row(b + 1)), start) : a.T;
        out.pad = b == a.B;
        const int at = item - start / kRows - b;
        level = (end - start + kRows - 1) / kRows - 1 - at;
        if (at < 0 || level < 0) return false;   // (before the first sequence; behind b's last block)
    }
    out.start = start;
    out.len = end - start;
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

// The products of a turn, in order: scores of the wave's next keys (32 keys `a` of
// them, 16 columns b) between values of these (16 keys a, 32 columns b).  NH: 32s
// of keys.
struct Step {
    bool values;
    int a, b;
};
template <int KS, int MT, int NH>
struct Turn {
    static constexpr int kSteps = NH * (KS + 2 * MT);
    static constexpr Step step(int f) {
        if (f < KS) return {false, 0, f};
        f -= KS;
        for (int s = 0; s < 2 && NH == 2; ++s) {
            if (f < MT) return {true, s, f};
            f -= MT;
            if (f < KS / 2) return {false, 1, s * (KS / 2) + f};
            f -= KS / 2;
        }
        return {true, 2 * (NH - 1) + f / MT, f % MT};
    }
    // elements of a lane's 16 NH whose probabilities are made before step f: 8 (s + 1) of
    // them before the values of keys 16 s take the first
    static constexpr int made(int f) {
        constexpr int len[6] = {KS, MT, KS / 2, MT, KS / 2, MT}, el[6] = {12, 4, 4, 4, 4, 4};
        int n = 0;
        for (int i = 0; i < 2 + 4 * (NH - 1); ++i) {
            if (f <= len[i]) return n + el[i] * f / len[i];
            n += el[i];
            f -= len[i];
        }
        return n;
    }
};

// LDS of a workgroup: two slots, the first keys and the queries, or the key groups' sums
template <int D, int V, int RG, int KG, int NK>
constexpr int lds_bytes() {
    const int slots = 2 * KG * NK * 2 * (D + V), start = KG * NK * 2 * D + RG * KG * 32 * 2 * D;
    const int sums = KG > 1 ? RG * KG * (V / 32 * 4 * 64 * 16 + 64 * 8) : 0;
    const int most = slots > start ? slots : start;
    return most > sums ? most : sums;
}

template <int D, int V, int RG, int KG, int NK>
__global__ void __launch_bounds__(64 * RG * KG, KG > 1 || NK > 32 ? 2 : D == 64 ? 4 : 3)
prompt_attention_kernel(PromptArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int KP = D / 8, VP = V / 8;                       // 16-byte pieces of a row
    constexpr int kWaves = RG * KG, kThreads = 64 * kWaves, kRows = 32 * RG;
    constexpr int kTile = KG * NK, kKeyB = kTile * D * 2, kTileB = kKeyB + kTile * V * 2;
    constexpr int KI = kKeyB / 1024 / kWaves, VI = kTile * V * 2 / 1024 / kWaves;  // copies of a wave
    constexpr int kAhead = D >= 128 ? 3 : 4;                    // operand reads in flight
    constexpr bool kFew = KG == 1 && NK == 32;
    constexpr int KS = D / 16, MT = V / 32, NH = NK / 32;       // steps of the first product, blocks of the second
    constexpr int kLds = lds_bytes<D, V, RG, KG, NK>();
    static_assert(kLds <= 160 * 1024, "LDS");
    const int wave = uniform((int)threadIdx.x >> 6), rg = wave % RG, kg = wave / RG;
    const int lane = lane_id(), n = lane & 31, h = lane >> 5;

    // heads of one key/value head go to one XCD (workgroups go to the 8 in turn)
    const int j = (int)(blockIdx.x % (unsigned)a.H);
    const int head = a.H % 8 == 0 ? (j & 7) * (a.H >> 3) + (j >> 3) : j;
    Block blk;
    if (!find_block<kRows>(a, (int)(blockIdx.x / (unsigned)a.H), blk)) return;
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

    const int r0 = blk.r0 + 32 * rg;   // this wave's first row in the sequence
    const bool active = 32 * rg < rows;
    // (never 0: a score of -inf has to stay one)
    const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);

    // ---- copies: a wave's part of a tile, 1024 bytes each; first of all the first keys and
    //      the wave's queries, behind them, then the second slot, where the queries were ----
    const uint32_t lds0 = lds_address(smem);
    const Copies<KP, KI> kc(wave, lane, a.k.row);
    const Copies<VP, VI> vc(wave, lane, a.v.row);
    const int t_first = (blk.r0 + rows - 1) / kTile, last = blk.len - 1 - kTile * t_first;
    kc.last_tile(kbase + (int64_t)kTile * t_first * a.k.row, lds0, last);
    const uint32_t q_at = lds0 + kKeyB + wave * (32 * 2 * D);
    if (active) {
        const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q.p) + blk.start * a.q.row + head * a.q.head;
        const Copies<KP, D / 16> qc(0, lane, a.q.row);
        qc.last_tile(qp + (int64_t)r0 * a.q.row, q_at, min(31, blk.len - 1 - r0));
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    asm volatile("" ::: "memory");
    v8bf Q[KS];   // B operand of 32 rows x 16 columns
    if (active) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Q[ks] = lds_read<v8bf>(q_at + n * (2 * D) + 16 * ((2 * ks + h) ^ permute<KP>(n)));
            if (a.scale_log2 < 0.f) {   // the products then take the scale's magnitude
                v4i u = __builtin_bit_cast(v4i, Q[ks]);
                u ^= (int)0x80008000;
                Q[ks] = __builtin_bit_cast(v8bf, u);
            }
        }
    }
    tile_barrier();
    if (t_first > 0) kc.tile(kbase + (int64_t)kTile * (t_first - 1) * a.k.row, lds0 + kTileB);
    vc.last_tile(vbase + (int64_t)kTile * t_first * a.v.row, lds0 + kTileB + kKeyB, last);   // (no other tile can pass the sequence's last row)
    v16f O[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[mt][i] = 0.f;
    // the reference starts below every score that is not -inf, so that a row's first one moves it
    float m = -3.402823466e38f, l = 0.f;
    bool far = false;
    v16f S0[NH], S1[NH];    // scores of this turn's keys and the next one's, in turn
    float top = 0.f;        // the highest of the next one's
    v4i P[2 * NH];               // probabilities of keys 16 s ..
    float by = 0.f, off = 0.f, sum = 0.f, even = 0.f;
    auto weigh = [&](const v16f (&S)[NH], int e) {   // element e of a lane's 16 NH
        const float x = __builtin_amdgcn_exp2f(fmaf(S[e / 16][e % 16], by, -off));
        sum += x;
        if (e % 2) P[e / 8][e % 8 / 2] = (int)pack_bf16(even, x);
        even = x;
    };

    // operand addresses in the first slot; a step's columns differ in bits of the permuted piece
    constexpr int KPX = KP % 16 == 0 ? 16 : 8;
    const uint32_t k_at = lds0 + (kg * NK + n) * (2 * D) + 16 * (h ^ permute<KP>(n));
    const int v_row = 4 * h + (lane >> 2 & 3);
    const uint32_t v_at = lds0 + kKeyB + (kg * NK + v_row) * (2 * V) +
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
    auto highest = [&](const v16f (&S)[NH], int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i) top = fmaxf(top, S[i / 16][i % 16]);
    };
    using T = Turn<KS, MT, NH>;
    auto read = [&](auto f) {
        constexpr Step st = T::step(decltype(f)::value);
        if constexpr (st.values) return read_v(st.a, st.b);
        else return read_k(st.a, st.b);
    };

    // A turn: the probabilities of the tile with scores S, its values, and the next tile's
    // scores N (behind the last tile: of keys that are none, for nothing).
    auto turn = [&](v16f (&S)[NH], v16f (&N)[NH], bool first) __attribute__((always_inline)) {
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
                for (int kt = 0; kt < NH; ++kt)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = S[kt][i] * scale;
                        S[kt][i] = here ? x - m : S[kt][i];
                    }
            }
        }
        top = -__builtin_inff();
#pragma unroll
        for (int kt = 0; kt < NH; ++kt)
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
            if constexpr (f >= kLast) highest(N, (f - kLast) * 16 * NH / MT, (f - kLast + 1) * 16 * NH / MT);
        });
        // (made here, beside the products, not where it is known that they are used)
        asm volatile("" : "+v"(sum), "+v"(top));
        __builtin_amdgcn_sched_barrier(0);
        l += sum;
    };

    // ---- the tiles, from t_first down.  A slot holds the values of a turn's tile t and the
    //      keys of the next, t - 1; while a turn is taken the slot of the next one is copied.
    //      Every wave meets the others once a turn, with or without work. ----
    const int own = r0 / NK;                          // the last NK keys that this wave's rows see, cut by the mask
    const int t_mine = own >= kg ? (own - kg) / KG : -1;   // the tile with the last of this wave's keys that they see
    int t = t_first + 1;
    auto next_turn = [&]() {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the slot
        tile_barrier();
        const uint32_t at = lds0 + (slot ^ 1) * kTileB;
        if (t > 1) kc.tile(kbase + (int64_t)kTile * (t - 2) * a.k.row, at);
        if (t > 0) vc.tile(vbase + (int64_t)kTile * (t - 1) * a.v.row, at + kKeyB);
    };
    auto done = [&]() {
        --t;
        slot ^= 1;
        // (where registers are few: addresses of one slot at a time)
        if constexpr (kFew) asm volatile("" : "+s"(slot));
    };
    // (turn t_first + 1, in which no values are taken, has begun above)
    while (t > 0 && (!active || t - 1 > t_mine)) {
        done();
        next_turn();
    }
    if (t > 0) {
        {
            v8bf F[kAhead];
#pragma unroll
            for (int f = 0; f < kAhead; ++f) F[f] = read_k(f / KS, f % KS);
#pragma unroll
            for (int kt = 0; kt < NH; ++kt)
#pragma unroll
                for (int i = 0; i < 16; ++i) S0[kt][i] = 0.f;
#pragma unroll
            for (int f = 0; f < NH * KS; ++f) {
                __builtin_amdgcn_sched_barrier(0);
                S0[f / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F[f % kAhead], Q[f % KS], S0[f / KS], 0, 0, 0);
                if (f + kAhead < NH * KS) F[f % kAhead] = read_k((f + kAhead) / KS, (f + kAhead) % KS);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        done();
        const bool cut = KG * t + kg == own;
        const int mine = cut ? r0 % NK + n - 4 * h : NK;
        top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 16 * NH; ++i)
            if (32 * (i / 16) + 8 * (i % 16 / 4) + i % 4 > mine) S0[i / 16][i % 16] = -__builtin_inff();
        highest(S0, 0, 16 * NH);
        next_turn();
        turn(S0, S1, true);
        if (cut) {
            float z = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i) z = fmaf(O[mt][i], 0.f, z);
            if (wave_ballot(z != z)) {
                // once more: finite elements as before, the others by which rows see them
                v8bf see[2 * NH];
#pragma unroll
                for (int s = 0; s < 2 * NH; ++s) {
                    v4i u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * s + 8 * (i / 2) + 2 * (i % 2);
                        u[i] = (key <= mine ? 0x3F80 : 0) | (key + 1 <= mine ? 0x3F800000 : 0);
                    }
                    see[s] = __builtin_bit_cast(v8bf, u);
                }
#pragma unroll
                for (int e = 0; e < 16 * NH; ++e) weigh(S0, e);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) O[mt][i] = 0.f;
#pragma unroll
                    for (int s = 0; s < 2 * NH; ++s) {
                        v4i w = __builtin_bit_cast(v4i, read_v(s, mt));
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = (int)finite((uint32_t)w[i]);
                        O[mt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w),
                                                                        __builtin_bit_cast(v8bf, P[s]), O[mt], 0, 0, 0);
                    }
#pragma unroll
                    for (const uint32_t sign : {0u, 0x8000u}) {
                        __builtin_amdgcn_sched_barrier(0);   // (one sign's counts at a time: registers)
                        v16f seen;
#pragma unroll
                        for (int i = 0; i < 16; ++i) seen[i] = 0.f;
#pragma unroll
                        for (int s = 0; s < 2 * NH; ++s) {
                            v4i w = __builtin_bit_cast(v4i, read_v(s, mt));
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = (int)not_finite((uint32_t)w[i], sign);
                            seen = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w), see[s], seen, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (seen[i] > 0.f) O[mt][i] += sign ? -__builtin_inff() : __builtin_inff();
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

    if constexpr (KG > 1) {   // ---- join the key groups: a row's sums through LDS to the first ----
        constexpr int kSums = 4 * MT * 64 * 16;   // bytes of a wave's
        v4f* there = reinterpret_cast<v4f*>(smem + wave * kSums) + lane;
        float2* ml = reinterpret_cast<float2*>(smem + kWaves * kSums) + wave * 64 + lane;
        tile_barrier();
        if (kg > 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    there[(4 * mt + i) * 64] = v4f{O[mt][4 * i], O[mt][4 * i + 1], O[mt][4 * i + 2], O[mt][4 * i + 3]};
            *ml = float2{m, l};
        }
        tile_barrier();
        if (kg > 0) return;
        float2 x[KG];
        x[0] = float2{m, l};
#pragma unroll
        for (int i = 1; i < KG; ++i) {
            x[i] = ml[i * RG * 64];
            m = fmaxf(m, x[i].x);
        }
        l = 0.f;
#pragma unroll
        for (int i = 0; i < KG; ++i) {
            x[i].x = __builtin_amdgcn_exp2f(x[i].x - m);
            l += x[i].y * x[i].x;
        }
#pragma unroll
        for (int e = 0; e < 4 * MT; ++e) {
            v4f o = v4f{O[e / 4][e % 4 * 4], O[e / 4][e % 4 * 4 + 1], O[e / 4][e % 4 * 4 + 2], O[e / 4][e % 4 * 4 + 3]} *
                    x[0].x;
#pragma unroll
            for (int i = 1; i < KG; ++i) o += there[i * RG * (kSums / 16) + e * 64] * x[i].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) O[e / 4][e % 4 * 4 + j] = o[j];
            if (e % 4 == 3) asm volatile("" : "+v"(O[e / 4]) : : "memory");   // (a block's reads at a time: registers)
        }
    }

    // ---- write: rows through LDS, so that a store takes whole ones ----
    l += __shfl_xor(l, 32, kWave);
    constexpr int kOutB = 2 * V + 16;
    unsigned char* rows_at = smem + rg * (KG > 1 ? MT * 4 * 64 * 16 : 32 * kOutB);
    static_assert(32 * kOutB <= MT * 4 * 64 * 16 && RG * 32 * kOutB <= kLds, "the rows fit the sums' or tiles' place");
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
    const int64_t first_row = out_row + (int64_t)(32 * rg) * a.H;
#pragma unroll
    for (int i = 0; i < VP / 2; ++i) {
        const int r = i * (64 / VP) + lane / VP, c = lane % VP;
        const v4i x = *reinterpret_cast<const v4i*>(rows_at + r * kOutB + 16 * c);
        if (32 * rg + r < rows) *reinterpret_cast<v4i*>(a.out + (first_row + (int64_t)r * a.H) * V + 8 * c) = x;
    }
    if (a.lse && h == 0 && 32 * rg + n < rows)
        a.lse[first_row + (int64_t)n * a.H] = l == 0.f ? -__builtin_inff() : (m + log2f(l)) * 0.693147180559945f;
}

int64_t blocks_of(int T, int B, int H, int rows) { return ((int64_t)T / rows + B + 1) * H; }

template <int D, int V, int RG, int KG, int NK>
hipError_t run(const PromptArgs& a, hipStream_t stream) {
    static PerDevice<int> once;
    constexpr int lds = lds_bytes<D, V, RG, KG, NK>();
    const hipError_t e = set_lds_limit(once, (const void*)prompt_attention_kernel<D, V, RG, KG, NK>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((prompt_attention_kernel<D, V, RG, KG, NK>),
                       dim3((unsigned)blocks_of(a.T, a.B, a.H, 32 * RG)), dim3(64 * RG * KG), lds, stream, a);
    return hipGetLastError();
}

// The form of a call, by about how many blocks of 64 and 128 rows there are (256 CUs
// hold 512 workgroups of four waves, 256 of eight) and the sequences' mean length, all
// that the host knows (rows of no sequence and empty sequences enter it, and it says
// little of very unequal ones: 8192 rows of one head take 68 us, beside 100 sequences
// of up to 5 rows 120):
// blocks of 64 rows and four key groups while each has a CU of its own, or two in a
// row where they are long; 128 rows and two key groups for up to two workgroups a
// CU; else 128 rows and one group, which with 64 and 128 columns and many sequences
// that are not long takes tiles of 32 keys: half of the scores in registers, 128 and
// 168 a lane, for four and three workgroups a CU (192 columns do not fit 168).
// Of 128 columns, in that order, us: 128 rows of 8 heads 7.9, 8.2, 7.9; 512 of 32
// 12.3, 14.0, 14.4; 512 of 40 17.1, 14.1, 14.5; 1024 of 32 23.8, 20.7, 22.4; 2048 of 8
// 23.5, 31.0, 36.5, of 16 32.1, 32.3, 36.9, of 32 62.4, 46.7, 48.2; 8192 of 1 65.8, 96.9,
// 121, of 4 90, 106, 125, of 8 174, 147, 169, of 12 264, 230, 226.
// Tiles of 64 and 32 keys, 128 columns: 64 sequences of 128 rows, 32 heads 46.0 and
// 39.6; 32 of 512, 32 heads 133 and 120; 16 of 1000, 4 heads 30.8 and 34.3, 8 heads 55.0
// and 55.0, 16 heads 93.2 and 87.8; 8 of 2048, 16 heads 158 and 154; 6 of 4096, 8 heads
// 206 and 220, 64 heads 1615 and 1583.  64 columns: 16 of 128, 32 heads 9.4 and 9.4, 64
// heads 16.7 and 13.7; 16 of 512, 8 heads 13.9 and 15.1; 32 of 512, 32 heads 73.3 and
// 68.8; 16 of 1000, 64 heads 214 and 214; one of 8192, 16 heads 168 and 178.
template <int D, int V>
hipError_t run(const PromptArgs& a, hipStream_t stream) {
    const int64_t mean = a.T / a.B;
    const int64_t narrow = (2 * ((int64_t)a.T / 64) + a.B) * a.H / 2, wide = (2 * ((int64_t)a.T / 128) + a.B) * a.H / 2;
    if ((narrow <= 300 && mean > 128) || (narrow <= 540 && mean >= 2048)) return run<D, V, 2, 4, 32>(a, stream);
    if (wide <= 560 && mean >= 512) return run<D, V, 4, 2, 64>(a, stream);
    if constexpr (D < 192)
        if (wide > 768 && mean <= (D == 64 ? 512 : 2048)) return run<D, V, 4, 1, 32>(a, stream);
    return run<D, V, 4, 1, 64>(a, stream);
}

}  // namespace

// At most floor(T / 128) whole blocks and a rest of each of the B sequences and of the rows behind them.
int64_t prompt_blocks(int T, int B, int H) { return blocks_of(T, B, H, 128); }

hipError_t launch_prompt_attention(const PromptArgs& a, int D, hipStream_t stream) {
    if (a.T <= 0) return hipSuccess;
    return D == 64 ? run<64, 64>(a, stream) : D == 128 ? run<128, 128>(a, stream) : run<192, 128>(a, stream);
}

}  // namespace dsaidx
