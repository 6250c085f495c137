// What the kernels of attention over the paged latent cache share: the tile's
// layout in LDS, the copies into it, and the walk over a query's keys.
#pragma once

#include "common.h"
#include "latent.h"

namespace dsaidx {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v2i lds_v2i;

constexpr int kLatentPage = 64;
constexpr int kTile = 64;      // keys of a tile
constexpr int kV = 512;        // value columns of a row
constexpr float kSlack = 16.f; // a softmax reference moves when a score passes it by 2^kSlack

// A tile in LDS, bf16.  The 64 banks serve 16 lanes of a 16-byte read at once
// (lanes 0-3, 12-15 and 20-27 are one such group, 4-11, 16-19 and 28-31 the
// next), 32 lanes of an 8-byte one.  A row is its 512 value columns padded by
// 32 bytes: consecutive rows start 8 banks apart, and both an operand read (16
// rows, lane groups 16 bytes apart) and a transposed one (8 rows of 32 bytes)
// use every bank once: 235 bytes a clock and CU against 127 with a padding of
// 16.  The rotary columns lie behind, 128 bytes a row, their 16-byte pieces
// permuted within the row.
constexpr int kRowB = 2 * kV + 32;
constexpr int kMainB = kTile * kRowB;
constexpr int kRopeB = kTile * 128;
constexpr int kTileB = kMainB + kRopeB;

// What an entry without a row is copied from.
static __device__ __align__(16) const unsigned char kZeroRow[1152] = {};

struct LatentPlan {
    int rows;              // query rows of a workgroup
    int n_prefix, n_own;   // workgroups of each part (multiples of 8)
    int rb;                // prefix: row blocks of all T * H rows
    int sp, lp;            // prefix: splits, tiles of a split
    int hb;                // own keys or selection: row blocks of one query's H rows
    int so, lo;            //   splits, tiles of a split
    int joint;             //   prefix tiles in front of the own ones (no prefix part)
    int slots;             // partial results per row (1: written directly)
    float* part_o;         // [slots][T * H][V]
    float2* part_ml;       // [slots][T * H] (maximum, sum)
};

// Workgroup barrier that waits for this wave's LDS accesses only: the copies
// in flight are waited for by vmcnt where their tile is needed.
__device__ __forceinline__ void tile_barrier() {
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
// The same, 4 bytes per lane.
__device__ __forceinline__ void copy4_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory");
}

// Eight E4M3 codes -> eight bf16 (exact).
__device__ __forceinline__ v4i widen8(uint2 c) {
    return v4i{(int)fp8x2_to_bf16x2<false>((int)c.x), (int)fp8x2_to_bf16x2<true>((int)c.x),
               (int)fp8x2_to_bf16x2<false>((int)c.y), (int)fp8x2_to_bf16x2<true>((int)c.y)};
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char*)p;
}

// The keys of a workgroup's rows: tiles t0 .. t1-1 of 64 entries.  Lane i
// holds entry i of a tile.  While a tile is computed the next one is copied,
// the rows of the one behind it are found (resolve), and page ids and entries
// of the next two are loads in flight (LatentAhead).
struct LatentAhead {
    int s2, page2;   // entries and page ids of the tile behind the resolved one,
    int s3;          // entries of the next
};

template <bool TOPK>
struct LatentKeys {
    int r0, nrows, slot;            // query rows (of T * H), place of their results
    int t0, t1;
    const int32_t* table;           // pages of the own positions or the selection's
    const int32_t* idx;             // the selection
    int len;                        // own positions, or entries of the selection
    const int32_t* ptable;          // pages of the prefix
    int tp, plen;                   // tiles and positions of the prefix in front
    int max_pages, num_pages;
    int lane;
    int row;                        // the resolved tile's rows of the pool, -1: no row,
    uint64_t mask;                  // and which entries have one

    // Workgroups go to the 8 XCDs in turn; the ones that read the same keys
    // follow each other on one XCD.
    __device__ __forceinline__ bool start(const LatentArgs& a, const LatentPlan& p) {
        lane = lane_id();
        max_pages = a.max_pages;
        num_pages = a.num_pages;
        row = -1;
        mask = 0;
        idx = nullptr;
        ptable = a.prefix_table;
        const int id = blockIdx.x;
        if (!TOPK && id < p.n_prefix) {
            const int w = (id & 7) * (p.n_prefix >> 3) + (id >> 3);
            slot = w / p.rb;
            if (slot >= p.sp) return false;
            r0 = (w % p.rb) * p.rows;
            nrows = min(p.rows, a.T * a.H - r0);
            table = nullptr;
            len = 0;
            plen = a.prefix_len;
            tp = (plen + kTile - 1) / kTile;
            t0 = slot * p.lp;
            t1 = min(t0 + p.lp, tp);
            return true;
        }
        const int id2 = id - p.n_prefix;
        const int w = (id2 & 7) * (p.n_own >> 3) + (id2 >> 3);
        const int q = w / (p.hb * p.so), s = w / p.hb % p.so, h = w % p.hb * p.rows;
        if (q >= a.T) return false;
        r0 = q * a.H + h;
        nrows = min(p.rows, a.H - h);
        slot = p.sp + s;
        t0 = s * p.lo;
        tp = plen = 0;
        if constexpr (TOPK) {
            const int b = a.seq_ids ? a.seq_ids[q] : q;
            const bool ok = b >= 0 && b < a.B;
            table = a.block_table + (int64_t)(ok ? b : 0) * a.max_pages;
            idx = a.idx + (int64_t)q * a.K;
            len = a.K;   // (known before b is, so that the first entries' loads do not wait for it)
            if (!ok) max_pages = 0;
        } else {
            table = a.block_table + (int64_t)q * a.max_pages;
            len = min(max(a.context_lens[q], 0), a.max_ctx);
            if (p.joint) {
                plen = a.prefix_len;
                tp = (plen + kTile - 1) / kTile;
            }
        }
        t1 = min(t0 + p.lo, tp + (len + kTile - 1) / kTile);
        return true;
    }

    // Position of entry `lane` of tile t, -1: none.
    __device__ __forceinline__ int entry(int t) const {
        if constexpr (TOPK) {
            const int j = t * kTile + lane;
            return j < len ? idx[j] : -1;
        }
        const int j = (t < tp ? t : t - tp) * kTile + lane;
        return j < (t < tp ? plen : len) ? j : -1;
    }
    // The same, where `s` was loaded earlier; own and prefix positions are not worth keeping.
    __device__ __forceinline__ int entry_of(int t, int s) const {
        if constexpr (TOPK) return s;
        return entry(t);
    }
    __device__ __forceinline__ int page(int s, int t) const {
        if constexpr (TOPK) return s >= 0 && s / kLatentPage < max_pages ? table[s / kLatentPage] : -1;
        int zero;   // keeps this load among the vector loads, which the waits in the tile loop count on
        asm volatile("v_mov_b32 %0, 0" : "=v"(zero));
        return t < t1 ? (t < tp ? ptable + t : table + (t - tp))[zero] : -1;
    }
    __device__ __forceinline__ void resolve(int s, int page) {
        const bool ok = s >= 0 && page >= 0 && page < num_pages;
        mask = wave_ballot(ok);
        row = ok ? page * kLatentPage + (s & (kLatentPage - 1)) : -1;
    }
    // First tile at or behind t with a row, resolved, and what is ahead of it; t1: none.
    __device__ __forceinline__ int seek(int t, LatentAhead& ahead) {
        int s = entry(t);
        LatentAhead h;
        h.s2 = entry(t + 1);
        h.s3 = entry(t + 2);
        resolve(-1, -1);
        for (;;) {
            const int id = page(s, t);
            h.page2 = page(h.s2, t + 1);
            if (t >= t1) break;
            resolve(s, id);
            if (mask) break;
            ++t;
            s = h.s2;
            h.s2 = h.s3;
            h.s3 = entry(t + 2);
        }
        ahead = h;
        return t;
    }
};

// Address of a row of RB bytes; an entry without a row takes a row of zeros:
// its probability is zero, and zero its values must be.
template <int RB>
__device__ __forceinline__ const unsigned char* row_address(const void* cache, int row) {
    const unsigned char* base = row >= 0 ? reinterpret_cast<const unsigned char*>(cache) : kZeroRow;
    return base + (uint64_t)(uint32_t)max(row, 0) * RB;   // (no branch)
}
// A 64-bit value of lane `lane`, as a scalar pointer.
__device__ __forceinline__ const unsigned char* lane_pointer(uint64_t p, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)p, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(p >> 32), lane);
    return reinterpret_cast<const unsigned char*>((uint64_t)hi << 32 | lo);
}
// fp8 rows: the exponents' references are raised by log2 of the scale of the
// run's first row, so that probabilities are rounded to bf16, after the product
// with their rows' scales, in units of it.  A run of one row, or of rows of one
// scale, then rounds only probabilities: the scale's own rounding, which all the
// heads would share, stays out.  The sums have the same reference, and the
// exponents the shift's length: at a scale of 2^-20 a part's lse is off by some
// 2^-19 more than scores alone would make it, at 2^-7 by 2^-21.
template <bool TOPK>
__device__ __forceinline__ float scale_shift(const LatentKeys<TOPK>& keys, const float* scales) {
    if (keys.mask == 0) return 0.f;
    const float s = fabsf(scales[__builtin_amdgcn_readlane(keys.row, __builtin_ctzll(keys.mask))]);
    const float shift = s >= 0x1p-40f && s <= 0x1p40f ? __builtin_amdgcn_logf(s) : 0.f;
    return __int_as_float(uniform(__float_as_int(shift)));
}
// Scores times the softmax's scale, rounded before their maximum is taken off
// them: of a product left whole (in an fma), scores past 2^31 would keep more
// than 2^7 that their maximum, rounded, has not, and 2 to that is infinite.
__device__ __forceinline__ v4f scaled_scores(v4f s, float scale) {
#pragma clang fp contract(off)
    return s * scale;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
}

// Blocks of 64 and 128 query rows (csrc/latent_rows.hip).
hipError_t launch_latent_rows(const LatentArgs& a, const LatentPlan& p, bool fp8, hipStream_t stream);

}  // namespace dsaidx
