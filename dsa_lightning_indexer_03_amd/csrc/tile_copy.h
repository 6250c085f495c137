// What the attention kernels share: copies straight into LDS, the barrier that
// does not wait for them, fp8 codes and probabilities as bf16 operands.
#pragma once

#include "common.h"

namespace dsaidx {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v2i lds_v2i;

constexpr float kSlack = 16.f;  // a softmax reference moves when a score passes it by 2^kSlack

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

}  // namespace dsaidx
