// entq_int8_tile.h -- what the tiled products share: direct global-to-LDS
// loads of 128-byte row pieces and the order of a grid's tiles.
#pragma once

#include "entq_int8.h"

namespace entq {

// LDS rows of the tiles are 128 bytes: 8 chunks of 16, chunk c of row r at
// position c ^ swizzle(r). A row fills half of the 64 banks; 16 consecutive
// rows read at one chunk, which ds_read_b128 takes at once, touch every bank
// once (with c ^ (r & 7) the counters showed half of all LDS cycles lost to
// conflicts).
constexpr uint32_t kRowBytes = 128;
__device__ __forceinline__ uint32_t swizzle(uint32_t row) { return row / 2 % 8; }

// One 16-byte load per active lane from base + offset straight into LDS at
// lds + 16 lane. The compiler does not
// count this load; wait_loads_and_meet() does. (s_nop: a written m0 needs one
// wait state before such a load.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const void *base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// All loads of this wave but the last N have landed and every LDS read of it
// is done; then all waves of the workgroup are here.
template <int N>
__device__ __forceinline__ void wait_loads_and_meet() {
    static_assert(N >= 0 && N < 64, "");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void *p) { return (uint32_t)(uintptr_t)p; }

__device__ __forceinline__ v4i read_lds16(uint32_t at) {
    return *(const __attribute__((address_space(3))) v4i *)(uintptr_t)at;
}

// Workgroup `id` of a grid of nb_a x nb_b tiles (a: tokens) -> its tile.
// Workgroups go to the 8 XCDs in turn; each XCD takes one contiguous piece of
// the tiles, in bands of kBand tiles along a, so that the 32 tiles of 256
// tokens that it runs together form a block of 4 x 8 and share their operands
// in its L2. Measured with bands of 2, 4, 8 and 16 (us): gated 4096 x 28672 x
// 8192 1573, 1555, 1587, 1627, product 4096 x 8192 x 28672 767, 758, 764, 773.
constexpr uint32_t kBand = 4;
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t nb_a, uint32_t nb_b, uint32_t &ta, uint32_t &tb) {
    const uint32_t total = nb_a * nb_b, xcd = id % 8, i = id / 8;
    const uint32_t q = total / 8, r = total % 8;
    const uint32_t t = xcd * q + min(xcd, r) + i;
    const uint32_t group = t / (kBand * nb_b), first = group * kBand;
    const uint32_t in = min(kBand, nb_a - first), rest = t - group * kBand * nb_b;
    ta = first + rest % in;
    tb = rest / in;
}

}  // namespace entq
