// Tiles of rows in LDS that are filled straight from memory, without passing
// registers, and read as operands of 16x16 matrix products.
#pragma once

#include "gdn_mla.hpp"

namespace gdn {

// Rows of RU 16-byte units for KS steps of 32 columns, unit u of row j at place
// u ^ (j & XM) of its row, so that what a read takes of eight (sixteen) rows at
// once lies in different banks without padding (a load to LDS leaves no gaps).
template <bool BF, int KS> struct LdsTile {
    static constexpr int V = Op<BF>::VEC, RU = (32 * KS / V + 7) / 8 * 8, XM = RU % 16 ? 7 : 15;
};

// Sixteen bytes of every lane from global memory to 64 units of LDS that follow each other
// (dst, the same for all lanes). Counted as a vector memory load: a wait for
// those and a barrier make it visible. Written by hand, since the compiler would
// have every LDS read behind it wait for it, the other tile's as well. (m0: the compiler
// keeps nothing there, it writes it before each use of its own, of which there are none here.)
__device__ __forceinline__ void load_to_lds(const void *src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(src)
                 : "memory");
}
// where a place in LDS is, as load_to_lds takes it
__device__ __forceinline__ uint32_t lds_place(const u32x4 *p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u32x4 *)p);
}

// Where a lane reads its operands in a tile: u ^ x for units u that differ by
// constants is a constant away from one of a few places, so those are formed once
// and every read has its distance in the instruction.
template <class P> struct TileReads {
    // steps of the rows' units (two bits of a unit choose the lane group, bf16), of the columns'
    static constexpr bool BF = P::V == 8;
    static constexpr int RB = BF ? (P::XM + 1) / 4 : (P::XM + 1) / 8, CB = BF ? (P::XM + 1) / 2 : (P::XM + 1) / 4;
    int row[RB][BF ? 1 : 2], col[CB][BF ? 1 : 4]; // bytes
    __device__ __forceinline__ void init(int lane) {
        const int r = lane & 15, g = lane >> 4, x = r & P::XM;
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
            for (int h = 0; h < (BF ? 1 : 2); ++h)
                row[k][h] = 16 * (r * P::RU + ((BF ? 4 * k + g : 8 * k + 2 * g + h) ^ x));
#pragma unroll
        for (int v = 0; v < CB; ++v)
#pragma unroll
            for (int e = 0; e < (BF ? 1 : 4); ++e) {
                const int j = BF ? 4 * g + (r >> 2) : 4 * g + e, y = j & P::XM;
                const int u = BF ? 2 * v + (r >> 1 & 1) : 4 * v + (r >> 2);
                col[v][e] = 16 * (j * P::RU + (u ^ y)) + (BF ? 8 * (r & 1) : 4 * (r & 3));
            }
    }
    // eight values of row j0 + lane % 16 (j0 a multiple of 16) in step k of 32 columns
    __device__ __forceinline__ Frag<BF> rows(const u32x4 *T, int j0, int k) const {
        const char *p = (const char *)(T + j0 * P::RU + k / RB * RB * (BF ? 4 : 8));
        if constexpr (BF) return {*reinterpret_cast<const bf16x8 *>(p + row[k % RB][0])};
        else return {*reinterpret_cast<const f32x4 *>(p + row[k % RB][0]), *reinterpret_cast<const f32x4 *>(p + row[k % RB][1])};
    }
    // operand column 16 v + lane % 16 over the 32 rows from j0, in the K order of two accumulator tiles (as col8)
    __device__ __forceinline__ Frag<BF> cols(const u32x4 *T, int j0, int v) const {
        const char *p = (const char *)(T + j0 * P::RU + v / CB * CB * (BF ? 2 : 4));
        if constexpr (BF) {
            auto half = [&](int j) {
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(p + j * P::RU * 16 + col[v % CB][0]));
            };
            return {join8(half(0), half(16))};
        } else {
            Frag<false> f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f.lo[e] = *reinterpret_cast<const float *>(p + col[v % CB][e]);
                f.hi[e] = *reinterpret_cast<const float *>(p + 16 * P::RU * 16 + col[v % CB][e]);
            }
            return f;
        }
    }
};

} // namespace gdn
