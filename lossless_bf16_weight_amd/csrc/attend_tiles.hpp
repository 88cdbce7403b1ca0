// What the two attention kernels over tiles of rows share (attend_prompt.hip,
// attend_chunk.hip): where a step's keys and values lie in LDS, and how a
// tile's results are written.
//
// The queries of the heads that share a kv head are the rows of one matrix:
// row r is query r / group of head r % group.  A workgroup takes kPromptTile of
// them, a wave 32, and steps over the keys kPromptKeys at a time.
#pragma once
#include "serve_device.hpp"
#include "serve_internal.hpp"

namespace df11 {

// The K and V tiles in LDS: 16-byte chunk `chunk` of key row `row` lies at
// place k_chunk (v_chunk) of its row, and the other way round.  K: 32 rows are
// read at one chunk a time; V: four neighbouring rows, 32 bytes of each, by a
// transposing read.  The exclusive or puts them into different banks.
template <int D>
__device__ __forceinline__ uint32_t k_chunk(uint32_t row, uint32_t chunk) {
    return D == 128 ? chunk ^ (row & 15) : chunk ^ ((row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ uint32_t v_chunk(uint32_t row, uint32_t chunk) {
    return D == 128 ? chunk ^ ((row & 3) << 2) : chunk ^ (((row >> 1) & 1) << 2);
}
template <int D>
__device__ __forceinline__ uint32_t k_at(uint32_t row, uint32_t chunk) {
    return row * (2 * D) + (k_chunk<D>(row, chunk) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t chunk) {
    return row * (2 * D) + (v_chunk<D>(row, chunk) << 4);
}

// Size of the K and V descriptors, and an offset that is outside (the host
// keeps a tile's rows within it).
constexpr uint32_t kOutOfRange = 0x80000000u;

// row / group (the host gives the multiplier, exact below 2^31).
template <class Args>
__device__ __forceinline__ uint32_t over_group(const Args &a, uint32_t row) {
    return a.group == 1 ? row : __umulhi(row, a.group_magic) >> a.group_shift;
}

// Writes 16 of a product's 32 rows as BF16, the lane's column to 16 words from
// `to`.  The lane has four of each eight neighbours (a, then b), the lane 32
// away the others: they exchange halves and write eight each.
__device__ __forceinline__ void store_16(f32x4 a, f32x4 b, uint16_t *to, uint32_t half, bool real) {
    uint32_t w[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const auto r = __builtin_amdgcn_permlane32_swap(pack_bf16(a[2 * x], a[2 * x + 1]), pack_bf16(b[2 * x], b[2 * x + 1]), false, false);
        w[0][x] = r[0];
        w[1][x] = r[1];
    }
    if (real) *reinterpret_cast<u32x4 *>(to + 8 * half) = u32x4{w[0][0], w[0][1], w[1][0], w[1][1]};
}

// All 32 rows.  (The same steps: through store_16 attend_prompt's kernels came
// out otherwise.)
__device__ __forceinline__ void store_tile(const f32x16 &o, uint16_t *to, uint32_t half, bool real) {
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
        uint32_t w[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const auto r = __builtin_amdgcn_permlane32_swap(pack_bf16(o[4 * g + 2 * x], o[4 * g + 2 * x + 1]),
                                                            pack_bf16(o[4 * g + 4 + 2 * x], o[4 * g + 5 + 2 * x]), false, false);
            w[0][x] = r[0];
            w[1][x] = r[1];
        }
        if (real) *reinterpret_cast<u32x4 *>(to + 8 * (g + half)) = u32x4{w[0][0], w[0][1], w[1][0], w[1][1]};
    }
}

}  // namespace df11
