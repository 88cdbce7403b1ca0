// What the kernels share whose waves take the queries of one token as the 16
// columns of products (attend_token.hip, and attend_chunk.hip for sequences of
// one new token): a wave goes over 32 keys at a time, alone, with rows of K and
// then V in a tile of its own in LDS.
//
// Matrix instructions, 16 x 16 x 32: S^T = K Q^T puts a query in each lane
// (column) and four keys in its registers, so that the row statistics are per
// lane, and P^T is the second product's operand as it stands: O^T = V^T P^T
// sums over keys in any order, so the key of operand slot (lane group c, j) is
// 4c + j for j < 4 and 16 + 4c + j - 4 above, the keys that the lane holds.
// V^T comes from row-major V in LDS by transposing reads.
#pragma once
#include "serve_device.hpp"
#include "serve_internal.hpp"

namespace df11 {

// Where 16-byte chunk `chunk` of key row `row` lies in a wave's tile of 32
// rows.  The exclusive or puts what is read together into different banks of
// a 256-byte line.  K: 16 rows at one chunk.  V, by transposing reads of 16
// elements of a row: words, two chunks of rows 0 .. 7 (8 .. 15, ...); bytes,
// one chunk of rows 0 .. 7 and 16 .. 23 (8 .. 15 and 24 .. 31).
template <int kRowBytes>
__device__ __forceinline__ uint32_t column_k_at(uint32_t row, uint32_t chunk) {
    return row * kRowBytes + ((chunk ^ (row / (256 / kRowBytes) & (kRowBytes / 16 - 1))) << 4);
}
template <int kRowBytes, bool kInt8>
__device__ __forceinline__ uint32_t column_v_at(uint32_t row, uint32_t chunk) {
    uint32_t x;
    if (kInt8) x = kRowBytes == 128 ? (row >> 1 & 3) | (row >> 4 & 1) << 2 : (row >> 2 & 1) | (row >> 4 & 1) << 1;
    else x = kRowBytes == 256 ? (row & 7) << 1 : (row >> 1 & 3) << 1;
    return row * kRowBytes + ((chunk ^ x) << 4);
}

// The element of a row where operand i of lane group grp begins.  Words: step i
// holds d = 32 i + 8 grp ..; bytes: two steps share a 16-byte chunk, so steps 2t
// and 2t + 1 hold d = 64 t + 16 grp + 0 and 8 ..
template <bool kInt8>
__device__ __forceinline__ uint32_t column_operand_at(uint32_t i, uint32_t grp) {
    return kInt8 ? 64 * (i / 2) + 16 * grp + 8 * (i % 2) : 32 * i + 8 * grp;
}

// Scores of two times 16 keys: the lane has keys 16 t + 4 grp + i of query col.
// query(i): operand i.
template <int D, bool kInt8, class Query>
__device__ __forceinline__ void column_scores(const uint8_t *tile, uint32_t lane, const Query &query, f32x4 (&s)[2]) {
    constexpr int kRow = kInt8 ? D : 2 * D, kChunks = kRow / 16;
    const uint32_t col = lane & 15u, grp = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kChunks / 4; ++i) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(tile + column_k_at<kRow>(16 * t + col, 4 * i + grp));
            if (kInt8) {
                s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(bf16_of_bytes8(u32x2{w.x, w.y})), as_bf16x8(query(2 * i)), s[t], 0, 0, 0);
                s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(bf16_of_bytes8(u32x2{w.z, w.w})), as_bf16x8(query(2 * i + 1)), s[t], 0, 0, 0);
            } else {
                s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(query(i)), s[t], 0, 0, 0);
            }
        }
    }
}

// Takes the step's scores (times `scale`, in base 2) and its values into the
// maximum, the sum and the accumulators.
template <int D, bool kInt8>
__device__ __forceinline__ void column_update(const uint8_t *tile, uint32_t lane, const f32x4 (&s)[2], const f32x4 (&v_scale)[2], float scale,
                                              float log2_n, f32x4 (&o)[D / 16], float &m, float &l) {
    constexpr int kRow = kInt8 ? D : 2 * D, kDTiles = D / 16;
    const uint32_t grp = lane >> 4;
    float top = -__builtin_inff();
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][i]);
    f32x2 two = with_lane_16(top);
    two = with_lane_32(fmaxf(two.x, two.y));
    top = fmaxf(two.x, two.y) * scale;
    if (__any(top > m - log2_n)) {
        const float next = fmaxf(m, top + (kSlack + log2_n));
        const float keep = exp2_fast(m - (next == -__builtin_inff() ? 0.0f : next));
        m = next;
        l *= keep;
#pragma unroll
        for (int i = 0; i < kDTiles; ++i) o[i] *= keep;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
    // weights as the sum of two operands, for the product has matrix rate to
    // spare: rounded once they would add as much error as the rounding of the
    // result (0.0027 of the norm against 0.0017)
    u32x4 p, p_low;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            e[i] = exp2_fast(__builtin_fmaf(s[t][i], scale, -base));
            l += e[i];
            if (kInt8) e[i] *= v_scale[t][i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x2 two = two_operands<kInt8>(e[2 * i], e[2 * i + 1]);
            p[2 * t + i] = two.x;
            p_low[2 * t + i] = two.y;
        }
    }
#pragma unroll
    for (int i = 0; i < kDTiles; ++i) {
        u32x4 w;
        if (kInt8) {
            // 8 rows x 16 bytes a transposing read: rows of the lane's slots are
            // 4 grp + 0..3 and 16 + 4 grp + 0..3
            const uint32_t j = lane & 15u, r = j >> 1;
            const uint32_t row = (r < 4 ? 0 : 12) + 4 * grp + r;
            const i32x2 b = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (DF11_LDS i32x2 *)(tile + column_v_at<kRow, kInt8>(row, i) + 8 * (j & 1)));
            w = bf16_of_bytes8(u32x2{(uint32_t)b.x, (uint32_t)b.y});
        } else {
            const uint32_t j = lane & 15u, row = 4 * grp + (j >> 2), chunk = 2 * i + ((j & 3) >> 1);
            const s16x4 b0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(tile + column_v_at<kRow, kInt8>(row, chunk) + 8 * (j & 1)));
            const s16x4 b1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(tile + column_v_at<kRow, kInt8>(row + 16, chunk) + 8 * (j & 1)));
            const u32x2 w0 = __builtin_bit_cast(u32x2, b0), w1 = __builtin_bit_cast(u32x2, b1);
            w = u32x4{w0.x, w0.y, w1.x, w1.y};
        }
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(p), o[i], 0, 0, 0);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(p_low), o[i], 0, 0, 0);
    }
}

}  // namespace df11
