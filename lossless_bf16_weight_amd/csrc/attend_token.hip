// Attention of one new token of each sequence over the paged cache, for
// gfx950.
//
// For query head h of kv head h / group: s_j = <q, k_j>, p_j = 2^(c s_j - m)
// with c = scale log2(e) and m the running maximum of c s_j (and a constant:
// see kSlack), out = sum p_j v_j / sum p_j.  One pass over the keys: when a
// step raises m, the sums are scaled by 2^(old - new).  Keys in 8 bits keep their codes as exact BF16
// operands: a key's scale multiplies its score, a value's scale its weight.
//
// Every key and value is read once and used by `group` queries, so HBM
// traffic bounds it.  A workgroup takes up to `range` keys of one kv head
// (work along a long sequence is split over workgroups, and a second kernel
// joins the parts); its four waves (twelve, where they take a sequence whole)
// take 32 keys a step in turn, each with its own maximum, sum and
// accumulators, joined through LDS at the end.  Each wave holds the next step's
// keys and values in registers, 16 KB of them for words of head_dim 128, and
// three workgroups of four waves run on a compute unit at a time: 192 KB of
// loads in flight there (half in 8 bits; head_dim 64 has half for each wave and
// registers for five waves a SIMD).  LDS only turns a wave's own rows around (a
// wave waits for no other until the end).
//
// Measured with 32 heads over 8 kv heads of 128, join included: 64 sequences
// of up to 4096 tokens 94 us (505 MB, 5.6 TB/s in the first kernel's 90 us),
// two of up to 100,001 tokens 84 us (440 MB, 5.5 TB/s in 80), 48 of up to
// 16,384 in 8 bits 139 us (734 MB, 5.3 TB/s).  A read of the same bytes with
// nothing computed reaches 6.6 TB/s.  With heads of 64 the same take 53, 48 and
// 82 us for half the bytes (4.6 to 4.7 TB/s).
//
// Matrix instructions, 16 x 16 x 32: S^T = K Q^T puts a query in each lane
// (column) and four keys in its registers, so that the row statistics are per
// lane, and P^T is the second product's operand as it stands: O^T = V^T P^T
// sums over keys in any order, so the key of operand slot (lane group c, j) is
// 4c + j for j < 4 and 16 + 4c + j - 4 above, the keys that the lane holds.
// V^T comes from row-major V in LDS by transposing reads.
#include "serve_device.hpp"
#include "serve_internal.hpp"

namespace df11 {

namespace {

constexpr uint32_t kMostPages = (kTokenRangeMax > kTokenWholeMax ? kTokenRangeMax : kTokenWholeMax) / 16;

// Where 16-byte chunk `chunk` of key row `row` lies in a wave's tile of 32
// rows.  The exclusive or puts what is read together into different banks of
// a 256-byte line.  K: 16 rows at one chunk.  V, by transposing reads of 16
// elements of a row: words, two chunks of rows 0 .. 7 (8 .. 15, ...); bytes,
// one chunk of rows 0 .. 7 and 16 .. 23 (8 .. 15 and 24 .. 31).
template <int kRowBytes>
__device__ __forceinline__ uint32_t k_at(uint32_t row, uint32_t chunk) {
    return row * kRowBytes + ((chunk ^ (row / (256 / kRowBytes) & (kRowBytes / 16 - 1))) << 4);
}
template <int kRowBytes, bool kInt8>
__device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t chunk) {
    uint32_t x;
    if (kInt8) x = kRowBytes == 128 ? (row >> 1 & 3) | (row >> 4 & 1) << 2 : (row >> 2 & 1) | (row >> 4 & 1) << 1;
    else x = kRowBytes == 256 ? (row & 7) << 1 : (row >> 1 & 3) << 1;
    return row * kRowBytes + ((chunk ^ x) << 4);
}

// kOnce: no other workgroup reads the same rows (at most 16 heads share a kv head).
template <int D, bool kInt8, uint32_t kWaves, bool kOnce>
__global__ __launch_bounds__(64 * kWaves, 3) void attend_token_kernel(TokenArgs a) {
    constexpr uint32_t kThreads = 64 * kWaves;
    constexpr int kRow = kInt8 ? D : 2 * D;            // bytes of a stored row
    constexpr int kChunks = kRow / 16;                 // 16-byte chunks of it
    constexpr int kLoads = kTokenKeys * kChunks / 64;  // chunks a lane loads of a step's K rows, and of its V rows
    constexpr int kDTiles = D / 16;
    constexpr int kOStride = D + 4;
    constexpr uint32_t kTileBytes = kTokenKeys * kRow;
    constexpr uint32_t kJoinBytes = kWaves * 16 * kOStride * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * kTileBytes > kJoinBytes ? kWaves * kTileBytes : kJoinBytes];
    __shared__ uint32_t table[kMostPages];
    __shared__ float ml[kWaves][2][16];
    __shared__ u32x4 q[D / 32][64];

    const uint32_t lane0 = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = lane0, col = lane & 15u, grp = lane >> 4;
    // (a kv head's tiles of 16 queries go to one XCD, eight workgroups apart,
    // so that the second finds the first one's rows in its L2)
    const uint32_t block = blockIdx.x / (8 * a.q_tiles), in_block = blockIdx.x % (8 * a.q_tiles);
    const uint32_t q_tile = in_block / 8, unit = 8 * block + in_block % 8;
    if (unit >= a.n_seqs * a.c.kv_heads) return;
    const uint32_t kv_head = unit % a.c.kv_heads, seq = unit / a.c.kv_heads;
    const uint32_t split = blockIdx.z * gridDim.y + blockIdx.y;     // (past the last: begins past every length)

    const uint32_t len = (uint32_t)min((int64_t)max(a.lens[seq], 0), (int64_t)a.t.width << a.c.shift);
    const uint32_t begin = split * a.range;
    if (begin >= len && split) return;
    const uint32_t n = min(len - begin, a.range);      // this workgroup's keys

    // the first row of this head in each page of the range (the host keeps the
    // number of rows below 2^32)
    const int32_t *const pages = a.t.pages + seq * a.t.stride + (begin >> a.c.shift);
    for (uint32_t i = threadIdx.x; i < ((n + (1u << a.c.shift) - 1) >> a.c.shift); i += kThreads)
        table[i] = (min((uint32_t)pages[i], a.c.n_pages - 1) * a.c.kv_heads + kv_head) << a.c.shift;

    // queries: columns past the group are zero
    const uint32_t in_group = q_tile * 16 + col;
    const uint32_t head = kv_head * a.group + in_group;
    const bool real = in_group < a.group;
    // (in LDS, in the order of the operands' lanes, for the registers are full)
    for (uint32_t i = wave; i < D / 32; i += kWaves) {
        // words: step i holds d = 32 i + 8 grp ..; bytes: two steps share a
        // 16-byte chunk, so steps 2t and 2t + 1 hold d = 64 t + 16 grp + 0 and 8 ..
        const uint32_t d = kInt8 ? 64 * (i / 2) + 16 * grp + 8 * (i % 2) : 32 * i + 8 * grp;
        u32x4 w = {0, 0, 0, 0};
        if (real) w = *reinterpret_cast<const u32x4 *>(a.q.data + seq * a.q.row + head * a.q.head + d);
        q[i][lane] = w;
    }
    __syncthreads();

    f32x4 o[kDTiles];
#pragma unroll
    for (int i = 0; i < kDTiles; ++i) o[i] = f32x4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0;
    const float log2_n = log2_up(len);      // (of the sequence: its parts are joined)
    uint8_t *const tile = lds + wave * kTileBytes;

    // A step's 32 rows of K and V, held in registers from one step before:
    // the loads of the next step are in flight while this one is computed.
    // Each half of them, 16 rows, lies in one page, whole lines that nobody
    // reads again; the wave's tile in LDS, first K's and then V's, hands them
    // to the lanes that compute.  Rows past the end are what the page holds
    // (their scores are masked, their V rows cleared below), halves past the
    // end repeat the last one.
    u32x4 kw[kLoads], vw[kLoads];
    f32x4 ks[2], vs[2];
    uint32_t half_row[2];
    const uint32_t in_page = (1u << a.c.shift) - 1, last_half = (n - 1) & ~15u;
    const auto find_rows = [&](uint32_t key0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t key = min(key0 + 16 * t, last_half);
            half_row[t] = __builtin_amdgcn_readfirstlane(table[key >> a.c.shift] + (key & in_page));
        }
    };
    const auto load = [&](const uint8_t *pages, u32x4 *w) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const u32x4 *const half = reinterpret_cast<const u32x4 *>(pages + (uint64_t)half_row[2 * i / kLoads] * kRow);
            const u32x4 *const from = half + i % (kLoads / 2) * 64 + lane;
            w[i] = kOnce ? __builtin_nontemporal_load(from) : *from;
        }
    };
    // LDS keeps a wave's accesses in order; this keeps the compiler's.
    const auto handed_over = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
    };
    const auto load_scales = [&] {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            ks[t] = reinterpret_cast<const f32x4 *>(a.c.k_scale + half_row[t])[grp];
            vs[t] = reinterpret_cast<const f32x4 *>(a.c.v_scale + half_row[t])[grp];
        }
    };
    uint32_t key0 = wave * kTokenKeys;
    if (key0 < n) {
        find_rows(key0);
        load(a.c.k, kw);
        load(a.c.v, vw);
        if (kInt8) load_scales();
    }
    for (; key0 < n; key0 += kWaves * kTokenKeys) {
        // (the tile's addresses are computed anew in each step: kept in
        // registers over the loop they would cost a wave of occupancy)
        uint32_t lane = lane0;
        asm volatile("" : "+v"(lane));
        const uint32_t col = lane & 15u, grp = lane >> 4;
        handed_over();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t at = i * 64 + lane;
            *reinterpret_cast<u32x4 *>(tile + k_at<kRow>(at / kChunks, at % kChunks)) = kw[i];
        }
        handed_over();
        find_rows(key0 + kWaves * kTokenKeys);      // (past the end: loads that nobody uses)
        load(a.c.k, kw);
        __builtin_amdgcn_sched_barrier(0);     // (loads of V moved up past here would not fit in registers)
        // scores of two times 16 keys: lane has keys 16 t + 4 grp + i of query col
        f32x4 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kChunks / 4; ++i) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(tile + k_at<kRow>(16 * t + col, 4 * i + grp));
                if (kInt8) {
                    s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(bf16_of_bytes8(u32x2{w.x, w.y})), as_bf16x8(q[2 * i][lane]), s[t], 0, 0, 0);
                    s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(bf16_of_bytes8(u32x2{w.z, w.w})), as_bf16x8(q[2 * i + 1][lane]), s[t], 0, 0, 0);
                } else {
                    s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(q[i][lane]), s[t], 0, 0, 0);
                }
            }
        }
        if (key0 + kTokenKeys > n) {
            // weights of rows past the end are 0, and 0 times an infinity would be NaN
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (key0 + (i * 64 + lane) / kChunks >= n) vw[i] = u32x4{0, 0, 0, 0};
        }
        handed_over();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t at = i * 64 + lane;
            *reinterpret_cast<u32x4 *>(tile + v_at<kRow, kInt8>(at / kChunks, at % kChunks)) = vw[i];
        }
        handed_over();
        load(a.c.v, vw);
        f32x4 v_scale[2];
        if (kInt8) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                s[t] *= ks[t] * a.log2_scale;
                v_scale[t] = vs[t];
            }
            load_scales();
        }
        const float scale = kInt8 ? 1.0f : a.log2_scale;
        if (key0 + kTokenKeys > n) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (key0 + 16 * t + 4 * grp + i >= n) {
                        s[t][i] = -__builtin_inff();
                        if (kInt8) v_scale[t][i] = 0;
                    }
        }
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
        // weights as the sum of two BF16 operands, for the product has matrix
        // rate to spare: rounded once they would add as much error as the
        // rounding of the result (0.0027 of the norm against 0.0017).  The
        // first is the BF16 number before the one that the weight begins with:
        // what is left for the second is then above zero and within 2^-14 of
        // the weight as a BF16, and a value that is infinite times both is
        // that infinity (times 0 or less it would make the result NaN).
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
                const uint32_t cut = __float_as_uint(e[2 * i]) >> 16 | (__float_as_uint(e[2 * i + 1]) & 0xFFFF0000u);
                const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, cut), u16x2{1, 1}));
                p[2 * t + i] = w;
                p_low[2 * t + i] = pack_bf16(e[2 * i] - __uint_as_float(w << 16), e[2 * i + 1] - __uint_as_float(w & 0xFFFF0000u));
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
                    (DF11_LDS i32x2 *)(tile + v_at<kRow, kInt8>(row, i) + 8 * (j & 1)));
                w = bf16_of_bytes8(u32x2{(uint32_t)b.x, (uint32_t)b.y});
            } else {
                const uint32_t j = lane & 15u, row = 4 * grp + (j >> 2), chunk = 2 * i + ((j & 3) >> 1);
                const s16x4 b0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(tile + v_at<kRow, kInt8>(row, chunk) + 8 * (j & 1)));
                const s16x4 b1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(tile + v_at<kRow, kInt8>(row + 16, chunk) + 8 * (j & 1)));
                const u32x2 w0 = __builtin_bit_cast(u32x2, b0), w1 = __builtin_bit_cast(u32x2, b1);
                w = u32x4{w0.x, w0.y, w1.x, w1.y};
            }
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(p), o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(p_low), o[i], 0, 0, 0);
        }
    }
    f32x2 two = with_lane_16(l);
    two = with_lane_32(two.x + two.y);
    l = two.x + two.y;

    // join the waves
    if (lane < 16) {
        ml[wave][0][lane] = m;
        ml[wave][1][lane] = l;
    }
    __syncthreads();                                   // (also: every wave is done with its tile)
    float *const parts = reinterpret_cast<float *>(lds);
    float most = -__builtin_inff();
#pragma unroll 4
    for (int w = 0; w < (int)kWaves; ++w) most = fmaxf(most, ml[w][0][col]);
    const float base = most == -__builtin_inff() ? 0.0f : most;
    const float weight = exp2_fast(m - base);
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
        *reinterpret_cast<f32x4 *>(parts + (wave * 16 + col) * kOStride + 16 * i + 4 * grp) = o[i] * weight;
    __syncthreads();
    const uint32_t heads_here = min(16u, a.group - q_tile * 16);
    for (uint32_t at = threadIdx.x; at < heads_here * (D / 4); at += kThreads) {
        const uint32_t c = at / (D / 4), d = at % (D / 4) * 4;
        f32x4 sum = {0, 0, 0, 0};
        float most_c = -__builtin_inff(), l_c = 0;
#pragma unroll
        for (int w = 0; w < (int)kWaves; ++w) most_c = fmaxf(most_c, ml[w][0][c]);
        const float base_c = most_c == -__builtin_inff() ? 0.0f : most_c;
#pragma unroll
        for (int w = 0; w < (int)kWaves; ++w) {
            sum += *reinterpret_cast<const f32x4 *>(parts + (w * 16 + c) * kOStride + d);
            l_c += ml[w][1][c] * exp2_fast(ml[w][0][c] - base_c);
        }
        const uint32_t h = kv_head * a.group + q_tile * 16 + c;
        if (a.splits == 1) {
            const float inv = l_c == 0.0f ? 0.0f : 1.0f / l_c;
            *reinterpret_cast<u32x2 *>(a.out.data + seq * a.out.row + h * a.out.head + d) =
                u32x2{pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv)};
        } else {
            const uint64_t at_part = ((uint64_t)seq * a.heads + h) * a.splits + split;
            *reinterpret_cast<f32x4 *>(a.part + at_part * D + d) = sum;
            if (d == 0) *reinterpret_cast<f32x2 *>(a.part_ml + 2 * at_part) = f32x2{most_c, l_c};
        }
    }
}

// Joins the parts of one query head: out = sum_a w_a o_a / sum_a w_a l_a with
// w_a = 2^(m_a - max m).
template <int D>
__global__ __launch_bounds__(256) void join_token_kernel(TokenArgs a) {
    __shared__ float sums[4][D];
    __shared__ float ls[4];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t seq = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    const uint32_t len = (uint32_t)min((int64_t)max(a.lens[seq], 0), (int64_t)a.t.width << a.c.shift);
    const uint32_t n = max(1u, (len + a.range - 1) / a.range);     // parts that were written
    const uint64_t first = (uint64_t)blockIdx.x * a.splits;
    const f32x2 *const ml = reinterpret_cast<const f32x2 *>(a.part_ml) + first;
    float most = -__builtin_inff();
    for (uint32_t i = lane; i < n; i += 64) most = fmaxf(most, ml[i].x);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
    const float base = most == -__builtin_inff() ? 0.0f : most;
    float sum[D / 64] = {}, l = 0;
#pragma unroll 4
    for (uint32_t i = wave; i < n; i += 4) {
        const float w = exp2_fast(ml[i].x - base);
        l += w * ml[i].y;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) sum[j] += w * a.part[(first + i) * D + (D / 64) * lane + j];
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) sums[wave][(D / 64) * lane + j] = sum[j];
    if (lane == 0) ls[wave] = l;
    __syncthreads();
    if (threadIdx.x < D / 2) {
        const float total = ls[0] + ls[1] + ls[2] + ls[3];
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        const uint32_t d = 2 * threadIdx.x;
        const float x = sums[0][d] + sums[1][d] + sums[2][d] + sums[3][d];
        const float y = sums[0][d + 1] + sums[1][d + 1] + sums[2][d + 1] + sums[3][d + 1];
        *reinterpret_cast<uint32_t *>(a.out.data + seq * a.out.row + h * a.out.head + d) = pack_bf16(x * inv, y * inv);
    }
}

template <uint32_t kWaves, bool kOnce>
void launch_as(const TokenArgs &a, uint32_t head_dim, bool int8, dim3 grid, hipStream_t stream) {
    const auto kernel = head_dim == 64 ? (int8 ? attend_token_kernel<64, true, kWaves, kOnce> : attend_token_kernel<64, false, kWaves, kOnce>)
                                       : (int8 ? attend_token_kernel<128, true, kWaves, kOnce> : attend_token_kernel<128, false, kWaves, kOnce>);
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), 0, stream, a);
}

template <uint32_t kWaves>
void launch(const TokenArgs &a, uint32_t head_dim, bool int8, dim3 grid, hipStream_t stream) {
    if (a.q_tiles == 1) launch_as<kWaves, true>(a, head_dim, int8, grid, stream);
    else launch_as<kWaves, false>(a, head_dim, int8, grid, stream);
}

}  // namespace

hipError_t launch_attend_token(const TokenArgs &a, uint32_t head_dim, bool int8, hipStream_t stream) {
    // (a table of 2^28 positions has 262,144 parts of 1024, a grid's y and z dimensions hold 65,535)
    const uint32_t parts = a.splits < 65535 ? a.splits : 65535;
    const dim3 grid(a.q_tiles == 1 ? a.n_seqs * a.c.kv_heads : (a.n_seqs * a.c.kv_heads + 7) / 8 * 8 * a.q_tiles, parts,
                    (a.splits + parts - 1) / parts);
    if (a.whole) launch<12>(a, head_dim, int8, grid, stream);
    else launch<4>(a, head_dim, int8, grid, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    hipLaunchKernelGGL(head_dim == 64 ? join_token_kernel<64> : join_token_kernel<128>, dim3(a.n_seqs * a.heads), dim3(256), 0,
                       stream, a);
    return hipGetLastError();
}

}  // namespace df11
