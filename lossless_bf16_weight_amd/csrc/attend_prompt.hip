// Attention over packed prompts for gfx950, causal or not, with grouped heads.
//
// Query i of a sequence with n_q queries and n_k keys sees the keys below
// lim_i = i + 1 + n_k - n_q (causal) or n_k.  s_j = <q_i, k_j>, p_j =
// 2^(c s_j - m), c = scale log2(e), m the running maximum of c s_j (and a
// constant: see kSlack), out = sum p_j v_j / sum p_j; a row that sees no key is
// 0.  One pass over the keys: when a step raises m, the sums are scaled by
// 2^(old - new).
//
// The queries of the heads that share a kv head are the rows of one matrix:
// row r is query r / group of head r % group.  A workgroup takes 128 rows of a
// kv head, its four waves 32 each, and steps over the keys 64 at a time through
// LDS, the next step's on their way.  Matrix instructions, 32 x 32 x 16: S^T =
// K Q^T puts a query in each lane (column) with 16 keys of 32 in its registers
// (the lane 32 away has the others), so that the row statistics are per lane,
// and P^T is the second product's operand as it stands: O^T = V^T P^T sums over
// keys in any order, so the key of operand slot (half h, j) is 4h + j for j < 4
// and 8 + 4h + j - 4 above.  V^T comes from row-major V in LDS by transposing
// reads.
//
// The matrix rate and, beside it, the exponentials bound it.  Measured with 32
// heads over 8 kv heads of 128, causal: a prompt of 16,384 tokens 1.9 to 2.1 ms
// (2.2 TFLOP: 1.05 to 1.16 PFLOP/s; a product of 16,384-square matrices reaches
// 1.37), its matrix units busy 60% of the cycles at the 1.76 GHz that the power
// limit leaves; 64 prompts of 1024 tokens 0.70 ms, 11 of up to 2,113 172 us
// (0.82 PFLOP/s of the visible pairs), 64 tokens 7.4 us.  With heads of 64
// 16,384 tokens take 1.10 ms (1.0 PFLOP/s: as many exponentials for half the
// products); 8192 not causal 0.97 ms (1.13 PFLOP/s).  With twice the rows a
// workgroup (eight waves) 16,384 tokens are 2.5% faster and shorter prompts
// slower; steps of 32 keys, with a third wave for each SIMD or four stages in
// LDS, are no faster.
#include <type_traits>

#include "serve_device.hpp"
#include "serve_internal.hpp"

namespace df11 {

namespace {

constexpr uint32_t kWaves = 4, kThreads = 64 * kWaves;
constexpr uint32_t kWaveRows = 32;
constexpr int kHalves = kPromptKeys / 32;      // of a step: 32 keys are a product's rows
constexpr int kAhead = 4;                      // reads of K ahead of the products

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
__device__ __forceinline__ uint32_t over_group(const PromptArgs &a, uint32_t row) {
    return a.group == 1 ? row : __umulhi(row, a.group_magic) >> a.group_shift;
}

// The tile of rows that work item `slot` stands for, and its sequence; false
// where there is none.  The last tiles of a sequence, which see the most keys
// of a causal prompt, come first, and so do the sequences with the most keys
// where there are few: a heavy tile at the end would keep the others' compute
// units waiting (11 sequences of 1 to 2113 tokens, shortest first: with 12
// heads over 4 71 us, unranked 80 us; with 32 over 8 177 and 180 us).  Each
// workgroup pays for the ranking: sequences that are equal, or come longest
// first, are better off without (16 of 256 tokens: 28.8 us, unranked 26.0; the
// 11 longest first 72 and 70 us), and with more sequences it levels out (64 of
// 1024 tokens: 703 us, ranked 749 us; 64 of 256: 96 and 114 us).
constexpr uint32_t kRanked = 16;

__device__ __forceinline__ bool pick_tile(const PromptArgs &a, uint32_t slot, uint32_t *tile, int32_t *q0, int32_t *q1,
                                          int32_t *k0, int32_t *k1) {
    if (a.n_seqs > 64) {
        const uint32_t s = sequence_of_slot(a.q_starts, a.n_seqs, a.tile_slots - 1 - slot, a.group, 7, tile);
        *q0 = a.q_starts[s], *q1 = a.q_starts[s + 1], *k0 = a.k_starts[s], *k1 = a.k_starts[s + 1];
        if (*q0 < 0 || *q1 < *q0 || (uint32_t)*q1 > a.n_q || *k0 < 0 || *k1 < *k0 || (uint32_t)*k1 > a.n_k) return false;
        const uint32_t n_rows = (uint32_t)(*q1 - *q0) * a.group;
        return *tile <= n_rows / kPromptTile && *tile * kPromptTile < n_rows;
    }
    // a lane a sequence: one trip to memory gives all starts
    const uint32_t lane = threadIdx.x & 63u, at = min(lane, a.n_seqs - 1);
    const int32_t qa = a.q_starts[at], qb = a.q_starts[at + 1], ka = a.k_starts[at], kb = a.k_starts[at + 1];
    const bool ok = lane < a.n_seqs && qa >= 0 && qb >= qa && (uint32_t)qb <= a.n_q && ka >= 0 && kb >= ka && (uint32_t)kb <= a.n_k;
    const uint32_t tiles = ok ? ((uint32_t)(qb - qa) * a.group + kPromptTile - 1) / kPromptTile : 0;
    uint32_t before = 0;        // slots before the sequence's
    if (a.n_seqs <= kRanked) {
        // (the order of two sequences whose keys differ by less than 64 does not
        // matter, that of two lanes must be one or the other)
        const uint32_t rank = (ok ? kb - ka : 0) & ~63u | (63u - lane);
        for (uint32_t j = 0; j < a.n_seqs; j += 8) {
#pragma unroll
            for (uint32_t x = 0; x < 8; ++x)
                before += (uint32_t)__builtin_amdgcn_readlane(rank, j + x) > rank ? __builtin_amdgcn_readlane(tiles, j + x) : 0;
        }
    } else {
        before = ((uint32_t)qa * a.group >> 7) + lane;      // (at least as many slots as tiles: see sequence_of_slot)
    }
    const uint64_t found = __ballot(slot >= before && slot - before < tiles);
    if (!found) return false;
    const uint32_t s = (uint32_t)__builtin_ctzll(found);
    *tile = __builtin_amdgcn_readlane(tiles, s) - 1 - (slot - __builtin_amdgcn_readlane(before, s));
    *q0 = __builtin_amdgcn_readlane(qa, s);
    *q1 = __builtin_amdgcn_readlane(qb, s);
    *k0 = __builtin_amdgcn_readlane(ka, s);
    *k1 = __builtin_amdgcn_readlane(kb, s);
    return true;
}

// Keys of a sequence that a query sees.
__device__ __forceinline__ uint32_t keys_seen(const PromptArgs &a, uint32_t query, uint32_t n_q, uint32_t n_k) {
    if (!a.causal) return n_k;
    const int64_t l = (int64_t)query + 1 + n_k - n_q;
    return l < 0 ? 0 : l > n_k ? n_k : (uint32_t)l;
}

// Keys of one part of a sequence's.  A part that begins past the keys which its
// tile sees is neither written nor read, and a tile of one part is not joined.
__device__ __forceinline__ uint32_t keys_a_part(const PromptArgs &a, uint32_t n_k) {
    // (the quotient, or one more; whole steps, above n_k / splits)
    return max((__umulhi(n_k, a.split_magic) + kPromptKeys) / kPromptKeys * kPromptKeys, a.part_keys);
}

// Writes a product's 32 x 32 results as BF16, the lane's column to 32 words
// from `to`.  The lane has four of each eight neighbours, the lane 32 away the
// others: with two such eights they exchange halves and write one each.
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

template <int D, bool kSplit>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : 2) void attend_prompt_kernel(PromptArgs a) {
    constexpr int kChunks = D / 8;                           // 16-byte chunks of a row
    constexpr int kLoads = kPromptKeys * kChunks / kThreads; // chunks a thread stages
    constexpr int kDTiles = D / 32;
    constexpr int kDSteps = D / 16;
    __shared__ __attribute__((aligned(16))) uint8_t kt0[kPromptKeys * D * 2], kt1[kPromptKeys * D * 2];
    __shared__ __attribute__((aligned(16))) uint8_t vt0[kPromptKeys * D * 2], vt1[kPromptKeys * D * 2];

    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane_of_wave = lane, col = lane & 31u, half = lane >> 5;

    // (workgroups are dealt to the eight XCDs in turn: kv heads vary fastest,
    // so that the tiles of one meet in one L2)
    const uint32_t kv_head = blockIdx.x % a.kv_heads;
    uint32_t tile;
    int32_t q0, q1, k0, k1;
    if (!pick_tile(a, blockIdx.x / a.kv_heads, &tile, &q0, &q1, &k0, &k1)) return;
    const uint32_t n_q = q1 - q0, n_k = k1 - k0, n_rows = n_q * a.group;
    const uint32_t row0 = tile * kPromptTile;

    const auto limit = [&](uint32_t query) { return keys_seen(a, query, n_q, n_k); };
    const uint32_t most_keys = limit(over_group(a, min(row0 + kPromptTile, n_rows) - 1));
    uint32_t key_begin = 0, key_end = most_keys;
    bool whole = true;
    if (kSplit) {
        const uint32_t per = keys_a_part(a, n_k);
        const uint64_t b = (uint64_t)blockIdx.y * per;
        if (b >= most_keys && b) return;
        key_begin = (uint32_t)b;
        key_end = b + per < most_keys ? (uint32_t)(b + per) : most_keys;
        whole = most_keys <= per;
    }
    const uint32_t wave_first = row0 + wave * kWaveRows, row = wave_first + col;
    const bool real = row < n_rows;
    const uint32_t query = over_group(a, row), head = kv_head * a.group + row - query * a.group;
    // (rows past the last compute on zero queries, and are not stored)
    const uint32_t lim = real ? limit(query) : n_k;
    // the wave's rows all see the keys below `clear`, and none from wave_end on
    const uint32_t clear = limit(over_group(a, wave_first));
    const uint32_t wave_end = wave_first < n_rows ? limit(over_group(a, min(wave_first + kWaveRows, n_rows) - 1)) : 0;

    u32x4 q[kDSteps];
#pragma unroll
    for (int i = 0; i < kDSteps; ++i) {
        q[i] = u32x4{0, 0, 0, 0};
        if (real) q[i] = *reinterpret_cast<const u32x4 *>(a.q.data + (int64_t)(q0 + query) * a.q.row + head * a.q.head + 16 * i + 8 * half);
    }

    f32x16 o[kDTiles];
    float m, l;
    const float log2_n = log2_up(n_k);
    const auto start = [&] {
#pragma unroll
        for (int i = 0; i < kDTiles; ++i) o[i] = f32x16{};
        m = -__builtin_inff();
        l = 0;
    };

    const uint16_t *const kp = a.k.data + (int64_t)k0 * a.k.row + kv_head * a.k.head;
    const uint16_t *const vp = a.v.data + (int64_t)k0 * a.v.row + kv_head * a.v.head;

    // A step's K and V rows go from memory into LDS without passing through
    // registers, one step ahead: the chunk that lane `at` of the tile holds is
    // the one that belongs there.  A thread's chunks are 16 (or 32) rows apart
    // and share their place in the row, so that one offset serves all; rows
    // past the sequence (another one's) are out of the descriptor's range and
    // arrive as zeros.
    constexpr uint32_t kRowsALoad = kThreads / kChunks;
    const uint32_t tile_row = threadIdx.x / kChunks, place = threadIdx.x % kChunks;
    const uint32_t k_offset = 2 * (tile_row * (uint32_t)a.k.row + 8 * k_chunk<D>(tile_row, place));
    const uint32_t v_offset = 2 * (tile_row * (uint32_t)a.v.row + 8 * v_chunk<D>(tile_row, place));
    const auto load = [&](uint32_t key0, uint8_t *kt, uint8_t *vt) {
        const __amdgpu_buffer_rsrc_t kr = __builtin_amdgcn_make_buffer_rsrc((void *)(kp + key0 * a.k.row), 0, kOutOfRange, 0x00020000);
        const __amdgpu_buffer_rsrc_t vr = __builtin_amdgcn_make_buffer_rsrc((void *)(vp + key0 * a.v.row), 0, kOutOfRange, 0x00020000);
        const uint32_t left = n_k - key0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool in = tile_row + i * kRowsALoad < left;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (DF11_LDS void *)(kt + (i * kThreads + wave * 64) * 16), 16,
                                                     in ? k_offset : kOutOfRange, 2 * i * kRowsALoad * (uint32_t)a.k.row, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (DF11_LDS void *)(vt + (i * kThreads + wave * 64) * 16), 16,
                                                     in ? v_offset : kOutOfRange, 2 * i * kRowsALoad * (uint32_t)a.v.row, 0, 0);
        }
    };
    const auto arrived = [&] {
        __builtin_amdgcn_s_waitcnt(0x0F70);        // vmcnt(0): this wave's rows
        __syncthreads();                           // and the others'; and all are done with the step before
    };

    // One step's keys.  kCareful: values that are infinite or NaN at keys which
    // only some rows see do not reach the others.
    const auto step = [&](auto careful, uint32_t key0, const uint8_t *kt, const uint8_t *vt) {
        constexpr bool kCareful = decltype(careful)::value;
        if (key0 >= wave_end) return;
        // (the careful pass computes its LDS addresses in each step: there are
        // no registers to keep them in)
        uint32_t own = lane_of_wave;
        if (kCareful) asm volatile("" : "+v"(own));
        const uint32_t lane = own, col = own & 31u, half = own >> 5;

        f32x16 s[kHalves];
#pragma unroll
        for (int t = 0; t < kHalves; ++t) s[t] = f32x16{};
#pragma unroll
        for (int i = 0; i < kDSteps; ++i)
#pragma unroll
            for (int t = 0; t < kHalves; ++t) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(kt + k_at<D>(32 * t + col, 2 * i + half));
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), as_bf16x8(q[i]), s[t], 0, 0, 0);
            }
        // (four reads of K ahead of the products)
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kHalves * kDSteps - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
        if (key0 + kPromptKeys > clear) {
#pragma unroll
            for (int t = 0; t < kHalves; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t key = key0 + 32 * t + 8 * (i / 4) + 4 * half + i % 4;
                    if (key >= lim) s[t][i] = -__builtin_inff();
                }
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < kHalves; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        const f32x2 halves = with_lane_32(top);
        top = fmaxf(halves.x, halves.y) * a.log2_scale;
        if (__any(top > m - log2_n)) {
            const float next = fmaxf(m, top + (kSlack + log2_n));
            const float keep = exp2_fast(m - (next == -__builtin_inff() ? 0.0f : next));
            m = next;
            l *= keep;
#pragma unroll
            for (int i = 0; i < kDTiles; ++i) o[i] *= keep;
        }
        const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
        for (int t = 0; t < kHalves; ++t) {
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                u32x4 p;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = exp2_fast(__builtin_fmaf(s[t][8 * st + 2 * j], a.log2_scale, -base));
                    const float y = exp2_fast(__builtin_fmaf(s[t][8 * st + 2 * j + 1], a.log2_scale, -base));
                    l += x + y;
                    p[j] = pack_bf16(x, y);
                }
#pragma unroll
                for (int i = 0; i < kDTiles; ++i) {
                    const uint32_t j = lane & 15u, r = 32 * t + 16 * st + 4 * half + (j >> 2);
                    const uint32_t chunk = 4 * i + 2 * ((lane >> 4) & 1u) + ((j & 3) >> 1);
                    const s16x4 b0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(vt + v_at<D>(r, chunk) + 8 * (j & 1)));
                    const s16x4 b1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(vt + v_at<D>(r + 8, chunk) + 8 * (j & 1)));
                    const u32x2 w0 = __builtin_bit_cast(u32x2, b0), w1 = __builtin_bit_cast(u32x2, b1);
                    u32x4 w = {w0.x, w0.y, w1.x, w1.y};
                    if (kCareful) {
                        // Values that are not finite leave the product (0 times
                        // one of them is not 0) and are counted apart, over the
                        // keys that the row sees (whose score is not that of a
                        // masked one): ones where they are +inf or NaN, and
                        // where they are -inf or NaN.
                        u32x4 seen, up, down;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            seen[x] = up[x] = down[x] = 0;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t h = w[x] >> (16 * y) & 0xFFFFu, one = 0x3F80u << (16 * y);
                                const bool odd = (h & 0x7F80u) == 0x7F80u, nan = odd && (h & 0x7Fu);
                                if (s[t][8 * st + 2 * x + y] != -__builtin_inff()) seen[x] |= one;
                                if (nan || h == 0x7F80u) up[x] |= one;
                                if (nan || h == 0xFF80u) down[x] |= one;
                                if (odd) w[x] &= 0xFFFF0000u >> (16 * y);
                            }
                        }
                        f32x16 n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(up), as_bf16x8(seen), f32x16{}, 0, 0, 0);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (n[x] > 0) o[i][x] += __builtin_inff();
                        __builtin_amdgcn_sched_barrier(0);
                        n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(down), as_bf16x8(seen), f32x16{}, 0, 0, 0);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (n[x] > 0) o[i][x] -= __builtin_inff();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), as_bf16x8(p), o[i], 0, 0, 0);
                }
            }
        }
    };
    start();
    if (key_begin < key_end) load(key_begin, kt0, vt0);
    for (uint32_t key0 = key_begin; key0 < key_end; key0 += 2 * kPromptKeys) {
        arrived();
        if (key0 + kPromptKeys < key_end) load(key0 + kPromptKeys, kt1, vt1);
        step(std::false_type{}, key0, kt0, vt0);
        if (key0 + kPromptKeys >= key_end) break;
        arrived();
        if (key0 + 2 * kPromptKeys < key_end) load(key0 + 2 * kPromptKeys, kt0, vt0);
        step(std::false_type{}, key0 + kPromptKeys, kt1, vt1);
    }
    if (a.causal) {
        // A result that is not finite may come from a value that its row does
        // not see: the product of its weight, 0, with an infinity is NaN.  Then
        // the workgroup takes its keys once more, with care.
        float most = 0;       // (NaN where one is)
#pragma unroll
        for (int i = 0; i < kDTiles; ++i)
#pragma unroll
            for (int x = 0; x < 16; ++x) most = __builtin_elementwise_maximum(most, __builtin_fabsf(o[i][x]));
        if (__syncthreads_or(!(most < __builtin_inff()))) {
            start();
            for (uint32_t key0 = key_begin; key0 < key_end; key0 += kPromptKeys) {
                load(key0, kt0, vt0);
                arrived();
                step(std::true_type{}, key0, kt0, vt0);
                __syncthreads();
            }
        }
    }
    const f32x2 l_halves = with_lane_32(l);
    l = l_halves.x + l_halves.y;
    if (kSplit && !whole) {
        if (wave_first >= n_rows) return;
        // as the lanes hold them, for the lanes of the join
        const uint64_t at = ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + wave;
        f32x4 *const part = reinterpret_cast<f32x4 *>(a.part) + at * (kDTiles * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < kDTiles; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) part[(4 * i + g) * 64] = f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
        if (half == 0) reinterpret_cast<f32x2 *>(a.part_ml)[at * kWaveRows + col] = f32x2{m, l};
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *const op = a.out.data + (int64_t)(q0 + query) * a.out.row + head * a.out.head;
#pragma unroll
    for (int i = 0; i < kDTiles; ++i) store_tile(o[i] * inv, op + 32 * i, half, real);
}

// Joins the parts of 32 rows (those of wave blockIdx.y of workgroup blockIdx.x):
// out = sum_a w_a o_a / sum_a w_a l_a with w_a = 2^(m_a - max m), the maximum
// taken as the parts come.  A wave takes 32 columns.  It is bound by the way
// to memory: the first parts are asked for before the number of parts is known.
template <int D>
__global__ __launch_bounds__(64 * D / 32) void join_prompt_kernel(PromptArgs a) {
    constexpr int kDTiles = D / 32;
    constexpr int kBatch = 2;       // parts in flight
    const uint32_t lane = threadIdx.x & 63u, i = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t col = lane & 31u, half = lane >> 5;
    const uint64_t at = (uint64_t)blockIdx.x * kWaves + blockIdx.y, step = (uint64_t)gridDim.x * kWaves;
    const f32x2 *const ml = reinterpret_cast<const f32x2 *>(a.part_ml) + at * kWaveRows + col;
    const f32x4 *const part = reinterpret_cast<const f32x4 *>(a.part) + (at * kDTiles + i) * 256 + lane;
    f32x2 p[kBatch];
    f32x4 v[kBatch][4];
    const auto load = [&](uint32_t s, uint32_t parts) {
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const uint32_t from = min(s + x, parts - 1);
            p[x] = ml[from * step * kWaveRows];
#pragma unroll
            for (int g = 0; g < 4; ++g) v[x][g] = __builtin_nontemporal_load(part + from * step * (kDTiles * 256) + g * 64);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    load(0, a.splits);
    uint32_t tile;
    int32_t q0, q1, k0, k1;
    if (!pick_tile(a, blockIdx.x / a.kv_heads, &tile, &q0, &q1, &k0, &k1)) return;
    const uint32_t first = tile * kPromptTile + blockIdx.y * kWaveRows, row = first + col, n_rows = (uint32_t)(q1 - q0) * a.group;
    if (first >= n_rows) return;
    const uint32_t n_k = k1 - k0, most_keys = keys_seen(a, over_group(a, min((tile + 1) * kPromptTile, n_rows) - 1), q1 - q0, n_k);
    const uint32_t per = keys_a_part(a, n_k);
    if (most_keys <= per) return;
    const uint32_t parts = __builtin_popcountll(__ballot(lane < a.splits && lane * per < most_keys));
    f32x16 o = {};
    float l = 0, m = -__builtin_inff();
    for (uint32_t s = 0; s < parts; s += kBatch) {
        if (s) load(s, parts);
        float next = m;
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
            if (s + x < parts) next = fmaxf(next, p[x].x);
        const float base = next == -__builtin_inff() ? 0.0f : next, keep = exp2_fast(m - base);
        m = next;
        l *= keep;
        o *= keep;
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            if (s + x >= parts) break;      // (a part past the last was not written)
            const float w = exp2_fast(p[x].x - base);
            l += w * p[x].y;
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] += w * v[x][y / 4][y % 4];
        }
    }
    const uint32_t query = over_group(a, row), head = blockIdx.x % a.kv_heads * a.group + row - query * a.group;
    store_tile(o * (l == 0.0f ? 0.0f : 1.0f / l), a.out.data + (int64_t)(q0 + query) * a.out.row + head * a.out.head + 32 * i, half, row < n_rows);
}

}  // namespace

hipError_t launch_attend_prompt(const PromptArgs &a, uint32_t head_dim, hipStream_t stream) {
    const dim3 grid(a.tile_slots * a.kv_heads, a.splits);
    const auto kernel = head_dim == 64 ? (a.splits > 1 ? attend_prompt_kernel<64, true> : attend_prompt_kernel<64, false>)
                                       : (a.splits > 1 ? attend_prompt_kernel<128, true> : attend_prompt_kernel<128, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    hipLaunchKernelGGL(head_dim == 64 ? join_prompt_kernel<64> : join_prompt_kernel<128>,
                       dim3(a.tile_slots * a.kv_heads, kWaves), dim3(2 * head_dim), 0, stream, a);
    return hipGetLastError();
}

}  // namespace df11
