// Attention of a chunk of new tokens of each sequence over the paged cache, for
// gfx950: a prompt's piece, a single token, a whole prompt.
//
// Query i of a sequence's n_q stands at position p = n_k - n_q + i of its n_k
// cached ones and sees the keys j <= p (causal), of these with a window of w
// the last w and the first `sinks`; or all keys.  s_j = <q_i, k_j>, p_j =
// 2^(c s_j - m), c = scale log2(e), m the running maximum of c s_j (and a
// constant: see kSlack), out = sum p_j v_j / sum p_j; a row that sees no key is
// 0.  Keys in 8 bits become exact BF16 operands; a key's scale multiplies its
// scores, a value's scale its weights, in 32 bits.
//
// Rows, tiles, products and the steps of 64 keys through LDS are those of
// attend_prompt.hip, but a workgroup may have eight waves and 256 rows; rows
// come from pages, 16 at a time from one page, whose numbers lie in the lanes of
// a register (64 entries of the table).  Words go from memory into LDS without
// passing through registers; codes pass through them, converted once by the
// workgroup.  The steps of a tile are those of the sinks and those of the
// window.
// Sequences of one new token, whose rows are few, go another way: see
// attend_single.
//
// How long the sequences are the host does not know.  Each workgroup finds
// from q_starts and lens how the work of the whole call is divided: the steps
// of all tiles over as many workgroups as run at a time give a quota, and a
// sequence's tiles are split into as many parts as their steps hold quotas.  A second kernel
// joins the parts.
//
// Long pieces are bound by the matrix units at the card's power limit: 2048
// queries of 32 heads over 8 of 128 on 32,049 keys take 915 to 943 us (1.12
// PFLOP/s, where a 16,384-square product reaches 1.31), a prompt of 16,384 in a
// window of 4096 905 to 943 us (1.05); heads of 64 575 to 595 us, of as many
// exponentials.  Codes cost the vector units, which hide behind the products of
// words: 1063 us, and six pieces of up to 701 queries 328 to 361 us for 284.  Four
// pieces of up to 512 behind up to 8192 with 28 single tokens take 156 to 176 us, for 520 MB, most of
// them the tokens' (alone 96 us, 5.2 TB/s); 64 queries on 2001 keys 17.5 us, a
// chain of reads, four steps and the join.
#include "attend_columns.hpp"
#include "attend_tiles.hpp"

namespace df11 {

// x * y, but 0 where either is 0, whatever the other.
__device__ float mul_or_zero(float x, float y) __asm("llvm.amdgcn.fmul.legacy");

namespace {

constexpr uint32_t kWaveRows = 32;             // a workgroup has four waves or eight
constexpr int kHalves = kPromptKeys / 32;      // of a step: 32 keys are a product's rows
constexpr int kAhead = 4;                      // reads of K ahead of the products
constexpr uint32_t kWorthLevelling = 24, kLevelled = 8;      // steps of a quota, sequences: see level_out
constexpr uint32_t kFewSteps = 8;              // of a tile: see the loops in 8 bits

// What a workgroup does: a part of a tile of a sequence.
struct Piece {
    uint32_t seq, n_q, n_k;
    int32_t q0;
    uint32_t tile, part, parts, per;      // of `parts`, each of `per` steps
    uint32_t place;                       // where the parts of the tile lie in the workspace
};

__device__ __forceinline__ uint32_t of_lane(uint32_t x, uint32_t lane) { return __builtin_amdgcn_readlane(x, lane); }

// Parts of the longest tiles of a single sequence of many rows: the number that
// ends soonest, in steps of a workgroup among as many as run at a time.  A part
// has two steps' time beside its own, and what is written and joined of it.
// Tiles behind a long prefix are equal, and their parts take whole rounds;
// where the first tiles are short (`least` steps, of `steps`), these even the
// end out.  (Few tiles have many parts, where rounding is harmless.)  Coefficients
// need not be exact: with none, half or twice of the join's 0.028, or none or twice
// of the two steps, 16 drawn pieces of 520 to 5000 tokens behind 1500 to 50,000 take
// 0.99 to 1.01 of the time on average.
__device__ __forceinline__ uint32_t parts_of_one(const ChunkArgs &a, uint32_t tiles, uint32_t least, uint32_t steps, uint32_t otherwise) {
#pragma clang fp contract(off)      // (both kernels are to find the same)
    if (tiles * 8 < a.at_a_time) return otherwise;
    const uint32_t lane = threadIdx.x & 63u, parts = lane + 1, per = (steps + parts - 1) / parts;
    const float at_once = 1.0f / (float)a.at_a_time, equal = (float)least / (float)steps, average = 0.5f * (float)(least + steps), over = parts > 1 ? 2.0f : 1.0f;
    const float items = fminf((float)(tiles * parts), (float)tiles * fmaxf(average / (float)per + 0.5f, 1.0f));
    const float in_rounds = __builtin_ceilf(items * at_once) * ((float)per + over), level = ((float)tiles * average + items * over) * at_once + 0.25f * (float)per;
    float cost = fmaxf((float)per + over, equal * in_rounds + (1.0f - equal) * level);
    if (parts > 1) cost += 2.0f + 0.028f * items * (float)a.c.kv_heads;
    const bool possible = parts == 1 || (parts <= steps >> a.least_shift && tiles * parts <= a.places);
    const uint32_t key = possible ? (__float_as_uint(cost) & ~63u) | lane : ~0u;
    return (of_lane(over_lanes(key, ~0u, Least{}), 63) & 63u) + 1;
}

// Work items before those of this lane's sequence, the longest parts first (one
// of them at the end would keep the others' compute units waiting).
__device__ __forceinline__ uint32_t items_before(uint32_t n_seqs, uint32_t per, uint32_t items) {
    const uint32_t rank = per << 6 | (threadIdx.x & 63u);
    uint32_t before = 0;
    for (uint32_t j = 0; j < n_seqs; ++j) before += of_lane(rank, j) > rank ? of_lane(items, j) : 0;
    return before;
}

// The quota, or less of it, with which the parts of several sequences (a lane
// each) end soonest, as far as these lower bounds say: the average, the longest
// part, and for one more than run at a time (or than twice as many) the two (three)
// that share a place.  A part has two steps' time beside its own, and what is
// written and joined of it (0 or twice of the join's 0.007: within 2%).  A call of up
// to eight sequences gains or loses by it: of 17 drawn ones each of 2 to 8 sequences,
// pieces of 20 to 1500 behind 300 to 16,000 tokens, from 14% less to 18% more than by
// the quota, 0.5% more on average (six of up to 701 on up to 12,701 in 8 bits 328 us
// and 346, with heads of 64 209 and 196).  With the search 10 to 16 sequences take 2
// to 5% more, 12 and 32 that have single tokens among them 5 and 13%.  0: no quota
// makes `item` one.
__device__ __forceinline__ uint32_t level_out(const ChunkArgs &a, uint32_t tiles, uint32_t steps, float total, uint32_t quota, uint32_t item) {
    const uint32_t smallest = (quota * 9 + 15) / 16;
    if (!__any(tiles && steps + smallest / 2 >= 2 * smallest)) return quota;      // (all tiles are whole)
    float least = __builtin_inff();
    uint32_t chosen = 0;
    for (uint32_t sixteenths = 9; sixteenths <= 16; sixteenths += sixteenths == 9 ? 4 : 3) {
        const uint32_t q = (quota * sixteenths + 15) / 16;
        const uint32_t parts = max(1u, min((steps + q / 2) / q, steps >> a.least_shift)), per = (steps + parts - 1) / parts, items = tiles * parts;
        const uint32_t all = of_lane(over_lanes(items, 0u, Add{}), 63), split = of_lane(over_lanes(parts > 1 ? items : 0u, 0u, Add{}), 63);
        if (sixteenths == 9 && item >= all) return 0;
        const uint32_t before = items_before(a.n_seqs, per, items), w = a.at_a_time;
        const auto at = [&](uint32_t k) {
            const uint64_t has = __ballot(before < k && k - before <= items);
            return has ? of_lane(per, (uint32_t)__builtin_ctzll(has)) + 2 : 0;
        };
        const uint32_t bound = max(max(at(1), all > w ? at(w) + at(w + 1) : 0), all > 2 * w ? at(2 * w - 1) + at(2 * w) + at(2 * w + 1) : 0);
        const float cost = fmaxf((float)bound, (total + 2.0f * (float)all) * a.by_parts) + (split ? 2.0f + 0.007f * (float)(split * a.c.kv_heads) : 0.0f);
        if (cost < least) {
            least = cost;
            chosen = q;
        }
    }
    return chosen;
}

// Finds work item `item` (kJoin: the tile of that number among those that are
// split).  False where there is none.
template <uint32_t kWaves, bool kSplit, bool kJoin>
__device__ __forceinline__ bool find_piece(const ChunkArgs &a, uint32_t item, Piece *p) {
#pragma clang fp contract(off)
    constexpr uint32_t kTile = kWaves * kWaveRows;
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t q0 = 0, n_q = 0, n_k = 0, tiles = 0, steps = 0;
    const auto look = [&](uint32_t s0) {
        const uint32_t s = min(s0 + lane, a.n_seqs - 1);
        const int32_t from = a.q_starts[s], to = a.q_starts[s + 1];
        const bool ok = s0 + lane < a.n_seqs && from >= 0 && to >= from && (uint32_t)to <= a.n_q;
        q0 = from;
        n_q = ok ? to - from : 0;
        n_k = (uint32_t)min((int64_t)max(a.lens[s], 0), (int64_t)a.t.width << a.c.shift);
        tiles = (n_q * a.group + kTile - 1) / kTile;
        steps = min((n_k + kPromptKeys - 1) / kPromptKeys, a.most_steps);
    };
    uint32_t quota = 0;
    if (kSplit && kJoin && kWaves == 4) {
        quota = *a.quota;
    } else if (kSplit) {
        float total = 0;
        for (uint32_t s0 = 0; s0 < a.n_seqs; s0 += 64) {
            look(s0);
            total += (float)tiles * (float)steps;
        }
        total = __uint_as_float(of_lane(__float_as_uint(over_lanes(total, 0.0f, Add{})), 63));
        // (above the quotient, whatever the sum's rounding: see chunk_split)
        quota = (uint32_t)fminf(total * a.by_parts * (1.0f + 0x1p-18f), 4.0e9f) + 1;
        if (kWaves == 4) {
            if (a.n_seqs > 1 && a.n_seqs <= kLevelled && a.n_q > a.n_seqs && quota >= kWorthLevelling && quota < 1u << 27) quota = level_out(a, tiles, steps, total, quota, item);
            if (quota == 0) return false;
            if (blockIdx.x == 0 && threadIdx.x == 0) *a.quota = quota;
        }
    } else if (kWaves == 4 && a.n_seqs > 64) {
        uint32_t tile;
        const uint32_t s = sequence_of_slot(a.q_starts, a.n_seqs, item, a.group, 7, &tile);
        const int32_t from = a.q_starts[s], to = a.q_starts[s + 1];
        if (from < 0 || to < from || (uint32_t)to > a.n_q) return false;
        const uint32_t n_rows = (uint32_t)(to - from) * a.group;
        if (tile > n_rows / kTile || tile * kTile >= n_rows) return false;
        p->seq = s, p->q0 = from, p->n_q = to - from;
        p->n_k = (uint32_t)min((int64_t)max(a.lens[s], 0), (int64_t)a.t.width << a.c.shift);
        p->tile = tile, p->part = 0, p->parts = 1, p->per = ~0u, p->place = 0;
        return true;
    }
    uint32_t sum_before = 0, places_before = 0;
    for (uint32_t s0 = 0; s0 < a.n_seqs; s0 += 64) {
        if (!kSplit || (kJoin && kWaves == 4) || a.n_seqs > 64) look(s0);
        uint32_t parts = kSplit ? max(1u, min((steps + quota / 2) / quota, steps >> a.least_shift)) : 1;
        // (a few parts more than run at a time would take as long as twice as many)
        if (kSplit && kWaves == 4 && a.n_seqs == 1 && tiles * parts > a.at_a_time && tiles <= a.at_a_time) parts = a.at_a_time / tiles;
        if (kSplit && kWaves == 8) {
            const uint32_t before = n_k > n_q ? n_k - n_q : 0;       // (the first tile's steps, without its own keys')
            parts = parts_of_one(a, of_lane(tiles, 0), a.causal ? min(of_lane(steps, 0), of_lane(before, 0) / kPromptKeys + 1) : of_lane(steps, 0), of_lane(steps, 0), parts);
        }
        const uint32_t places = parts > 1 ? tiles * parts : 0, items = kJoin ? (parts > 1 ? tiles : 0) : tiles * parts;
        const uint32_t items_to = over_lanes(items, 0u, Add{}), places_to = kSplit ? over_lanes(places, 0u, Add{}) : 0;
        uint32_t before = sum_before + items_to - items;
        if (kWaves == 4 && kSplit && !kJoin && a.n_seqs <= 64) before = items_before(a.n_seqs, (steps + parts - 1) / parts, items);
        const uint64_t found = __ballot(item >= before && item - before < items);
        if (found) {
            const uint32_t x = (uint32_t)__builtin_ctzll(found);
            p->seq = s0 + x;
            p->q0 = of_lane(q0, x);
            p->n_q = of_lane(n_q, x);
            p->n_k = of_lane(n_k, x);
            p->parts = of_lane(parts, x);
            p->per = kSplit ? (of_lane(steps, x) + p->parts - 1) / p->parts : ~0u;
            const uint32_t in = item - of_lane(before, x), by = kJoin ? 1 : p->parts, at = in / by;
            p->part = in - at * by;
            // (the last tiles of a sequence, which see the most keys, come first)
            p->tile = of_lane(tiles, x) - 1 - at;
            p->place = places_before + of_lane(places_to - places, x) + at * p->parts;
            // (starts that do not ascend may make more of them than there are places)
            return p->parts == 1 || p->place + p->parts <= a.places;
        }
        sum_before += of_lane(items_to, 63);
        places_before += of_lane(places_to, 63);
    }
    return false;
}

// The keys that a query sees: those below `end`, of these those from `begin` on
// and the sinks.
struct Seen {
    uint32_t begin, end;
};

__device__ __forceinline__ Seen seen_by(const ChunkArgs &a, uint32_t query, uint32_t n_q, uint32_t n_k) {
    if (!a.causal) return Seen{0, n_k};
    const int64_t l = (int64_t)query + 1 + n_k - n_q;
    const uint32_t end = l < 0 ? 0 : l > n_k ? n_k : (uint32_t)l;
    return Seen{a.window && end > a.window ? end - a.window : 0, end};
}

// The steps of a tile: those of the sinks, then those of the window.
struct Steps {
    uint32_t sinks, skipped, n;
    __device__ __forceinline__ uint32_t key(uint32_t step) const { return (step < sinks ? step : step + skipped) * kPromptKeys; }
};

__device__ __forceinline__ Steps steps_of(const ChunkArgs &a, const Piece &p, uint32_t tile_rows) {
    const uint32_t row0 = p.tile * tile_rows, n_rows = p.n_q * a.group;
    const Seen first = seen_by(a, over_group(a, row0), p.n_q, p.n_k);
    const uint32_t end = seen_by(a, over_group(a, min(row0 + tile_rows, n_rows) - 1), p.n_q, p.n_k).end;
    Steps s;
    s.sinks = min((a.sinks + kPromptKeys - 1) / kPromptKeys, first.begin / kPromptKeys);
    s.skipped = first.begin / kPromptKeys - s.sinks;
    s.n = (end + kPromptKeys - 1) / kPromptKeys - s.skipped;
    return s;
}

// 64 entries of a sequence's table, a lane each, asked for before they are used.
struct Entries {
    const int32_t *pages;
    uint32_t last, from, held;      // the last entry of the sequence; the first in `held`
    __device__ __forceinline__ void read(const ChunkArgs &a, uint32_t key) {
        from = key >> a.c.shift;
        held = (uint32_t)pages[min(from + (threadIdx.x & 63u), last)];
    }
    // those of n keys from `key` on
    __device__ __forceinline__ void need(const ChunkArgs &a, uint32_t key, uint32_t n) {
        if (key >> a.c.shift < from || (key + n - 1) >> a.c.shift > from + 63) read(a, key);
    }
    // The cache's row of key `key`, the first of 16 (the host keeps the rows'
    // number below 2^32).
    __device__ __forceinline__ uint32_t row(const ChunkArgs &a, uint32_t kv_head, uint32_t key) const {
        const uint32_t page = min(of_lane(held, (key >> a.c.shift) - from), a.c.n_pages - 1);
        return ((page * a.c.kv_heads + kv_head) << a.c.shift) + (key & ((1u << a.c.shift) - 1));
    }
};

// A part of a sequence of one new token (the queries of a kv head's group, at
// most 16, are columns): its waves take 32 keys in turn, as in attend_token.hip,
// each with the next ones' rows in registers and a tile of its own in LDS, and
// are joined through LDS at the end.  Bound by HBM traffic: 128 KB in flight on
// a compute unit, where the tiles of 128 rows have 64 (32 sequences of 1 to
// 8192 keys, 500 MB: 96 us, 5.2 TB/s).  own: the wave's LDS, of
// max(32 rows, 16 columns of D + 4 floats) bytes; area(w): wave w's.
template <int D, bool kInt8, class Area>
__device__ __forceinline__ void attend_single(const ChunkArgs &a, const Piece &p, const Steps &steps, uint32_t step_begin, uint32_t step_end, bool whole,
                                              uint32_t kv_head, uint32_t wave, const Area &area, float (*ml)[2][16]) {
    constexpr uint32_t kWaves = 4, kThreads = 64 * kWaves;
    constexpr int kRow = kInt8 ? D : 2 * D;            // bytes of a stored row
    constexpr int kChunks = kRow / 16;                 // 16-byte chunks of it
    constexpr int kLoads = kTokenKeys * kChunks / 64;  // chunks a lane loads of 32 K rows, and of V rows
    constexpr int kDTiles = D / 16;
    constexpr int kOStride = D + 4;
    const uint32_t lane0 = threadIdx.x & 63u, lane = lane0, col = lane & 15u, grp = lane >> 4;
    const Seen seen = seen_by(a, 0, 1, p.n_k);
    const uint32_t n_k = p.n_k;
    u32x4 q[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        q[i] = u32x4{0, 0, 0, 0};
        if (col < a.group)
            q[i] = *reinterpret_cast<const u32x4 *>(a.q.data + (int64_t)p.q0 * a.q.row + (kv_head * a.group + col) * a.q.head + column_operand_at<kInt8>(i, grp));
    }
    f32x4 o[kDTiles];
#pragma unroll
    for (int i = 0; i < kDTiles; ++i) o[i] = f32x4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0;
    const float log2_n = log2_up(n_k);
    uint8_t *const tile = area(wave);

    Entries entries{a.t.pages + p.seq * a.t.stride, (n_k - 1) >> a.c.shift, 0, 0};
    u32x4 kw[kLoads], vw[kLoads];
    f32x4 ks[2], vs[2];
    uint32_t half_row[2];
    const uint32_t last_half = (n_k - 1) & ~15u;
    const auto key_of = [&](uint32_t turn) { return steps.key(turn >> 1) + (turn & 1) * kTokenKeys; };
    // (halves past the end repeat the last one)
    const auto find_rows = [&](uint32_t key0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) half_row[t] = entries.row(a, kv_head, min(key0 + 16 * t, last_half));
    };
    const auto load = [&](const uint8_t *pages, u32x4 *w) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const u32x4 *const half = reinterpret_cast<const u32x4 *>(pages + (uint64_t)half_row[2 * i / kLoads] * kRow);
            w[i] = __builtin_nontemporal_load(half + i % (kLoads / 2) * 64 + lane0);
        }
    };
    const auto load_scales = [&] {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            ks[t] = reinterpret_cast<const f32x4 *>(a.c.k_scale + half_row[t])[grp];
            vs[t] = reinterpret_cast<const f32x4 *>(a.c.v_scale + half_row[t])[grp];
        }
    };
    // LDS keeps a wave's accesses in order; this keeps the compiler's.
    const auto handed_over = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
    };
    uint32_t turn = 2 * step_begin + wave;
    const uint32_t turns = 2 * step_end;
    if (turn < turns) entries.read(a, min(key_of(turn), last_half));
    // (the queries are here before the loop, so that its products do not wait for
    // what is loaded in it)
#pragma unroll
    for (int i = 0; i < D / 32; ++i) asm volatile("" : "+v"(q[i]));
    __builtin_amdgcn_s_waitcnt(0x0F70);
    if (turn < turns) {
        // (a turn past the sequence's end is not taken)
        find_rows(key_of(turn));
        if (turn + kWaves < turns) entries.need(a, min(key_of(turn + kWaves), last_half), kTokenKeys);
        load(a.c.k, kw);
        load(a.c.v, vw);
        if (kInt8) load_scales();
    }
    for (; turn < turns; turn += kWaves) {
        const uint32_t key0 = key_of(turn), next = turn + kWaves;
        if (key0 >= n_k) break;
        uint32_t lane = lane0;
        asm volatile("" : "+v"(lane));
        const uint32_t grp = lane >> 4;
        handed_over();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t at = i * 64 + lane;
            *reinterpret_cast<u32x4 *>(tile + column_k_at<kRow>(at / kChunks, at % kChunks)) = kw[i];
        }
        handed_over();
        if (next < turns) find_rows(key_of(next));
        if (next + kWaves < turns) entries.need(a, min(key_of(next + kWaves), last_half), kTokenKeys);
        load(a.c.k, kw);                       // (past the end: the last rows once more, which nobody uses)
        __builtin_amdgcn_sched_barrier(0);
        f32x4 s[2];
        column_scores<D, kInt8>(tile, lane, [&](int i) { return q[i]; }, s);
        const bool masked = key0 + kTokenKeys > seen.end || (key0 < seen.begin && key0 + kTokenKeys > a.sinks);
        const auto out_of_sight = [&](uint32_t key) { return (key >= seen.end) | ((key < seen.begin) & (key >= a.sinks)); };
        if (masked) {
            // weights of rows that are not seen are 0, and 0 times an infinity would be NaN
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool out = out_of_sight(key0 + (i * 64 + lane) / kChunks);
#pragma unroll
                for (int x = 0; x < 4; ++x) vw[i][x] = out ? 0 : vw[i][x];
            }
        }
        handed_over();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t at = i * 64 + lane;
            *reinterpret_cast<u32x4 *>(tile + column_v_at<kRow, kInt8>(at / kChunks, at % kChunks)) = vw[i];
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
        if (masked) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool out = out_of_sight(key0 + 16 * t + 4 * grp + i);
                    s[t][i] = out ? -__builtin_inff() : s[t][i];
                    if (kInt8) v_scale[t][i] = out ? 0 : v_scale[t][i];
                }
        }
        column_update<D, kInt8>(tile, lane, s, v_scale, kInt8 ? 1.0f : a.log2_scale, log2_n, o, m, l);
    }
    f32x2 two = with_lane_16(l);
    two = with_lane_32(two.x + two.y);
    l = two.x + two.y;

    // join the waves
    if (lane < 16) {
        ml[wave][0][lane] = m;
        ml[wave][1][lane] = l;
    }
    __syncthreads();
    float most = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < (int)kWaves; ++w) most = fmaxf(most, ml[w][0][col]);
    const float weight = exp2_fast(m - (most == -__builtin_inff() ? 0.0f : most));
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
        *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(tile) + col * kOStride + 16 * i + 4 * grp) = o[i] * weight;
    __syncthreads();
    for (uint32_t at = threadIdx.x; at < a.group * (D / 4); at += kThreads) {
        const uint32_t c = at / (D / 4), d = at % (D / 4) * 4;
        f32x4 sum = {0, 0, 0, 0};
        float most_c = -__builtin_inff(), l_c = 0;
#pragma unroll
        for (int w = 0; w < (int)kWaves; ++w) most_c = fmaxf(most_c, ml[w][0][c]);
        const float base_c = most_c == -__builtin_inff() ? 0.0f : most_c;
#pragma unroll
        for (int w = 0; w < (int)kWaves; ++w) {
            sum += *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(area(w)) + c * kOStride + d);
            l_c += ml[w][1][c] * exp2_fast(ml[w][0][c] - base_c);
        }
        if (whole) {
            const float inv = l_c == 0.0f ? 0.0f : 1.0f / l_c;
            *reinterpret_cast<u32x2 *>(a.out.data + (int64_t)p.q0 * a.out.row + (kv_head * a.group + c) * a.out.head + d) =
                u32x2{pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv)};
        } else {
            // where the lanes of a tile of 32 rows would hold it, for the join
            const uint64_t at_part = ((uint64_t)(p.place + p.part) * a.c.kv_heads + kv_head) * kWaves;
            reinterpret_cast<f32x4 *>(a.part)[at_part * (D / 32 * 4 * 64) + d / 8 * 64 + (d / 4 & 1) * 32 + c] = sum;
            if (d == 0) reinterpret_cast<f32x2 *>(a.part_ml)[at_part * kWaveRows + c] = f32x2{most_c, l_c};
        }
    }
}

template <int D, bool kInt8, bool kSplit, uint32_t kWaves>
__global__ __launch_bounds__(64 * kWaves, kWaves == 4 && D == 64 ? 3 : 2) void attend_chunk_kernel(ChunkArgs a) {
    constexpr uint32_t kThreads = 64 * kWaves, kTile = kWaves * kWaveRows;
    constexpr int kChunks = D / 8;                           // 16-byte chunks of a row of words
    constexpr int kLoads = kPromptKeys * kChunks / kThreads; // chunks of words a thread stages
    constexpr int kCodeLoads = (kLoads + 1) / 2;             // chunks of codes
    constexpr int kDTiles = D / 32;
    constexpr int kDSteps = D / 16;
    __shared__ __attribute__((aligned(16))) uint8_t kt0[kPromptKeys * D * 2], kt1[kPromptKeys * D * 2];
    __shared__ __attribute__((aligned(16))) uint8_t vt0[kPromptKeys * D * 2], vt1[kPromptKeys * D * 2];
    __shared__ __attribute__((aligned(16))) float sc0[kInt8 ? 2 * kPromptKeys : 4], sc1[kInt8 ? 2 * kPromptKeys : 4];

    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane_of_wave = lane, col = lane & 31u, half = lane >> 5;

    // (workgroups are dealt to the eight XCDs in turn: kv heads vary fastest,
    // so that the tiles of one meet in one L2)
    const uint32_t kv_head = blockIdx.x % a.c.kv_heads;
    Piece p;
    if (!find_piece<kWaves, kSplit, false>(a, blockIdx.x / a.c.kv_heads, &p)) return;
    const uint32_t n_q = p.n_q, n_k = p.n_k, n_rows = n_q * a.group;
    const uint32_t row0 = p.tile * kTile;
    const Steps steps = steps_of(a, p, kTile);
    uint32_t step_begin = 0, step_end = steps.n;
    bool whole = true;
    if (kSplit) {
        step_begin = p.part * p.per;
        if (step_begin >= steps.n && p.part) return;
        step_end = min(step_begin + p.per, steps.n);
        whole = steps.n <= p.per;
    }

    if constexpr (kWaves == 4) {
        if (n_q == 1 && a.group <= 16) {
            __shared__ float ml[kWaves][2][16];
            const auto area = [&](uint32_t w) { return w == 0 ? kt0 : w == 1 ? kt1 : w == 2 ? vt0 : vt1; };
            attend_single<D, kInt8>(a, p, steps, step_begin, step_end, whole, kv_head, wave, area, ml);
            return;
        }
    }

    const uint32_t wave_first = row0 + wave * kWaveRows, row = wave_first + col;
    const bool real = row < n_rows;
    const uint32_t query = over_group(a, row), head = kv_head * a.group + row - query * a.group;
    // (rows past the last compute on zero queries, and are not stored)
    const Seen seen = real ? seen_by(a, query, n_q, n_k) : Seen{0, n_k};
    // The wave's rows see no key from wave_end on and none below wave_begin but
    // sinks; they all see those from clear_begin (and the sinks) to clear_end.
    const Seen wave_low = seen_by(a, over_group(a, wave_first), n_q, n_k);
    const Seen wave_high = seen_by(a, over_group(a, min(wave_first + kWaveRows, n_rows) - 1), n_q, n_k);
    const uint32_t wave_begin = wave_low.begin, wave_end = wave_first < n_rows ? wave_high.end : 0;
    const uint32_t clear_begin = wave_high.begin, clear_end = wave_low.end;

    u32x4 q[kDSteps];
#pragma unroll
    for (int i = 0; i < kDSteps; ++i) {
        q[i] = u32x4{0, 0, 0, 0};
        if (real) q[i] = *reinterpret_cast<const u32x4 *>(a.q.data + (int64_t)(p.q0 + query) * a.q.row + head * a.q.head + 16 * i + 8 * half);
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

    Entries entries{a.t.pages + p.seq * a.t.stride, (n_k - 1) >> a.c.shift, 0, 0};
    const auto need_entries = [&](uint32_t key0) { entries.need(a, key0, kPromptKeys); };
    const auto row_of = [&](uint32_t key) { return entries.row(a, kv_head, key); };

    // Words: a step's K and V rows go from memory into LDS without passing
    // through registers, one step ahead: the chunk that lane `at` of the tile
    // holds is the one that belongs there.  Rows past the sequence's end are
    // out of the descriptor's range and arrive as zeros.
    constexpr uint32_t kRowsALoad = kThreads / kChunks;
    const uint32_t tile_row = threadIdx.x / kChunks, chunk = threadIdx.x % kChunks;
    const uint32_t k_offset = (tile_row & 15) * (2 * D) + 16 * k_chunk<D>(tile_row, chunk);
    const uint32_t v_offset = (tile_row & 15) * (2 * D) + 16 * v_chunk<D>(tile_row, chunk);
    const auto load = [&](uint32_t key0, uint8_t *kt, uint8_t *vt) {
        const uint32_t left = n_k - key0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint64_t at = (uint64_t)row_of(key0 + i * kRowsALoad + (kRowsALoad > 16 ? wave * (64 / kChunks) & ~15u : 0)) * (2 * D);
            const __amdgpu_buffer_rsrc_t kr = __builtin_amdgcn_make_buffer_rsrc((void *)(a.c.k + at), 0, kOutOfRange, 0x00020000);
            const __amdgpu_buffer_rsrc_t vr = __builtin_amdgcn_make_buffer_rsrc((void *)(a.c.v + at), 0, kOutOfRange, 0x00020000);
            const bool in = tile_row + i * kRowsALoad < left;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (DF11_LDS void *)(kt + (i * kThreads + wave * 64) * 16), 16, in ? k_offset : kOutOfRange, 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (DF11_LDS void *)(vt + (i * kThreads + wave * 64) * 16), 16, in ? v_offset : kOutOfRange, 0, 0, 0);
        }
    };
    const auto arrived = [&] {
        __builtin_amdgcn_s_waitcnt(0x0F70);        // vmcnt(0): this wave's rows
        __syncthreads();                           // and the others'; and all are done with the step before
    };

    // 8 bits: codes go through registers, one step ahead, and become words on
    // their way into LDS; scales beside them, K's of 64 rows and then V's.  Rows
    // past the sequence's end are what the last page holds: codes are finite, and
    // masked scores and weights of 0 do not look at the scales.
    constexpr uint32_t kCodeChunks = D / 16, kCodeRows = kThreads / kCodeChunks;
    const uint32_t code_row = threadIdx.x / kCodeChunks, code_chunk = threadIdx.x % kCodeChunks;
    const bool codes_here = kCodeRows <= kPromptKeys || wave < kWaves / 2;      // (eight waves, heads of 64: half of them have none)
    u32x4 kw[kCodeLoads], vw[kCodeLoads];
    float scale_w;
    const auto load_codes = [&](uint32_t key0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kCodeLoads; ++i) {
            if (!codes_here) break;
            // (a wave's rows: 8 or 16 neighbours)
            const uint32_t first = key0 + i * kCodeRows + wave * (64 / kCodeChunks);
            const uint64_t at = ((uint64_t)row_of(first & ~15u) + (first & 15)) * D;
            const uint32_t from = (lane / kCodeChunks) * D + 16 * code_chunk;
            kw[i] = *reinterpret_cast<const u32x4 *>(a.c.k + at + from);
            vw[i] = *reinterpret_cast<const u32x4 *>(a.c.v + at + from);
        }
        // (16 lanes share a page's row; the waves from 2 on repeat 0 and 1)
        uint32_t r = row_of(key0);
#pragma unroll
        for (int g = 1; g < 4; ++g) {
            const uint32_t other = row_of(key0 + 16 * g);
            r = (int)(lane >> 4) == g ? other : r;
        }
        scale_w = (wave & 1 ? a.c.v_scale : a.c.k_scale)[r + (lane & 15)];
    };
    const auto store_codes = [&](uint8_t *kt, uint8_t *vt, float *sc) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kCodeLoads; ++i) {
            if (!codes_here) break;
            const uint32_t r = code_row + i * kCodeRows;
            *reinterpret_cast<u32x4 *>(kt + k_at<D>(r, 2 * code_chunk)) = bf16_of_bytes8(u32x2{kw[i].x, kw[i].y});
            *reinterpret_cast<u32x4 *>(kt + k_at<D>(r, 2 * code_chunk + 1)) = bf16_of_bytes8(u32x2{kw[i].z, kw[i].w});
            *reinterpret_cast<u32x4 *>(vt + v_at<D>(r, 2 * code_chunk)) = bf16_of_bytes8(u32x2{vw[i].x, vw[i].y});
            *reinterpret_cast<u32x4 *>(vt + v_at<D>(r, 2 * code_chunk + 1)) = bf16_of_bytes8(u32x2{vw[i].z, vw[i].w});
        }
        if (wave < 2) sc[threadIdx.x] = wave ? scale_w : scale_w * a.log2_scale;     // (V's from wave 1, K's, of scores in base 2, from wave 0)
    };

    // One step's keys.  kCareful: values that are infinite or NaN at keys which
    // only some rows see do not reach the others; in 8 bits (where values are
    // finite) a weight is the sum of two operands, as in attend_columns.hpp.
    // Else a weight is rounded to one operand (errors of 0.0018 to 0.0023 of the
    // norm, of two operands 0.0013 to 0.0017): a second one is as many products
    // again with V, where products bound it (64 queries on 2001 keys 18.2 us, with
    // two operands 20.7; 2048 on 32,049 897 us and 1291, in 8 bits 1041 and 1424;
    // 16 prompts of up to 1024 tokens 91 and 110).
    const auto step = [&](auto careful, uint32_t key0, const uint8_t *kt, const uint8_t *vt, const float *sc) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(careful)::value;
        if (key0 >= wave_end || (key0 + kPromptKeys <= wave_begin && key0 >= a.sinks)) return;
        // (the careful pass computes its LDS addresses in each step: there are
        // no registers to keep them in)
        uint32_t own = lane_of_wave;
        if (kCareful) asm volatile("" : "+v"(own));
        const uint32_t lane = own, col = own & 31u, half = own >> 5;
        // (in 8 bits with heads of 64 those of K, for registers of three waves)
        uint32_t k_lane = own;
        if (kInt8 && D == 64) asm volatile("" : "+v"(k_lane));

        f32x16 s[kHalves];
#pragma unroll
        for (int t = 0; t < kHalves; ++t) s[t] = f32x16{};
#pragma unroll
        for (int i = 0; i < kDSteps; ++i)
#pragma unroll
            for (int t = 0; t < kHalves; ++t) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(kt + k_at<D>(32 * t + (k_lane & 31u), 2 * i + (k_lane >> 5)));
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
        // in base 2, less the maximum so far
        const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
        for (int t = 0; t < kHalves; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 by = {a.log2_scale, a.log2_scale, a.log2_scale, a.log2_scale};
                if (kInt8) by = *reinterpret_cast<const f32x4 *>(sc + 32 * t + 8 * g + 4 * half);     // (times the keys' scales)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][4 * g + i] = __builtin_fmaf(s[t][4 * g + i], by[i], -base);
            }
        if (key0 + kPromptKeys > clear_end || (key0 < clear_begin && key0 + kPromptKeys > a.sinks)) {
#pragma unroll
            for (int t = 0; t < kHalves; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t key = key0 + 32 * t + 8 * (i / 4) + 4 * half + i % 4;
                    const bool hidden = (key >= seen.end) | ((key < seen.begin) & (key >= a.sinks));     // (without branches)
                    s[t][i] = hidden ? -__builtin_inff() : s[t][i];
                }
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < kHalves; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        const f32x2 halves = with_lane_32(top);
        top = fmaxf(halves.x, halves.y);
        if (__any(top > -log2_n || m == -__builtin_inff())) {
            const float next = fmaxf(m, base + top + (kSlack + log2_n)), more = (next == -__builtin_inff() ? 0.0f : next) - base;
            const float keep = exp2_fast(m - base - more);
            m = next;
            l *= keep;
#pragma unroll
            for (int i = 0; i < kDTiles; ++i) o[i] *= keep;
#pragma unroll
            for (int t = 0; t < kHalves; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[t][i] -= more;
        }
#pragma unroll
        for (int t = 0; t < kHalves; ++t) {
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                u32x4 p, p_low;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[i] = exp2_fast(s[t][8 * st + 4 * g + i]);
                        l += e[i];
                    }
                    if (kInt8) {
                        // (a weight of 0, a masked key's too, stays 0 whatever the scale)
                        const f32x4 w = *reinterpret_cast<const f32x4 *>(sc + kPromptKeys + 32 * t + 16 * st + 8 * g + 4 * half);
#pragma unroll
                        for (int i = 0; i < 4; ++i) e[i] = mul_or_zero(e[i], w[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (kInt8 && kCareful) {
                            const u32x2 two = two_operands<true>(e[2 * i], e[2 * i + 1]);
                            p[2 * g + i] = two.x;
                            p_low[2 * g + i] = two.y;
                        } else {
                            p[2 * g + i] = pack_bf16(e[2 * i], e[2 * i + 1]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kDTiles; ++i) {
                    const uint32_t j = lane & 15u, r = 32 * t + 16 * st + 4 * half + (j >> 2);
                    const uint32_t chunk = 4 * i + 2 * ((lane >> 4) & 1u) + ((j & 3) >> 1);
                    const s16x4 b0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(vt + v_at<D>(r, chunk) + 8 * (j & 1)));
                    const s16x4 b1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DF11_LDS s16x4 *)(vt + v_at<D>(r + 8, chunk) + 8 * (j & 1)));
                    const u32x2 w0 = __builtin_bit_cast(u32x2, b0), w1 = __builtin_bit_cast(u32x2, b1);
                    u32x4 w = {w0.x, w0.y, w1.x, w1.y};
                    if constexpr (kCareful && !kInt8) {
                        // Values that are not finite leave the product (0 times
                        // one of them is not 0) and are counted apart, over the
                        // keys that the row sees (whose score is not that of a
                        // masked one): ones where they are +inf or NaN, and
                        // where they are -inf or NaN.
                        u32x4 here, up, down;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            here[x] = up[x] = down[x] = 0;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t h = w[x] >> (16 * y) & 0xFFFFu, one = 0x3F80u << (16 * y);
                                const bool odd = (h & 0x7F80u) == 0x7F80u, nan = odd && (h & 0x7Fu);
                                if (s[t][8 * st + 2 * x + y] != -__builtin_inff()) here[x] |= one;
                                if (nan || h == 0x7F80u) up[x] |= one;
                                if (nan || h == 0xFF80u) down[x] |= one;
                                if (odd) w[x] &= 0xFFFF0000u >> (16 * y);
                            }
                        }
                        f32x16 n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(up), as_bf16x8(here), f32x16{}, 0, 0, 0);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (n[x] > 0) o[i][x] += __builtin_inff();
                        __builtin_amdgcn_sched_barrier(0);
                        n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(down), as_bf16x8(here), f32x16{}, 0, 0, 0);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (n[x] > 0) o[i][x] -= __builtin_inff();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), as_bf16x8(p), o[i], 0, 0, 0);
                    if constexpr (kInt8 && kCareful) {
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), as_bf16x8(p_low), o[i], 0, 0, 0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
    };

    start();
    if (step_begin < step_end) entries.read(a, steps.key(step_begin));
    if constexpr (kInt8) {
        if (step_begin < step_end) {
            load_codes(steps.key(step_begin));
            if (step_begin + 1 < step_end) need_entries(steps.key(step_begin + 1));
            store_codes(kt0, vt0, sc0);
        }
        const auto go = [&](auto careful, uint32_t i, const uint8_t *kt, const uint8_t *vt, const float *sc, uint8_t *kt_next, uint8_t *vt_next, float *sc_next) __attribute__((always_inline)) {
            __syncthreads();
            const bool more = i + 1 < step_end;
            if (more) load_codes(steps.key(i + 1));
            if (i + 2 < step_end) need_entries(steps.key(i + 2));
            step(careful, steps.key(i), kt, vt, sc);
            if (more) store_codes(kt_next, vt_next, sc_next);
        };
        // (the queries are here too: said outside the loop, so that its products
        // do not wait for what is loaded in it)
        __builtin_amdgcn_s_waitcnt(0x0F70);
        // A weight times its value's scale is rounded: that of a key which carries
        // most of a row, too, where words have a power of two.  Over many keys
        // that adds as much as rounding the result does (0.0022 of the norm
        // against 0.0017), where keys are few up to 0.0027; tiles of few steps
        // therefore have weights of two operands (0.0017; 16 prompts of up to
        // 1024 tokens 108 us and 96).
        if (steps.n > kFewSteps) {
            for (uint32_t i = step_begin; i < step_end; i += 2) {
                go(std::false_type{}, i, kt0, vt0, sc0, kt1, vt1, sc1);
                if (i + 1 < step_end) go(std::false_type{}, i + 1, kt1, vt1, sc1, kt0, vt0, sc0);
            }
        } else {
            for (uint32_t i = step_begin; i < step_end; ++i) {
                const bool odd = (i - step_begin) & 1;
                go(std::true_type{}, i, odd ? kt1 : kt0, odd ? vt1 : vt0, odd ? sc1 : sc0, odd ? kt0 : kt1, odd ? vt0 : vt1, odd ? sc0 : sc1);
            }
        }
    } else {
        if (step_begin < step_end) load(steps.key(step_begin), kt0, vt0);
        if (step_begin + 1 < step_end) need_entries(steps.key(step_begin + 1));
        const auto go = [&](uint32_t i, const uint8_t *kt, const uint8_t *vt, uint8_t *kt_next, uint8_t *vt_next) {
            arrived();
            if (i + 1 < step_end) load(steps.key(i + 1), kt_next, vt_next);
            if (i + 2 < step_end) need_entries(steps.key(i + 2));
            step(std::false_type{}, steps.key(i), kt, vt, nullptr);
        };
        for (uint32_t i = step_begin; i < step_end; i += 2) {
            go(i, kt0, vt0, kt1, vt1);
            if (i + 1 < step_end) go(i + 1, kt1, vt1, kt0, vt0);
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
                for (uint32_t i = step_begin; i < step_end; ++i) {
                    need_entries(steps.key(i));
                    load(steps.key(i), kt0, vt0);
                    arrived();
                    step(std::true_type{}, steps.key(i), kt0, vt0, nullptr);
                    __syncthreads();
                }
            }
        }
    }
    const f32x2 l_halves = with_lane_32(l);
    l = l_halves.x + l_halves.y;
    if (kSplit && !whole) {
        if (wave_first >= n_rows) return;
        // as the lanes hold them, for the lanes of the join
        const uint64_t at = ((uint64_t)(p.place + p.part) * a.c.kv_heads + kv_head) * kWaves + wave;
        f32x4 *const part = reinterpret_cast<f32x4 *>(a.part) + at * (kDTiles * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < kDTiles; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) part[(4 * i + g) * 64] = f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
        if (half == 0) reinterpret_cast<f32x2 *>(a.part_ml)[at * kWaveRows + col] = f32x2{m, l};
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *const op = a.out.data + (int64_t)(p.q0 + query) * a.out.row + head * a.out.head;
#pragma unroll
    for (int i = 0; i < kDTiles; ++i) store_tile(o[i] * inv, op + 32 * i, half, real);
}

// Tiles that may be split: of a kv head, each in two parts at least.
__host__ __device__ __forceinline__ uint32_t split_tiles(const ChunkArgs &a) { return a.places / 2 < a.tile_slots ? a.places / 2 : a.tile_slots; }

// Joins the parts of 32 rows (those of one wave of a split tile) after another:
// out = sum_a w_a o_a / sum_a w_a l_a with w_a = 2^(m_a - max m), the maximum
// taken as the parts come.  A wave takes 16 columns, so that few tiles are many
// waves' work and the parts of most are all in flight at once.  How many tiles
// are split the host does not know: as many workgroups are launched as run at a
// time, and end when there are no more (one for each tile that the workspace
// could hold took 8 to 10 us to find nothing).
template <int D, uint32_t kWaves>
__global__ __launch_bounds__(64 * D / 16) void join_chunk_kernel(ChunkArgs a) {
    constexpr int kDTiles = D / 32;
    constexpr int kBatch = 8;       // parts in flight
    const uint32_t lane = threadIdx.x & 63u, i = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t col = lane & 31u, half = lane >> 5;
    for (uint32_t n = blockIdx.x; n < split_tiles(a) * a.c.kv_heads * kWaves; n += gridDim.x) {
        const uint32_t kv_head = n % a.c.kv_heads, wave = n / a.c.kv_heads % kWaves;
        Piece p;
        if (!find_piece<kWaves, true, true>(a, n / a.c.kv_heads / kWaves, &p)) return;
        const uint32_t first = (p.tile * kWaves + wave) * kWaveRows, row = first + col, n_rows = p.n_q * a.group;
        const uint32_t n_steps = steps_of(a, p, kWaves * kWaveRows).n;
        if (first >= n_rows || n_steps <= p.per) continue;
        const uint32_t parts = (n_steps + p.per - 1) / p.per;
        const uint64_t at = ((uint64_t)p.place * a.c.kv_heads + kv_head) * kWaves + wave, next_part = (uint64_t)a.c.kv_heads * kWaves;
        const f32x2 *const ml = reinterpret_cast<const f32x2 *>(a.part_ml) + at * kWaveRows + col;
        const f32x4 *const part = reinterpret_cast<const f32x4 *>(a.part) + at * (kDTiles * 256) + i * 128 + lane;
        f32x4 o[2] = {};
        float l = 0, m = -__builtin_inff();
        for (uint32_t s = 0; s < parts; s += kBatch) {
            f32x2 stat[kBatch];
            f32x4 v[kBatch][2];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                if (s + x >= parts) break;      // (a part past the last was not written)
                stat[x] = ml[(s + x) * next_part * kWaveRows];
#pragma unroll
                for (int g = 0; g < 2; ++g) v[x][g] = part[(s + x) * next_part * (kDTiles * 256) + g * 64];
            }
            float next = m;
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                if (s + x >= parts) break;
                next = fmaxf(next, stat[x].x);
            }
            const float base = next == -__builtin_inff() ? 0.0f : next, keep = exp2_fast(m - base);
            m = next;
            l *= keep;
            o[0] *= keep;
            o[1] *= keep;
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                if (s + x >= parts) break;
                const float w = exp2_fast(stat[x].x - base);
                l += w * stat[x].y;
                o[0] += w * v[x][0];
                o[1] += w * v[x][1];
            }
        }
        const uint32_t query = over_group(a, row), head = kv_head * a.group + row - query * a.group;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        store_16(o[0] * inv, o[1] * inv, a.out.data + (int64_t)(p.q0 + query) * a.out.row + head * a.out.head + 16 * i, half, row < n_rows);
    }
}

template <int D, bool kInt8, uint32_t kWaves>
auto kernel_of(bool split) {
    return split ? attend_chunk_kernel<D, kInt8, true, kWaves> : attend_chunk_kernel<D, kInt8, false, kWaves>;
}

template <uint32_t kWaves>
hipError_t launch(const ChunkArgs &a, uint32_t head_dim, bool int8, hipStream_t stream) {
    const bool split = a.places != 0;
    const auto kernel = head_dim == 64 ? (int8 ? kernel_of<64, true, kWaves>(split) : kernel_of<64, false, kWaves>(split))
                                       : (int8 ? kernel_of<128, true, kWaves>(split) : kernel_of<128, false, kWaves>(split));
    // (a single sequence is whole, or all of its parts have places)
    const uint32_t items = kWaves == 4 ? a.tile_slots + a.places : a.tile_slots > a.places ? a.tile_slots : a.places;
    hipLaunchKernelGGL(kernel, dim3(items * a.c.kv_heads), dim3(64 * kWaves), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !split) return e;
    // (2048 threads for each compute unit)
    const uint32_t rows_32 = split_tiles(a) * a.c.kv_heads * kWaves, at_a_time = a.at_a_time * a.c.kv_heads * kWaves / 2 * (128 / head_dim);
    hipLaunchKernelGGL((head_dim == 64 ? join_chunk_kernel<64, kWaves> : join_chunk_kernel<128, kWaves>), dim3(rows_32 < at_a_time ? rows_32 : at_a_time),
                       dim3(4 * head_dim), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_chunk(const ChunkArgs &a, uint32_t head_dim, bool int8, hipStream_t stream) {
    return a.tile_rows == 8 * kWaveRows ? launch<8>(a, head_dim, int8, stream) : launch<4>(a, head_dim, int8, stream);
}

}  // namespace df11
