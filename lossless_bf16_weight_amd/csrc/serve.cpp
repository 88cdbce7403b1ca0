// Host side of the serving operators (key-value cache and attention, C ABI in
// include/df11.h): argument checks, the split of the work, launches.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "serve_internal.hpp"

using namespace df11;

namespace {

constexpr uint64_t kMostGroups = (uint64_t(1) << 24) - 1;   // workgroups of 256 along x: threads stay below 2^32
constexpr int64_t kMostStride = int64_t(1) << 32;
// a step's key rows lie within 2^31 bytes of the first (attend_prompt.hip's descriptors)
constexpr int64_t kMostKeyStride = ((int64_t(1) << 31) - 256) / (2 * kPromptKeys);

struct Device {
    int prev = -1;
    hipError_t err = hipSuccess;
    explicit Device(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) prev = -1;
        if (prev != dev) err = hipSetDevice(dev);
        else prev = -1;
    }
    ~Device() {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

// Compute units of a device (256 where it cannot be asked: the split of the
// work follows it, no result does).
uint32_t compute_units(int dev) {
    static std::atomic<int> known[64];
    if (dev < 0 || dev >= 64) return 256;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) {
            (void)hipGetLastError();
            return 256;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return (uint32_t)n;
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

bool misaligned(const void *p) { return ((uintptr_t)p & 15) != 0; }

df11_status check_rows(const char *what, const df11_rows &r, uint64_t n, uint64_t heads, uint64_t d, bool written) {
    if (n == 0) return DF11_OK;
    if (!r.data || misaligned(r.data)) return report_error(DF11_E_ARG, "%s: NULL or not 16-byte aligned", what);
    if (r.row_stride < 0 || r.head_stride < 0 || r.row_stride >= kMostStride || r.head_stride >= kMostStride ||
        (r.row_stride | r.head_stride) & 7)
        return report_error(DF11_E_ARG, "%s: strides must be multiples of 8 from 0 to below 2^32", what);
    if (!written) return DF11_OK;
    const uint64_t row = n > 1 ? (uint64_t)r.row_stride : ~uint64_t(0), head = heads > 1 ? (uint64_t)r.head_stride : ~uint64_t(0);
    const bool heads_inside = head >= d && row >= (heads > 1 ? (heads - 1) * head : 0) + d;
    const bool rows_inside = row >= d && head >= (n > 1 ? (n - 1) * row : 0) + d;
    if (!heads_inside && !rows_inside) return report_error(DF11_E_ARG, "%s: rows that are written overlap", what);
    return DF11_OK;
}

Rows rows_of(const df11_rows &r) { return Rows{(uint16_t *)r.data, r.row_stride, r.head_stride}; }

df11_status check_cache_sizes(const df11_kv_cache &c) {
    if (c.store > DF11_KV_INT8) return report_error(DF11_E_ARG, "cache: store %u", c.store);
    if (c.head_dim != 64 && c.head_dim != 128) return report_error(DF11_E_UNSUPPORTED, "cache: head_dim %u, 64 and 128 are built", c.head_dim);
    if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)))
        return report_error(DF11_E_ARG, "cache: page_size %u, a power of two from 16 to 1024 is needed", c.page_size);
    if (c.n_pages == 0 || c.n_pages > 0x7FFFFFFFu || c.n_kv_heads == 0 || c.n_kv_heads > 65535)
        return report_error(DF11_E_ARG, "cache: %u pages, %u kv heads", c.n_pages, c.n_kv_heads);
    if ((uint64_t)c.n_pages * c.n_kv_heads * c.page_size > 0xFFFFFFFFull)
        return report_error(DF11_E_UNSUPPORTED, "cache: 2^32 rows or more");
    return DF11_OK;
}

df11_status check_cache(const df11_kv_cache &c) {
    df11_status st = check_cache_sizes(c);
    if (st) return st;
    if (!c.k || !c.v || misaligned(c.k) || misaligned(c.v)) return report_error(DF11_E_ARG, "cache: pages NULL or not 16-byte aligned");
    if (c.store == DF11_KV_INT8 && (!c.k_scale || !c.v_scale || misaligned(c.k_scale) || misaligned(c.v_scale)))
        return report_error(DF11_E_ARG, "cache: scales NULL or not 16-byte aligned");
    return DF11_OK;
}

CacheView view_of(const df11_kv_cache &c) {
    const uint32_t shift = (uint32_t)__builtin_ctz(c.page_size);
    return CacheView{(uint8_t *)c.k, (uint8_t *)c.v, c.k_scale, c.v_scale, (int64_t)c.n_pages << shift, c.n_pages, shift, c.n_kv_heads};
}

df11_status check_table(const df11_page_table &t, const df11_kv_cache &c) {
    if (!t.pages || ((uintptr_t)t.pages & 3)) return report_error(DF11_E_ARG, "page table: NULL or misaligned");
    if (t.row_stride < 0) return report_error(DF11_E_ARG, "page table: negative stride");
    if (t.width == 0) return report_error(DF11_E_ARG, "page table: no entries");
    if ((uint64_t)t.width * c.page_size > (uint64_t(1) << 28))
        return report_error(DF11_E_UNSUPPORTED, "page table: more than 2^28 positions a sequence");
    return DF11_OK;
}

Tables tables_of(const df11_page_table &t) { return Tables{t.pages, t.row_stride, t.width}; }

bool bad_index(const void *p, size_t size) { return !p || ((uintptr_t)p & (size - 1)); }

df11_status launched(hipError_t e, const char *what) {
    return e == hipSuccess ? DF11_OK : report_error(DF11_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

// x / n = (x * magic >> 32) >> shift for n > 1: with 2^shift < n <= 2^(shift + 1)
// and the multiplier rounded up from 2^(32 + shift) / n, the quotient is exact
// for x < 2^31.
void divide_by(uint32_t n, uint32_t *magic, uint32_t *shift) {
    *shift = n > 1 ? 31 - (uint32_t)__builtin_clz(n - 1) : 0;
    *magic = n > 1 ? (uint32_t)((((uint64_t)1 << (32 + *shift)) + n - 1) / n) : 0;
}

float log2_scale(float scale) { return (float)((double)scale * 1.4426950408889634074); }

df11_status check_rotation(const df11_rotation &r, uint32_t head_dim) {
    if (r.flags & ~DF11_ROTATE_NEIGHBOURS) return report_error(DF11_E_ARG, "rotation: flags %u", r.flags);
    if (r.pairs % 8 || r.pairs > head_dim / 2) return report_error(DF11_E_ARG, "rotation: %u pairs, a multiple of 8 up to %u is needed", r.pairs, head_dim / 2);
    if (r.pairs == 0) return DF11_OK;
    if (!r.turns || misaligned(r.turns)) return report_error(DF11_E_ARG, "rotation: turns NULL or not 16-byte aligned");
    if (misaligned(r.axes)) return report_error(DF11_E_ARG, "rotation: axes not 16-byte aligned");
    if (r.n_axes < 1 || r.n_axes > 4) return report_error(DF11_E_ARG, "rotation: %u axes, 1 to 4 are needed", r.n_axes);
    if (!r.positions || ((uintptr_t)r.positions & 3)) return report_error(DF11_E_ARG, "rotation: positions NULL or misaligned");
    if (r.position_stride < 0 || r.position_stride >= kMostStride) return report_error(DF11_E_ARG, "rotation: position_stride must be from 0 to below 2^32");
    if (!std::isfinite(r.factor)) return report_error(DF11_E_ARG, "rotation: a finite factor is needed");
    return DF11_OK;
}

df11_status check_norms(const void *q_weight, const void *k_weight, float eps) {
    if (misaligned(q_weight) || misaligned(k_weight)) return report_error(DF11_E_ARG, "weights: not 16-byte aligned");
    if ((q_weight || k_weight) && !(eps >= 0x1p-100f && std::isfinite(eps))) return report_error(DF11_E_ARG, "eps: a finite number from 2^-100 is needed");
    return DF11_OK;
}

// What rotate_heads and kv_append share: the rotation, the norms, and the
// waves.  A wave takes rows of one token, 64 lanes of 16 elements a step: three
// steps, which are faster than a token's five or six (15,183 tokens with norms
// 60.9 us and 66.6, 20,288 into the cache 97.1 and 101.6) and mostly than two (63.0
// and 97.3; 5,520 in 8 bits with their read 38.4 and 40.1, but 20,288 with heads of
// 64 57.0 and 55.5); fewer where tokens are few, for as many waves as run at a time.
df11_status heads_args(HeadsArgs *h, const df11_rotation &r, const void *q_weight, const void *k_weight, float eps, uint64_t n_tokens,
                       uint32_t rows, uint32_t head_dim, int dev) {
    const uint64_t steps = ceil_div((uint64_t)rows * head_dim, 64 * 16);
    const uint64_t want = std::max(ceil_div(32 * (uint64_t)compute_units(dev), n_tokens), ceil_div(steps, 3));
    h->run = (uint32_t)ceil_div(steps, std::min(want, steps));
    h->parts = (uint32_t)ceil_div(steps, h->run);
    if (n_tokens > 0x7FFFFFFFu || n_tokens * h->parts > 4 * kMostGroups)
        return report_error(DF11_E_UNSUPPORTED, "%llu tokens of %u heads", (unsigned long long)n_tokens, rows);
    h->turns = r.turns;
    h->axes = r.axes;
    h->positions = r.positions;
    h->position_stride = r.position_stride;
    h->pairs = r.pairs;
    h->n_axes = r.n_axes;
    h->factor = r.factor;
    h->q_weight = (const uint16_t *)q_weight;
    h->k_weight = (const uint16_t *)k_weight;
    h->eps = eps;
    h->eps_scaled = eps * 0x1p-68f * 0x1p-68f;
    h->n_tokens = (uint32_t)n_tokens;
    return DF11_OK;
}

// How attend_token splits: keys a workgroup takes and workgroups along a
// sequence, from the longest length that the table holds.  A step of the four
// waves is 128 keys and takes 1.3 us when little else runs, the join 2.7 us:
// one sequence of 1024 keys takes 7.7 us in parts of 128 keys and 10 us in
// parts of 384; 256 keys take 6.1 us in one part and 7.5 us in two.  Where the
// units fill the compute units, the three workgroups for each that run at a
// time are enough (16 sequences of 1024 keys: 14.9 us; with four 17.3 us; with
// head_dim 64 five would run, and three are taken all the same), in parts of at
// most 1280 keys: lengths are unequal, and no more parts than compute units
// leave some of these idle (sequences of 100001 and 7640 keys: 78 us, in parts
// of 2048 91 us; shorter parts of 512 84 us).
// Sequences of up to 1024 keys that would be split are taken whole instead by
// workgroups of twelve waves: one launch and no workspace, which a caller that
// launches call by call has 3.8 us sooner, and for 16 and more sequences the
// faster way (32 of 784 keys: 18.5 us, split 20.8 us; one of 784 keys: 9.8 us,
// split 7.4 us; of 1152 keys 11.8 us and 7.7 us).  In a captured graph, where
// the second launch costs the host nothing, one sequence would be faster split.
// The table's width stands for the lengths, which the host does not know: 64
// sequences of up to 4096 keys take 94 us with a table of that width and 107 us
// with one of 131,072 positions, whose workgroups past the lengths read a length
// and leave.
struct TokenSplit {
    uint32_t q_tiles, range, splits, whole;
};

// With a window the keys are those of its halves of 16 and the sinks', whose
// ranges begin anywhere.
struct Window {
    uint32_t keys, sinks;       // keys 0: none
};

// (one as long as the table is none)
Window window_of(uint32_t window, uint32_t sinks, uint64_t positions) {
    return window < positions ? Window{window, window ? (uint32_t)std::min<uint64_t>(sinks, positions) : 0} : Window{0, 0};
}

TokenSplit token_split(const df11_attend_token_args &a, const Window &w, int dev) {
    TokenSplit s;
    uint64_t most = (uint64_t)a.table.width * a.cache.page_size;
    if (w.keys) most = std::min<uint64_t>(most, (uint64_t)w.keys + 15 + ceil_div(w.sinks, 16) * 16);
    s.q_tiles = (uint32_t)ceil_div(a.n_heads / a.cache.n_kv_heads, 16);
    const uint64_t units = (uint64_t)a.n_seqs * a.cache.n_kv_heads * s.q_tiles;
    const uint64_t step = w.keys ? kTokenKeys * 4 : std::max(kTokenKeys * 4, a.cache.page_size);
    const uint64_t want = std::max<uint64_t>(1, 3 * compute_units(dev) / std::max<uint64_t>(units, 1));
    const uint64_t range = ceil_div(ceil_div(most, want), step) * step;
    const uint64_t longest = std::max<uint64_t>(kTokenRangeMax / step, 1) * step;   // (ranges begin with a page)
    s.range = (uint32_t)(most <= 2 * step ? 2 * step : std::min(range, longest));
    s.splits = (uint32_t)ceil_div(most, s.range);
    s.whole = s.splits > 1 && most <= kTokenWholeMax;
    if (s.whole) {
        s.range = (uint32_t)most;
        s.splits = 1;
    }
    return s;
}

uint64_t token_bytes(const df11_attend_token_args &a, const TokenSplit &s) {
    return s.splits == 1 ? 0 : (uint64_t)a.n_seqs * a.n_heads * s.splits * (a.cache.head_dim + 2) * sizeof(float);
}

df11_status check_token_sizes(const df11_attend_token_args &a) {
    df11_status st = check_cache_sizes(a.cache);
    if (st) return st;
    if (a.n_heads == 0 || a.n_heads % a.cache.n_kv_heads) return report_error(DF11_E_ARG, "%u heads over %u kv heads", a.n_heads, a.cache.n_kv_heads);
    if ((uint64_t)a.n_seqs * a.n_heads > kMostGroups) return report_error(DF11_E_UNSUPPORTED, "%u sequences of %u heads", a.n_seqs, a.n_heads);
    return DF11_OK;
}

uint64_t prompt_tile_slots(const df11_attend_prompt_args &a) { return a.n_q * (a.n_heads / a.n_kv_heads) / kPromptTile + a.n_seqs; }

// How attend_prompt splits the keys: where the tiles of rows (a piece of a
// prompt behind a long prefix) are fewer than compute units, into as many parts
// as give each of these two workgroups, or a few more (the rows are counted as
// if no tile but the last were part empty, each sequence's last one may be: 130
// and 35 queries of 32 heads over 8 count 42 for 56 tiles): 512 queries on 16384 keys take 148 us
// (205 us with one workgroup for each compute unit, 278 us unsplit).  How many
// keys a part has at least goes by the rows, whose parts the join reads: 256
// for less than a quarter of a tile a compute unit (32 queries on 1024 keys 14
// us, in parts of 512 17 us, unsplit 22 us; eight tokens on 2000 keys each 21
// us, unsplit 38 us), 512 for less than half (256 on 1024: 19 us, unsplit 22
// us), 1024 above (512 on 1024: 23 us, in parts of 256 28 us).  As many tiles
// as compute units are better left whole (2048 on 2048: 48 us, with the tiles
// that see more than 1024 keys in two parts 60 us).  The number of parts goes
// by the average of the sequences, whose lengths the host does not know, and
// the least by each: a tile that sees no more keys than one part has is not
// joined.
struct PromptSplit {
    uint32_t splits, part_keys;
};

PromptSplit prompt_split(const df11_attend_prompt_args &a, int dev) {
    if (a.n_q == 0 || a.n_seqs == 0) return {1, 0};
    const uint64_t full = ceil_div(a.n_q * a.n_heads, kPromptTile), cus = compute_units(dev);
    const uint64_t tiles = std::max(full, (uint64_t)a.n_seqs * a.n_kv_heads), keys = a.n_k / a.n_seqs;
    if (tiles >= cus) return {1, 0};
    const uint64_t least = 4 * full < cus ? 256 : 2 * full < cus ? 512 : 1024;
    return {(uint32_t)std::max<uint64_t>(1, std::min<uint64_t>({2 * cus / tiles, keys / least, 32})), (uint32_t)least};
}

uint64_t prompt_bytes(const df11_attend_prompt_args &a, uint32_t splits) {
    return splits == 1 ? 0 : splits * prompt_tile_slots(a) * a.n_kv_heads * kPromptTile * (a.head_dim + 2) * sizeof(float);
}

df11_status check_prompt_sizes(const df11_attend_prompt_args &a) {
    if (a.head_dim != 64 && a.head_dim != 128) return report_error(DF11_E_UNSUPPORTED, "head_dim %u, 64 and 128 are built", a.head_dim);
    if (a.n_kv_heads == 0 || a.n_heads == 0 || a.n_heads % a.n_kv_heads) return report_error(DF11_E_ARG, "%u heads over %u kv heads", a.n_heads, a.n_kv_heads);
    if (a.n_q > 0x7FFFFFFFu || a.n_k > 0x7FFFFFFFu) return report_error(DF11_E_UNSUPPORTED, "2^31 rows or more");
    // (each factor alone first: the product of two of 2^32 does not fit 64 bits)
    if (a.n_q * (a.n_heads / a.n_kv_heads) > 0x7FFFFFFFu || a.n_kv_heads > kMostGroups || a.n_seqs > kMostGroups ||
        prompt_tile_slots(a) * a.n_kv_heads > kMostGroups)
        return report_error(DF11_E_UNSUPPORTED, "%llu rows of %u heads in %u sequences", (unsigned long long)a.n_q, a.n_heads, a.n_seqs);
    return DF11_OK;
}

// What attend_chunk's workgroups need for dividing a call's work, whose lengths
// the host does not know: the parts of equal size that it would be, as many as
// workgroups run at a time, two for each compute unit (with heads of 64 three:
// three pieces of up to 1000 on 10,000 134 us, divided by two 157), and the least
// steps of one, four (64 queries on 2001 keys 17.9 us, with two 18.7, with eight 20.8;
// 36 single pieces of 16 to 200 on 700 to 30,000 keys take 2% less with two and 6%
// more with eight, 18 calls of 2, 4 and 16 sequences 3% more and 3% less).
// A tile's steps over the quota, rounded, are its parts: two from one and a half
// on, so that all split tiles have at most four thirds of the parts asked for;
// with nine sixteenths of the quota (level_out) 2.4 times as many, and so many
// places the workspace has.  (A quarter more parts for all are a second round of
// workgroups where parts are equal: 256 queries on 4256 keys 45 us and 38.)
// More than 512 sequences are taken whole, for each workgroup reads all their
// lengths: a piece of 500 on 16,000 beside 511 of 20 tokens takes 262 us, beside 512
// 466 (76 and 77 without it, alone 145).
//
// Behind a long prefix the tiles of a single sequence of 2048 rows and more have
// 256 rows and eight waves, one workgroup for each compute unit, which read keys
// and values half as often (2048 queries on 32,049 keys 936 us, with 128 rows
// 993; 1500 on 17,500 413 and 471; in 8 bits, where codes are converted half as
// often too, 1090 and 1187); and as they are nearly equal, the workgroups choose
// the parts that end soonest, among up to three times as many as run at a time.
// The length the host has from the table, of which callers give the columns in use
// (in one of 8192 positions a whole prompt of 512 tokens takes 25.6 us, in its own
// 18.1, of 2048 65 and 56): a table of four times the queries is taken for a long
// prefix (2048 on 8248 246 us and 250, 1024 on 4124 95 and 98;
// 2048 on 6144 184 and 183, on 4096 125 and 118, on 2048 68 and 60; 256 on 4256 39
// and 36).  Tiles of a whole prompt even out from 16,384 rows on (4096 tokens 151
// us and 160, 6000 306 and 299, 8192 520 and 530).  Of several sequences the
// larger tiles are harder to level out (16 prompts of up to 1024 tokens 88 us and
// 83, 64 of up to 256 61 and 55).
struct ChunkSplit {
    uint32_t most_steps, parts, places, least_shift, tile_rows;
};

constexpr uint32_t kChunkMostPlanned = 512;     // sequences

uint32_t chunk_tile_rows(const df11_attend_chunk_args &a) {
    const uint64_t rows = a.n_q * (a.n_heads / a.cache.n_kv_heads), positions = (uint64_t)a.table.width * a.cache.page_size;
    return a.n_seqs == 1 && rows >= 2048 && (rows >= 16384 || positions >= 4 * a.n_q) ? 256 : 128;
}

uint64_t chunk_tile_slots(const df11_attend_chunk_args &a) { return a.n_q * (a.n_heads / a.cache.n_kv_heads) / chunk_tile_rows(a) + a.n_seqs; }

ChunkSplit chunk_split(const df11_attend_chunk_args &a, int dev) {
    ChunkSplit s{~0u, 0, 0, 2, chunk_tile_rows(a)};
    const uint64_t group = a.n_heads / a.cache.n_kv_heads, positions = (uint64_t)a.table.width * a.cache.page_size;
    // (a tile's queries are (tile_rows - 1) / group + 2 at most, the windows of n of
    // them w + n - 1 keys, which lie in so many steps)
    const Window w = window_of(a.window, a.sinks, positions);
    if (w.keys) s.most_steps = (uint32_t)((w.keys + (s.tile_rows - 1) / group + 1 + 2 * (kPromptKeys - 1)) / kPromptKeys + ceil_div(w.sinks, kPromptKeys));
    const uint64_t steps = std::min<uint64_t>(ceil_div(positions, kPromptKeys), s.most_steps);
    const uint64_t parts = (s.tile_rows == 256 ? 1 : a.cache.head_dim == 64 ? 3 : 2) * compute_units(dev) / a.cache.n_kv_heads, of_tile = steps >> s.least_shift;
    if (a.n_q == 0 || a.n_seqs == 0 || a.n_seqs > kChunkMostPlanned || parts < 2 || of_tile < 2) return s;
    s.parts = (uint32_t)parts;
    s.places = (uint32_t)std::min(s.tile_rows == 256 ? 3 * parts : 5 * parts / 2, chunk_tile_slots(a) * of_tile);
    return s;
}

uint64_t chunk_bytes(const df11_attend_chunk_args &a, const ChunkSplit &s) {
    return s.places ? (uint64_t)s.places * a.cache.n_kv_heads * s.tile_rows * (a.cache.head_dim + 2) * sizeof(float) + 16 : 0;
}

df11_status check_chunk_sizes(const df11_attend_chunk_args &a) {
    df11_status st = check_cache_sizes(a.cache);
    if (st) return st;
    const uint32_t kv = a.cache.n_kv_heads;
    if (a.n_heads == 0 || a.n_heads % kv) return report_error(DF11_E_ARG, "%u heads over %u kv heads", a.n_heads, kv);
    if (a.n_q > 0x7FFFFFFFu || a.n_q * (a.n_heads / kv) > 0x7FFFFFFFu || a.n_seqs > kMostGroups ||
        chunk_tile_slots(a) * kv > kMostGroups / 2 - 4096)     // (512 threads, and the places)
        return report_error(DF11_E_UNSUPPORTED, "%llu rows of %u heads in %u sequences", (unsigned long long)a.n_q, a.n_heads, a.n_seqs);
    if (a.flags & ~DF11_ATTEND_CAUSAL) return report_error(DF11_E_ARG, "attend_chunk: flags %u", a.flags);
    if (a.window && !(a.flags & DF11_ATTEND_CAUSAL)) return report_error(DF11_E_ARG, "attend_chunk: a window needs DF11_ATTEND_CAUSAL");
    return DF11_OK;
}

df11_status check_workspace(const void *p, uint64_t have, uint64_t need) {
    if (need == 0) return DF11_OK;
    if (!p || misaligned(p)) return report_error(DF11_E_ARG, "workspace: NULL or not 16-byte aligned");
    if (have < need) return report_error(DF11_E_ARG, "workspace: %llu bytes, %llu needed", (unsigned long long)have, (unsigned long long)need);
    return DF11_OK;
}

df11_status check_scale(float s) {
    return s > 0 && std::isfinite(log2_scale(s)) ? DF11_OK : report_error(DF11_E_ARG, "scale: a finite number above 0 is needed (and below 2^127)");
}

}  // namespace

#define TRY(expr)                    \
    do {                             \
        df11_status st_ = (expr);    \
        if (st_) return st_;         \
    } while (0)

#define ON_DEVICE(dev)                                                                                     \
    Device guard(dev);                                                                                     \
    if (guard.err != hipSuccess) return report_error(DF11_E_HIP, "hipSetDevice(%d): %s", dev, hipGetErrorString(guard.err))

extern "C" df11_status df11_kv_write(const df11_kv_write_args *a, int hip_device, hipStream_t stream) {
    if (!a) return report_error(DF11_E_ARG, "kv_write: NULL arguments");
    TRY(check_cache(a->cache));
    const uint32_t d = a->cache.head_dim, heads = a->cache.n_kv_heads;
    if (a->n_tokens > kMostGroups * kWriteChunks / ((uint64_t)heads * (d / 8))) return report_error(DF11_E_UNSUPPORTED, "kv_write: %llu tokens", (unsigned long long)a->n_tokens);
    TRY(check_rows("k", a->k, a->n_tokens, heads, d, false));
    TRY(check_rows("v", a->v, a->n_tokens, heads, d, false));
    if (a->n_tokens == 0) return DF11_OK;
    if (bad_index(a->slots, 8)) return report_error(DF11_E_ARG, "kv_write: slots NULL or misaligned");
    ON_DEVICE(hip_device);
    const WriteArgs w{view_of(a->cache), rows_of(a->k), rows_of(a->v), a->slots, (uint32_t)a->n_tokens};
    return launched(launch_kv_write(w, d, a->cache.store == DF11_KV_INT8, stream), "kv_write");
}

extern "C" df11_status df11_rotate_heads(const df11_rotate_heads_args *a, int hip_device, hipStream_t stream) {
    if (!a) return report_error(DF11_E_ARG, "rotate_heads: NULL arguments");
    if (a->head_dim != 64 && a->head_dim != 128) return report_error(DF11_E_UNSUPPORTED, "head_dim %u, 64 and 128 are built", a->head_dim);
    if (a->n_heads > 65535 || a->n_kv_heads > 65535) return report_error(DF11_E_ARG, "%u heads, %u kv heads", a->n_heads, a->n_kv_heads);
    TRY(check_norms(a->q_weight, a->k_weight, a->eps));
    if (a->n_heads) {
        TRY(check_rows("q", a->q, a->n_tokens, a->n_heads, a->head_dim, false));
        TRY(check_rows("q_out", a->q_out, a->n_tokens, a->n_heads, a->head_dim, true));
    }
    if (a->n_kv_heads) {
        TRY(check_rows("k", a->k, a->n_tokens, a->n_kv_heads, a->head_dim, false));
        TRY(check_rows("k_out", a->k_out, a->n_tokens, a->n_kv_heads, a->head_dim, true));
    }
    if (a->n_tokens == 0 || a->n_heads + a->n_kv_heads == 0) return DF11_OK;
    TRY(check_rotation(a->rotation, a->head_dim));
    HeadsArgs h{};
    TRY(heads_args(&h, a->rotation, a->q_weight, a->k_weight, a->eps, a->n_tokens, a->n_heads + a->n_kv_heads, a->head_dim, hip_device));
    h.q = rows_of(a->q);
    h.k = rows_of(a->k);
    h.q_out = rows_of(a->q_out);
    h.k_out = rows_of(a->k_out);
    h.heads = a->n_heads;
    h.kv_heads = a->n_kv_heads;
    ON_DEVICE(hip_device);
    return launched(launch_heads(h, a->head_dim, kHeadsOnly, a->rotation.flags & DF11_ROTATE_NEIGHBOURS, stream), "rotate_heads");
}

extern "C" df11_status df11_kv_append(const df11_kv_append_args *a, int hip_device, hipStream_t stream) {
    if (!a) return report_error(DF11_E_ARG, "kv_append: NULL arguments");
    TRY(check_cache(a->cache));
    const uint32_t d = a->cache.head_dim, heads = a->cache.n_kv_heads;
    if (a->n_heads > 65535) return report_error(DF11_E_ARG, "%u heads", a->n_heads);
    TRY(check_norms(a->q_weight, a->k_weight, a->eps));
    TRY(check_rows("k", a->k, a->n_tokens, heads, d, false));
    TRY(check_rows("v", a->v, a->n_tokens, heads, d, false));
    if (a->n_heads) {
        TRY(check_rows("q", a->q, a->n_tokens, a->n_heads, d, false));
        TRY(check_rows("q_out", a->q_out, a->n_tokens, a->n_heads, d, true));
    }
    if (a->k_out.data) TRY(check_rows("k_out", a->k_out, a->n_tokens, heads, d, true));
    if (a->n_tokens == 0) return DF11_OK;
    if (bad_index(a->slots, 8)) return report_error(DF11_E_ARG, "kv_append: slots NULL or misaligned");
    TRY(check_rotation(a->rotation, d));
    HeadsArgs h{};
    TRY(heads_args(&h, a->rotation, a->q_weight, a->k_weight, a->eps, a->n_tokens, a->n_heads + 2 * heads, d, hip_device));
    h.c = view_of(a->cache);
    h.q = rows_of(a->q);
    h.k = rows_of(a->k);
    h.v = rows_of(a->v);
    h.q_out = rows_of(a->q_out);
    h.k_out = rows_of(a->k_out);
    h.slots = a->slots;
    h.heads = a->n_heads;
    h.kv_heads = heads;
    ON_DEVICE(hip_device);
    return launched(launch_heads(h, d, a->cache.store == DF11_KV_INT8 ? kHeadsInt8 : kHeadsBf16, a->rotation.flags & DF11_ROTATE_NEIGHBOURS, stream), "kv_append");
}

extern "C" df11_status df11_kv_read(const df11_kv_read_args *a, int hip_device, hipStream_t stream) {
    if (!a) return report_error(DF11_E_ARG, "kv_read: NULL arguments");
    TRY(check_cache(a->cache));
    const uint32_t d = a->cache.head_dim, heads = a->cache.n_kv_heads;
    const uint64_t tiles = a->n_tokens / kReadTile + a->n_seqs, slices = ceil_div((uint64_t)heads * kReadTile * d / 8, kReadSlice);
    if (a->n_tokens > 0x7FFFFFFFu || tiles > 4 * kMostGroups / slices)     // (four waves a workgroup; at most 65535 heads)
        return report_error(DF11_E_UNSUPPORTED, "kv_read: %llu tokens of %u sequences", (unsigned long long)a->n_tokens, a->n_seqs);
    TRY(check_rows("k", a->k, a->n_tokens, heads, d, true));
    TRY(check_rows("v", a->v, a->n_tokens, heads, d, true));
    if (a->n_tokens == 0 || a->n_seqs == 0) return DF11_OK;
    TRY(check_table(a->table, a->cache));
    if (bad_index(a->starts, 4)) return report_error(DF11_E_ARG, "kv_read: starts NULL or misaligned");
    ON_DEVICE(hip_device);
    const ReadArgs r{view_of(a->cache), tables_of(a->table), rows_of(a->k), rows_of(a->v), a->starts, a->n_seqs, (uint32_t)a->n_tokens, (uint32_t)tiles, (uint32_t)slices};
    return launched(launch_kv_read(r, d, a->cache.store == DF11_KV_INT8, stream), "kv_read");
}

static uint64_t token_workspace(const df11_attend_token_args *a, uint32_t window, uint32_t sinks, int hip_device) {
    if (!a || a->n_seqs == 0 || check_token_sizes(*a) || a->table.width == 0) return 0;
    return token_bytes(*a, token_split(*a, window_of(window, sinks, (uint64_t)a->table.width * a->cache.page_size), hip_device));
}

extern "C" uint64_t df11_attend_token_workspace(const df11_attend_token_args *a, int hip_device) { return token_workspace(a, 0, 0, hip_device); }

extern "C" uint64_t df11_attend_token_window_workspace(const df11_attend_token_window_args *a, int hip_device) {
    return a ? token_workspace(&a->token, a->window, a->sinks, hip_device) : 0;
}

static df11_status attend_token(const df11_attend_token_args *a, uint32_t window, uint32_t sinks, int hip_device, hipStream_t stream) {
    TRY(check_token_sizes(*a));
    TRY(check_cache(a->cache));
    TRY(check_scale(a->scale));
    const uint32_t d = a->cache.head_dim;
    TRY(check_rows("q", a->q, a->n_seqs, a->n_heads, d, false));
    TRY(check_rows("out", a->out, a->n_seqs, a->n_heads, d, true));
    if (a->n_seqs == 0) return DF11_OK;
    TRY(check_table(a->table, a->cache));
    if (bad_index(a->lens, 4)) return report_error(DF11_E_ARG, "attend_token: lens NULL or misaligned");
    const Window w = window_of(window, sinks, (uint64_t)a->table.width * a->cache.page_size);
    const TokenSplit s = token_split(*a, w, hip_device);
    TRY(check_workspace(a->workspace, a->workspace_bytes, token_bytes(*a, s)));
    ON_DEVICE(hip_device);
    TokenArgs t{};
    t.c = view_of(a->cache);
    t.t = tables_of(a->table);
    t.q = rows_of(a->q);
    t.out = rows_of(a->out);
    t.lens = a->lens;
    t.log2_scale = log2_scale(a->scale);
    t.n_seqs = a->n_seqs;
    t.heads = a->n_heads;
    t.group = a->n_heads / a->cache.n_kv_heads;
    t.q_tiles = s.q_tiles;
    t.range = s.range;
    t.splits = s.splits;
    t.whole = s.whole;
    t.window = w.keys;
    t.sinks = w.sinks;
    t.part = (float *)a->workspace;
    t.part_ml = t.part + (uint64_t)a->n_seqs * a->n_heads * s.splits * d;
    return launched(launch_attend_token(t, d, a->cache.store == DF11_KV_INT8, stream), "attend_token");
}

extern "C" df11_status df11_attend_token(const df11_attend_token_args *a, int hip_device, hipStream_t stream) {
    return a ? attend_token(a, 0, 0, hip_device, stream) : report_error(DF11_E_ARG, "attend_token: NULL arguments");
}

extern "C" df11_status df11_attend_token_window(const df11_attend_token_window_args *a, int hip_device, hipStream_t stream) {
    return a ? attend_token(&a->token, a->window, a->sinks, hip_device, stream) : report_error(DF11_E_ARG, "attend_token_window: NULL arguments");
}

extern "C" uint64_t df11_attend_chunk_workspace(const df11_attend_chunk_args *a, int hip_device) {
    if (!a || check_chunk_sizes(*a) || a->table.width == 0) return 0;
    return chunk_bytes(*a, chunk_split(*a, hip_device));
}

extern "C" df11_status df11_attend_chunk(const df11_attend_chunk_args *a, int hip_device, hipStream_t stream) {
    if (!a) return report_error(DF11_E_ARG, "attend_chunk: NULL arguments");
    TRY(check_chunk_sizes(*a));
    TRY(check_cache(a->cache));
    TRY(check_scale(a->scale));
    const uint32_t d = a->cache.head_dim, kv = a->cache.n_kv_heads;
    TRY(check_rows("q", a->q, a->n_q, a->n_heads, d, false));
    TRY(check_rows("out", a->out, a->n_q, a->n_heads, d, true));
    if (a->n_q == 0 || a->n_seqs == 0) return DF11_OK;
    TRY(check_table(a->table, a->cache));
    if (bad_index(a->q_starts, 4) || bad_index(a->lens, 4)) return report_error(DF11_E_ARG, "attend_chunk: q_starts or lens NULL or misaligned");
    const ChunkSplit s = chunk_split(*a, hip_device);
    TRY(check_workspace(a->workspace, a->workspace_bytes, chunk_bytes(*a, s)));
    ON_DEVICE(hip_device);
    ChunkArgs c{};
    c.c = view_of(a->cache);
    c.t = tables_of(a->table);
    c.q = rows_of(a->q);
    c.out = rows_of(a->out);
    c.q_starts = a->q_starts;
    c.lens = a->lens;
    c.log2_scale = log2_scale(a->scale);
    c.n_seqs = a->n_seqs;
    c.n_q = (uint32_t)a->n_q;
    c.group = a->n_heads / kv;
    c.causal = a->flags & DF11_ATTEND_CAUSAL;
    const Window w = window_of(a->window, a->sinks, (uint64_t)a->table.width * a->cache.page_size);
    c.window = w.keys;
    c.sinks = w.sinks;
    divide_by(c.group, &c.group_magic, &c.group_shift);
    c.most_steps = s.most_steps;
    c.tile_rows = s.tile_rows;
    c.tile_slots = (uint32_t)chunk_tile_slots(*a);
    c.at_a_time = s.parts;
    c.places = s.places;
    c.least_shift = s.least_shift;
    c.by_parts = s.parts ? 1.0f / s.parts : 0;
    c.part = (float *)a->workspace;
    c.part_ml = c.part + (uint64_t)s.places * kv * s.tile_rows * d;
    c.quota = (uint32_t *)(c.part_ml + (uint64_t)s.places * kv * s.tile_rows * 2);
    return launched(launch_attend_chunk(c, d, a->cache.store == DF11_KV_INT8, stream), "attend_chunk");
}

extern "C" uint64_t df11_attend_prompt_workspace(const df11_attend_prompt_args *a, int hip_device) {
    if (!a || check_prompt_sizes(*a)) return 0;
    return prompt_bytes(*a, prompt_split(*a, hip_device).splits);
}

extern "C" df11_status df11_attend_prompt(const df11_attend_prompt_args *a, int hip_device, hipStream_t stream) {
    if (!a) return report_error(DF11_E_ARG, "attend_prompt: NULL arguments");
    TRY(check_prompt_sizes(*a));
    TRY(check_scale(a->scale));
    if (a->flags & ~DF11_ATTEND_CAUSAL) return report_error(DF11_E_ARG, "attend_prompt: flags %u", a->flags);
    TRY(check_rows("q", a->q, a->n_q, a->n_heads, a->head_dim, false));
    TRY(check_rows("k", a->k, a->n_k, a->n_kv_heads, a->head_dim, false));
    TRY(check_rows("v", a->v, a->n_k, a->n_kv_heads, a->head_dim, false));
    TRY(check_rows("out", a->out, a->n_q, a->n_heads, a->head_dim, true));
    if (a->k.row_stride > kMostKeyStride || a->v.row_stride > kMostKeyStride)
        return report_error(DF11_E_UNSUPPORTED, "k, v: rows more than %lld elements apart", (long long)kMostKeyStride);
    if (a->n_q == 0 || a->n_seqs == 0) return DF11_OK;
    if (bad_index(a->q_starts, 4) || bad_index(a->k_starts, 4)) return report_error(DF11_E_ARG, "attend_prompt: starts NULL or misaligned");
    const PromptSplit split = prompt_split(*a, hip_device);
    const uint32_t splits = split.splits;
    TRY(check_workspace(a->workspace, a->workspace_bytes, prompt_bytes(*a, splits)));
    ON_DEVICE(hip_device);
    PromptArgs p{};
    p.q = rows_of(a->q);
    p.k = rows_of(a->k);
    p.v = rows_of(a->v);
    p.out = rows_of(a->out);
    p.q_starts = a->q_starts;
    p.k_starts = a->k_starts;
    p.log2_scale = log2_scale(a->scale);
    p.n_seqs = a->n_seqs;
    p.n_q = (uint32_t)a->n_q;
    p.n_k = (uint32_t)a->n_k;
    p.heads = a->n_heads;
    p.kv_heads = a->n_kv_heads;
    p.group = a->n_heads / a->n_kv_heads;
    divide_by(p.group, &p.group_magic, &p.group_shift);
    p.causal = a->flags & DF11_ATTEND_CAUSAL;
    p.tile_slots = (uint32_t)prompt_tile_slots(*a);
    p.splits = splits;
    p.split_magic = splits > 1 ? (uint32_t)((((uint64_t)1 << 32) + splits - 1) / splits) : 0;
    p.part_keys = split.part_keys;
    p.part = (float *)a->workspace;
    p.part_ml = p.part + splits * prompt_tile_slots(*a) * a->n_kv_heads * kPromptTile * a->head_dim;
    return launched(launch_attend_prompt(p, a->head_dim, stream), "attend_prompt");
}
