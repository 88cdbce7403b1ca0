// What the host code of the serving operators (serve.cpp) and their kernels
// (attend_chunk.hip, attend_prompt.hip, attend_token.hip, heads.hip,
// kv_cache.hip) share.
#pragma once
#include "df11_internal.hpp"

namespace df11 {

// Rows of heads: element (row, head, d) at data[row * row + head * head + d],
// strides in elements, head_dim contiguous.
struct Rows {
    uint16_t *data;
    int64_t row, head;
};

// A paged cache: pages of [kv_head][position][head_dim], scales (8-bit store)
// of [kv_head][position]; page_size = 1 << shift.
struct CacheView {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t n_slots;           // n_pages << shift
    uint32_t n_pages, shift, kv_heads;
};

// Page tables: row s lists the pages of sequence s in order.
struct Tables {
    const int32_t *pages;
    int64_t stride;
    uint32_t width;            // entries a row
};

struct WriteArgs {
    CacheView c;
    Rows k, v;
    const int64_t *slots;
    uint32_t n_tokens;
};

struct ReadArgs {
    CacheView c;
    Tables t;
    Rows k, v;
    const int32_t *starts;
    uint32_t n_seqs, n_tokens;
    uint32_t tile_slots, slices;         // tiles of kReadTile tokens, waves for each
};

// Where heads go: rows only, or keys and values also into a cache.
enum { kHeadsOnly = 0, kHeadsBf16 = 1, kHeadsInt8 = 2 };

struct HeadsArgs {
    CacheView c;
    Rows q, k, v, q_out, k_out;          // k_out.data may be null beside a cache
    const int64_t *slots;
    const uint64_t *turns;               // [pairs]: turns a position, times 2^64
    const uint8_t *axes;                 // [pairs], or null: the first
    const int32_t *positions;
    int64_t position_stride;
    const uint16_t *q_weight, *k_weight; // BF16 [head_dim], or null: no norm
    uint32_t n_tokens, heads, kv_heads;
    uint32_t pairs, n_axes;
    uint32_t parts, run;                 // waves a token, steps of each
    float factor, eps, eps_scaled;       // (the last: times 2^-136)
};

struct TokenArgs {
    CacheView c;
    Tables t;
    Rows q, out;
    const int32_t *lens;
    float log2_scale;          // scale * log2(e): weights are 2^(log2_scale * <q, k> - max)
    uint32_t n_seqs, heads, group, q_tiles;   // group = heads / kv_heads, in q_tiles tiles of 16
    uint32_t range, splits;    // keys a workgroup takes, workgroups along a sequence
    uint32_t whole;            // twelve waves a workgroup instead of four
    uint32_t window, sinks;    // window 0: none
    float *part;               // [seq][head][split][head_dim] unnormalised, then [..][2] maximum and sum
    float *part_ml;
};

struct PromptArgs {
    Rows q, k, v, out;
    const int32_t *q_starts, *k_starts;
    float log2_scale;
    uint32_t n_seqs, n_q, n_k, heads, kv_heads, group, causal;
    uint32_t group_magic, group_shift;   // x / group = (x * group_magic >> 32) >> group_shift for group > 1, x < 2^31
    uint32_t tile_slots, splits;
    uint32_t split_magic, part_keys;     // ceil(2^32 / splits), the least keys of a part
    float *part, *part_ml;     // [split][workgroup][wave][register / 4][lane][4], then [split][workgroup][wave][row][2]
};

struct ChunkArgs {
    CacheView c;
    Tables t;
    Rows q, out;
    const int32_t *q_starts, *lens;
    float log2_scale;
    uint32_t n_seqs, n_q, group, causal;
    uint32_t window, sinks;              // window 0: none
    uint32_t group_magic, group_shift;   // as in PromptArgs
    uint32_t most_steps;                 // of a tile with the window, whatever the length
    uint32_t tile_rows;                  // 128 or 256
    uint32_t tile_slots;                 // at least as many as tiles
    uint32_t at_a_time;                  // workgroups of a kv head that run at a time
    uint32_t places, least_shift;        // parts of a kv head's tiles that the workspace holds (0: none are split); log2 of the least steps of one
    float by_parts;                      // 1 / the parts that a kv head's work is divided into
    float *part, *part_ml;               // [place][kv_head][wave][register / 4][lane][4], then [place][kv_head][wave][row][2]
    uint32_t *quota;                     // the first kernel's, for the one that joins
};

constexpr uint32_t kWriteChunks = 512;   // 16-byte chunks of rows that a workgroup of kv_write takes
constexpr uint32_t kReadTile = 16;       // tokens of a tile that kv_read reads back
constexpr uint32_t kReadSlice = 256;     // 16-byte chunks of its rows that a wave takes
constexpr uint32_t kPromptTile = 128;    // rows (queries of the heads of a kv head) a workgroup takes
constexpr uint32_t kPromptKeys = 64;     // keys a step
constexpr uint32_t kTokenKeys = 32;      // keys a wave's step
constexpr uint32_t kTokenWholeMax = 1024; // and of one that twelve waves take whole
constexpr uint32_t kTokenRangeMax = 1280;  // keys a workgroup takes of a long sequence

hipError_t launch_kv_write(const WriteArgs &a, uint32_t head_dim, bool int8, hipStream_t stream);
hipError_t launch_kv_read(const ReadArgs &a, uint32_t head_dim, bool int8, hipStream_t stream);
hipError_t launch_heads(const HeadsArgs &a, uint32_t head_dim, int store, bool neighbours, hipStream_t stream);
hipError_t launch_attend_token(const TokenArgs &a, uint32_t head_dim, bool int8, hipStream_t stream);
hipError_t launch_attend_prompt(const PromptArgs &a, uint32_t head_dim, hipStream_t stream);

hipError_t launch_attend_chunk(const ChunkArgs &a, uint32_t head_dim, bool int8, hipStream_t stream);

}  // namespace df11
