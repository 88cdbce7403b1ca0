// What the host code of the serving operators (serve.cpp) and their kernels
// (attend_prompt.hip, attend_token.hip, kv_cache.hip) share.
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

struct TokenArgs {
    CacheView c;
    Tables t;
    Rows q, out;
    const int32_t *lens;
    float log2_scale;          // scale * log2(e): weights are 2^(log2_scale * <q, k> - max)
    uint32_t n_seqs, heads, group, q_tiles;   // group = heads / kv_heads, in q_tiles tiles of 16
    uint32_t range, splits;    // keys a workgroup takes, workgroups along a sequence
    uint32_t whole;            // twelve waves a workgroup instead of four
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
hipError_t launch_attend_token(const TokenArgs &a, uint32_t head_dim, bool int8, hipStream_t stream);
hipError_t launch_attend_prompt(const PromptArgs &a, uint32_t head_dim, hipStream_t stream);

}  // namespace df11
