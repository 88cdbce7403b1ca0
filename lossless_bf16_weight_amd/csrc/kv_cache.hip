// The paged key-value cache for gfx950: tokens' keys and values written into
// the cache's pages, as BF16 words or quantised to 8 bits on the way, and
// sequences read back as packed BF16 rows.
//
// 8 bits: for each token and head, a = max |x| (at least 2^-100), scale =
// a / 127, codes rint(x * (127 / a)): |x| <= a gives |code| <= 127 without a
// clamp (a * fl(127 / a) is within 2^-23 of 127), and two correctly rounded
// divisions a row.  The maximum is taken over the words' magnitude bits as
// integers, where NaN is above infinity: a row that holds either gets a scale
// of NaN or infinity and codes 0, and reads back as NaN.
//
// Both kernels are bound by HBM traffic: a lane moves 16 bytes of BF16 a step
// (a row of 128 is 16 lanes), several steps in flight.  Measured with 8 kv
// heads of 128: 20,288 tokens written as words 28 us (166 MB read and written,
// 5.9 TB/s; a copy of 2 GiB reaches 4.9), 5,520 tokens written in 8 bits 9.8 us
// and read back 8.5 us (34 MB; an empty kernel takes 2.5 us of it), 118,617
// tokens read back from 8 bits 131 us (736 MB, 5.6 TB/s), from words 170 us
// (972 MB, 5.7 TB/s).  64 tokens are written in 2.6 us.
#include "serve_device.hpp"
#include "serve_internal.hpp"

namespace df11 {

namespace {

constexpr int kThreads = 256;
constexpr int kWriteUnroll = 2, kReadUnroll = 4;
constexpr uint32_t kReadShift = 4;
static_assert(kWriteChunks == kThreads * kWriteUnroll);
static_assert(kReadTile == 1u << kReadShift && kReadSlice == 64 * kReadUnroll);

// Maximum over the kLanes neighbouring lanes that hold a row, in each of them.
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));    // lanes xor 1
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));    // lanes xor 2
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, true));   // mirrored in 8
    if (kLanes == 16) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xF, 0xF, true));   // in 16
    return x;
}

__device__ __forceinline__ float low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// Two codes from two words, as the low bytes of a dword.
__device__ __forceinline__ uint32_t codes2(uint32_t w, float inv) {
    const int a = (int)__builtin_rintf(low(w) * inv), b = (int)__builtin_rintf(high(w) * inv);
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8;
}

template <int D, bool kInt8>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(WriteArgs a) {
    constexpr uint32_t kLanes = D / 8;
    const bool is_v = blockIdx.y != 0;
    const Rows &x = is_v ? a.v : a.k;
    uint8_t *const store = is_v ? a.c.v : a.c.k;
    float *const scales = is_v ? a.c.v_scale : a.c.k_scale;
    const uint64_t n_units = (uint64_t)a.n_tokens * a.c.kv_heads * kLanes;
    const uint64_t first = (uint64_t)blockIdx.x * kWriteChunks + threadIdx.x;
    u32x4 w[kWriteUnroll];
    int64_t slot[kWriteUnroll];
    uint32_t head[kWriteUnroll];
#pragma unroll
    for (int i = 0; i < kWriteUnroll; ++i) {
        const uint64_t unit = first + (uint64_t)i * kThreads;
        slot[i] = -1;
        if (unit < n_units) {
            const uint32_t r = (uint32_t)(unit / kLanes);
            const uint32_t token = r / a.c.kv_heads;
            head[i] = r - token * a.c.kv_heads;
            slot[i] = a.slots[token];
            w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x.data + token * x.row + head[i] * x.head + (unit % kLanes) * 8));
        }
    }
#pragma unroll
    for (int i = 0; i < kWriteUnroll; ++i) {
        const uint32_t part = threadIdx.x % kLanes;
        uint32_t m = 0;
        if (kInt8) {
            if (slot[i] >= 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) m = max(m, max(w[i][j] << 16 & 0x7FFF0000u, w[i][j] & 0x7FFF0000u));
            }
            m = row_max<kLanes>(m);
        }
        if (slot[i] < 0 || slot[i] >= a.c.n_slots) continue;   // (a row's lanes go together)
        const int64_t page = slot[i] >> a.c.shift, pos = slot[i] & ((1 << a.c.shift) - 1);
        const int64_t row = ((page * a.c.kv_heads + head[i]) << a.c.shift) + pos;
        if (kInt8) {
            const float top = __builtin_bit_cast(float, m > 0x0D800000u ? m : 0x0D800000u);   // 2^-100
            const float inv = 127.0f / top;
            u32x2 c;
            c.x = codes2(w[i].x, inv) | codes2(w[i].y, inv) << 16;
            c.y = codes2(w[i].z, inv) | codes2(w[i].w, inv) << 16;
            *reinterpret_cast<u32x2 *>(store + row * D + 8 * part) = c;
            if (part == 0) scales[row] = top / 127.0f;
        } else {
            *reinterpret_cast<u32x4 *>(store + 2 * (row * D + 8 * part)) = w[i];
        }
    }
}

// A tile is 16 tokens of all heads: whole rows to write, and 16 neighbouring
// rows of each head's part of a page to read (a workgroup for one head, which
// writes a part of each row, takes 1.4 times as long).  A wave takes kReadSlice
// 16-byte chunks of it, four a lane, in the order of the rows that are written:
// few tokens of many heads are many waves' work (35 sequences, 2000 tokens of 24
// heads in all: 8 us, with a workgroup for a tile 15 us), and of one head the
// lanes have enough to do (56,000 tokens: 11 us, 16 us).  Stores past the
// caches are 5% sooner for 228,000 tokens, but the attention that reads these
// rows next is later by more (four times 16,000 tokens, with it 184 and 197 us).
template <int D, bool kInt8>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(ReadArgs a) {
    constexpr uint32_t kLanes = D / 8;
    const uint32_t lane = threadIdx.x & 63u, item = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t slot = item / a.slices, first = item % a.slices * kReadSlice;
    if (slot >= a.tile_slots) return;
    uint32_t tile;
    const uint32_t s = sequence_of_slot(a.starts, a.n_seqs, slot, 1, kReadShift, &tile);
    const int32_t begin = a.starts[s], end = a.starts[s + 1];
    if (begin < 0 || end < begin || (uint32_t)end > a.n_tokens) return;
    const uint32_t n = min((uint32_t)(end - begin), a.t.width << a.c.shift);
    if (tile > n >> kReadShift) return;
    const uint32_t pos0 = tile << kReadShift, units = min(n - pos0, 1u << kReadShift) * a.c.kv_heads * kLanes;
    if (first >= units) return;
    const bool is_v = blockIdx.y != 0;
    const Rows &x = is_v ? a.v : a.k;
    const uint8_t *const store = is_v ? a.c.v : a.c.k;
    const float *const scales = is_v ? a.c.v_scale : a.c.k_scale;
    const uint32_t part = lane % kLanes;
    // (16 positions from a multiple of 16 lie in one page)
    const uint32_t page = min((uint32_t)a.t.pages[s * a.t.stride + (pos0 >> a.c.shift)], a.c.n_pages - 1);
    const uint32_t in_page = pos0 & ((1u << a.c.shift) - 1);
    u32x4 w[kReadUnroll];
    u32x2 c[kReadUnroll];
    float scale[kReadUnroll];
    uint32_t pos[kReadUnroll], head[kReadUnroll];
#pragma unroll
    for (int i = 0; i < kReadUnroll; ++i) {
        const uint32_t r = min(first + i * 64 + lane, units - 1) / kLanes;
        pos[i] = r / a.c.kv_heads;
        head[i] = r - pos[i] * a.c.kv_heads;
        const uint64_t row = (((uint64_t)page * a.c.kv_heads + head[i]) << a.c.shift) + in_page + pos[i];
        if (kInt8) {
            c[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(store + row * D + 8 * part));
            scale[i] = scales[row];
        } else {
            w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(store + 2 * (row * D + 8 * part)));
        }
    }
#pragma unroll
    for (int i = 0; i < kReadUnroll; ++i) {
        if (first + i * 64 + lane >= units) continue;
        if (kInt8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = c[i][j / 2] >> (16 * (j % 2));
                w[i][j] = pack_bf16((float)(int8_t)two * scale[i], (float)(int8_t)(two >> 8) * scale[i]);
            }
        }
        *reinterpret_cast<u32x4 *>(x.data + (int64_t)(begin + pos0 + pos[i]) * x.row + head[i] * x.head + 8 * part) = w[i];
    }
}

}  // namespace

hipError_t launch_kv_write(const WriteArgs &a, uint32_t head_dim, bool int8, hipStream_t stream) {
    const uint64_t units = (uint64_t)a.n_tokens * a.c.kv_heads * (head_dim / 8);
    const dim3 grid((uint32_t)((units + kWriteChunks - 1) / kWriteChunks), 2);
    const auto kernel = head_dim == 64 ? (int8 ? kv_write_kernel<64, true> : kv_write_kernel<64, false>)
                                       : (int8 ? kv_write_kernel<128, true> : kv_write_kernel<128, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_kv_read(const ReadArgs &a, uint32_t head_dim, bool int8, hipStream_t stream) {
    const dim3 grid((a.tile_slots * a.slices + kThreads / 64 - 1) / (kThreads / 64), 2);
    const auto kernel = head_dim == 64 ? (int8 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>)
                                       : (int8 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace df11
