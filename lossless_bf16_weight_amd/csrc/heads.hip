// Query, key and value heads of new tokens for gfx950: RMS norms of each
// query and key head, the position rotation, and the keys' and values' way
// into the paged cache (as BF16 words or in 8 bits), in one pass.
//
// norm: y = x * w / sqrt(mean(x^2) + eps).  Rotation: pair i (a, b) of a head
// becomes (a c - b s, b c + a s), c and s of position * frequency_i.  A
// frequency is kept as F, turns a position times 2^64: position * F modulo
// 2^64 is the phase without any rounding, two 32-bit multiplications give its
// upper half, and the sine takes that as a fraction of a turn from -1/2 to
// 1/2.  Far positions are then as exact as near ones.  8 bits: as in
// kv_cache.hip, but of the 32-bit values, so that an element is rounded once.
//
// HBM traffic bounds it.  A lane holds 16 elements of a row, its pairs
// complete: with pairs of the two halves chunks of 8 that are half the rotated
// part apart, with neighbours two chunks side by side, pairs 8 l .. 8 l + 7 of
// lane l either way.  A wave takes the rows of one token eight (heads of 64:
// sixteen) at a time.  Their sines it computes once, a pair a lane, and keeps
// them and the weights in LDS, as eight waves for each SIMD have no registers
// for them (with each lane's eight pairs and the weights in registers, five
// waves for each SIMD, 15,183 tokens with norms took 7% longer, with heads of 64
// 14%, 5,520 tokens in 8 bits with their read 9%).
// Results are stored through the caches, though alone they are 8% faster past
// them: the attention that reads them next is later by more.
//
// Measured with 32 heads over 8 kv heads of 128: 15,183 tokens with norms and
// three axes 61 us (311 MB, 5.1 TB/s; heads of 64 38 us, 4.1 TB/s), 20,288 tokens
// into the cache 97 us (499 MB, 5.1 TB/s; a copy of 2 GiB reaches 4.95).
#include "serve_device.hpp"
#include "serve_internal.hpp"

namespace df11 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));    // lanes xor 1
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));    // lanes xor 2
    if (kLanes == 8) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, true));   // mirrored in 8
    return x;
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
    const auto from = [&](auto ctrl) { return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true)); };
    x += from(std::integral_constant<int, 0xB1>{});
    x += from(std::integral_constant<int, 0x4E>{});
    if (kLanes == 8) x += from(std::integral_constant<int, 0x141>{});
    return x;
}

template <int D, int kStore, bool kNeighbours>
__global__ __launch_bounds__(kThreads, 8) void heads_kernel(HeadsArgs a) {
    constexpr uint32_t kLanes = D / 16, kRows = 64 / kLanes, kWaves = kThreads / 64;
    __shared__ __attribute__((aligned(16))) float cosines[kWaves][D / 2], sines[kWaves][D / 2];
    __shared__ __attribute__((aligned(16))) uint16_t weights[kWaves][2 * D];      // queries', keys'
    const uint32_t lane = threadIdx.x & 63u, l = lane % kLanes, in_step = lane / kLanes;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), item = blockIdx.x * kWaves + wave;
    const uint32_t token = item / a.parts, part = item % a.parts;
    if (token >= a.n_tokens) return;
    const uint32_t n_rows = a.heads + (kStore == kHeadsOnly ? 1 : 2) * a.kv_heads;
    const uint32_t first = part * a.run * kRows, end = min(first + a.run * kRows, n_rows);

    const bool turned = l < a.pairs / 8;
    const uint32_t at0 = !kNeighbours && turned ? 8 * l : 16 * l, at1 = !kNeighbours && turned ? 8 * l + a.pairs : 16 * l + 8;

    int64_t slot = -1;
    if (kStore != kHeadsOnly) {
        slot = a.slots[token];
        if (slot < 0 || slot >= a.c.n_slots) slot = -1;
    }
    // The wave's sines, a lane each, and the weights wait in its part of LDS.
    const auto prepare = [&] {
        if (lane < a.pairs) {
            const int32_t *const at = a.positions + token * a.position_stride;
            const uint32_t axis = a.axes ? a.axes[lane] : 0;
            int32_t pos = at[0];
#pragma unroll
            for (int x = 1; x < 4; ++x)
                if (x < (int)a.n_axes) pos = axis >= (uint32_t)x ? at[x] : pos;
            const u32x2 f = reinterpret_cast<const u32x2 *>(a.turns)[lane];
            const uint32_t phase = (uint32_t)pos * f.y + __umulhi((uint32_t)pos, f.x) - (pos < 0 ? f.x : 0);
            const float t = (float)(int32_t)phase * 0x1p-32f;
            cosines[wave][lane] = __builtin_amdgcn_cosf(t) * a.factor;
            sines[wave][lane] = __builtin_amdgcn_sinf(t) * a.factor;
        }
        if (a.q_weight && lane < D / 8) reinterpret_cast<u32x4 *>(weights[wave])[lane] = reinterpret_cast<const u32x4 *>(a.q_weight)[lane];
        if (a.k_weight && lane < D / 8) reinterpret_cast<u32x4 *>(weights[wave] + D)[lane] = reinterpret_cast<const u32x4 *>(a.k_weight)[lane];
        // LDS keeps a wave's accesses in order; this keeps the compiler's.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
    };

    // row r of the token: its rows of queries, then keys, then values
    const auto source = [&](uint32_t r) -> const uint16_t * {
        const bool is_q = r < a.heads, is_k = r < a.heads + a.kv_heads;
        const uint16_t *const data = is_q ? a.q.data : is_k ? a.k.data : a.v.data;
        const int64_t row = is_q ? a.q.row : is_k ? a.k.row : a.v.row, head = is_q ? a.q.head : is_k ? a.k.head : a.v.head;
        return data + token * row + (r - (is_q ? 0 : is_k ? a.heads : a.heads + a.kv_heads)) * head;
    };

    bool begun = false;
    for (uint32_t r0 = first; r0 < end; r0 += kRows) {
        const uint32_t r = r0 + in_step;
        u32x4 w[2];
        if (r < end) {
            const uint16_t *const from = source(r);
            w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(from + at0));
            w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(from + at1));
        }
        if (!begun) prepare();
        begun = true;
        if (r >= end) continue;        // (a row's lanes go together)
        const bool is_q = r < a.heads, is_v = r >= a.heads + a.kv_heads, is_k = !is_q && !is_v;
        const uint32_t head = r - (is_q ? 0 : is_k ? a.heads : a.heads + a.kv_heads);
        float y[16];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            y[2 * x] = low(w[x / 4][x % 4]);
            y[2 * x + 1] = high(w[x / 4][x % 4]);
        }
        if (is_q ? a.q_weight != nullptr : is_k && a.k_weight) {
            float sum = 0;
#pragma unroll
            for (int x = 0; x < 16; ++x) sum = __builtin_fmaf(y[x], y[x], sum);
            sum = row_sum<kLanes>(sum);
            float mean = __builtin_fmaf(sum, 1.0f / D, a.eps);
            if (!(mean < __builtin_inff())) {
                // squares that pass 32 bits, alone or with eps (or an infinity): of
                // values 2^-68 as large, whose sum stays below 2^127
                sum = 0;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    y[x] *= 0x1p-68f;
                    sum = __builtin_fmaf(y[x], y[x], sum);
                }
                sum = row_sum<kLanes>(sum);
                mean = __builtin_fmaf(sum, 1.0f / D, a.eps_scaled);
            }
            const float by = __builtin_amdgcn_rsqf(mean);
            // (first of value and root, which is at most the root of D: a weight times
            // the root may pass 32 bits where the result does not)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const u32x4 eight = *reinterpret_cast<const u32x4 *>(weights[wave] + (is_q ? 0 : D) + (x ? at1 : at0));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[8 * x + 2 * i] = y[8 * x + 2 * i] * by * low(eight[i]);
                    y[8 * x + 2 * i + 1] = y[8 * x + 2 * i + 1] * by * high(eight[i]);
                }
            }
        }
        if (turned && !is_v) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const f32x4 c = *reinterpret_cast<const f32x4 *>(cosines[wave] + 8 * l + 4 * g), s = *reinterpret_cast<const f32x4 *>(sines[wave] + 8 * l + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = 4 * g + i;
                    float &p = kNeighbours ? y[2 * x] : y[x], &q = kNeighbours ? y[2 * x + 1] : y[x + 8];
                    const float p0 = p, q0 = q;
                    p = __builtin_fmaf(p0, c[i], -(q0 * s[i]));
                    q = __builtin_fmaf(q0, c[i], p0 * s[i]);
                }
            }
        }
        u32x4 out[2];
#pragma unroll
        for (int x = 0; x < 8; ++x) out[x / 4][x % 4] = is_v ? w[x / 4][x % 4] : pack_bf16(y[2 * x], y[2 * x + 1]);
        const Rows &to = is_q ? a.q_out : a.k_out;
        if (is_q || (is_k && a.k_out.data)) {
            uint16_t *const row = to.data + token * to.row + head * to.head;
            *reinterpret_cast<u32x4 *>(row + at0) = out[0];
            *reinterpret_cast<u32x4 *>(row + at1) = out[1];
        }
        if (kStore == kHeadsOnly || is_q || slot < 0) continue;
        const uint64_t row = ((((uint64_t)slot >> a.c.shift) * a.c.kv_heads + head) << a.c.shift) + (slot & ((1 << a.c.shift) - 1));
        uint8_t *const store = is_v ? a.c.v : a.c.k;
        if (kStore == kHeadsInt8) {
            uint32_t m = 0x0D800000u;      // 2^-100
#pragma unroll
            for (int x = 0; x < 16; ++x) m = max(m, __float_as_uint(y[x]) & 0x7FFFFFFFu);
            const float top = __uint_as_float(row_max<kLanes>(m)), inv = 127.0f / top;
            uint32_t codes[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                codes[x] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) codes[x] |= (uint32_t)((int)__builtin_rintf(y[4 * x + j] * inv) & 255) << (8 * j);
            }
            *reinterpret_cast<u32x2 *>(store + row * D + at0) = u32x2{codes[0], codes[1]};
            *reinterpret_cast<u32x2 *>(store + row * D + at1) = u32x2{codes[2], codes[3]};
            if (l == 0) (is_v ? a.c.v_scale : a.c.k_scale)[row] = top / 127.0f;
        } else {
            *reinterpret_cast<u32x4 *>(store + 2 * (row * D + at0)) = out[0];
            *reinterpret_cast<u32x4 *>(store + 2 * (row * D + at1)) = out[1];
        }
    }
}

template <int D, int kStore>
auto kernel_of(bool neighbours) {
    return neighbours ? heads_kernel<D, kStore, true> : heads_kernel<D, kStore, false>;
}

template <int D>
auto kernel_of(int store, bool neighbours) {
    return store == kHeadsOnly ? kernel_of<D, kHeadsOnly>(neighbours)
                               : store == kHeadsInt8 ? kernel_of<D, kHeadsInt8>(neighbours) : kernel_of<D, kHeadsBf16>(neighbours);
}

}  // namespace

hipError_t launch_heads(const HeadsArgs &a, uint32_t head_dim, int store, bool neighbours, hipStream_t stream) {
    const uint64_t waves = (uint64_t)a.n_tokens * a.parts;
    const auto kernel = head_dim == 64 ? kernel_of<64>(store, neighbours) : kernel_of<128>(store, neighbours);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((waves + kThreads / 64 - 1) / (kThreads / 64))), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace df11
