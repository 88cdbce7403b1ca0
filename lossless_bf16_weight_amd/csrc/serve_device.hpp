// Device code that the serving kernels share: vector types, the matrix
// instructions' operand types, BF16 packing, and the search of a tile's
// sequence.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

namespace df11 {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define DF11_LDS __attribute__((address_space(3)))

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// Two floats rounded to BF16 (nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Two weights as sums of two BF16 operands each (.x, .y), within 2^-14 of the
// weight as a BF16.
// Words: weights are from 0 on, and the first operand is the BF16 number before
// the one that the weight begins with: what is left for the second is then above
// zero, and a value that is infinite times both is that infinity (times 0 or less
// it would make the result NaN).
// 8 bits: weights have the values' scales in them, of either sign or infinite, and
// values are finite codes: the first operand is what the weight begins with, at
// most the largest finite number, so that the second is what is left (by one
// minimum for each sign; the step before it, of signed words, took 1 to 7% longer:
// 16 prompts of up to 1024 tokens 113.5 us, heads of 64 75.0, and 109.3, 70.3).
template <bool kInt8>
__device__ __forceinline__ u32x2 two_operands(float a, float b) {
    const uint32_t cut = __float_as_uint(a) >> 16 | (__float_as_uint(b) & 0xFFFF0000u);
    uint32_t w;
    if constexpr (kInt8) {
        w = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(i16x2, cut), i16x2{0x7F7F, 0x7F7F}));
        w = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, w), u16x2{0xFF7F, 0xFF7F}));
    } else {
        w = __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, cut), u16x2{1, 1}));
    }
    return u32x2{w, pack_bf16(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xFFFF0000u))};
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// x and the value 32 (16) lanes away, in either order.
__device__ __forceinline__ f32x2 with_lane_32(float x) {
    const uint32_t a = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    return f32x2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ f32x2 with_lane_16(float x) {
    const uint32_t a = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    return f32x2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

struct Add {
    template <class T>
    __device__ __forceinline__ T operator()(T x, T y) const { return x + y; }
};
struct Least {
    template <class T>
    __device__ __forceinline__ T operator()(T x, T y) const { return x < y ? x : y; }
};

// op over the lanes of a wave up to this one; the last lane has all of them.
template <class T, class Op>
__device__ __forceinline__ T over_lanes(T x, T identity, Op op) {
    const auto more = [&](auto ctrl, auto rows) {
        x = op(x, __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, identity), __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                    decltype(rows)::value, 0xF, false)));
    };
    constexpr std::integral_constant<int, 0xF> all{};
    more(std::integral_constant<int, 0x111>{}, all);      // from 1, 2, 4 and 8 lanes below, in 16
    more(std::integral_constant<int, 0x112>{}, all);
    more(std::integral_constant<int, 0x114>{}, all);
    more(std::integral_constant<int, 0x118>{}, all);
    more(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});   // the 16 below, the 32 below
    more(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
    return x;
}

// Softmax sums are kept against a base, m below, that is raised only when a
// row's maximum passes what it was by more than kSlack: most steps then need
// not scale the sums.  The base lies kSlack + log2(n) above that maximum for
// n keys, so that a weight is at most 1 / n and a sum of weights at most 1:
// sums of weighted values stay within the values, and no finite value
// overflows them.  (A power of two costs the weights no bits; those below
// 2^-126 n 2^8 of the largest are lost, which no sum in 32 bits sees.)
constexpr float kSlack = 8.0f;

// log2(n) rounded up (0 for none), in a scalar register.
__device__ __forceinline__ float log2_up(uint32_t n) {
    const float x = (float)(n > 1 ? 32 - __builtin_clz(n - 1) : 0);
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// The four signed bytes of w as BF16 words (exact: |code| <= 128 has eight
// significant bits, so the float's upper half is the whole value).
__device__ __forceinline__ u32x2 bf16_of_bytes(uint32_t w) {
    const uint32_t a = __builtin_bit_cast(uint32_t, (float)(int8_t)w);
    const uint32_t b = __builtin_bit_cast(uint32_t, (float)(int8_t)(w >> 8));
    const uint32_t c = __builtin_bit_cast(uint32_t, (float)(int8_t)(w >> 16));
    const uint32_t d = __builtin_bit_cast(uint32_t, (float)(int8_t)(w >> 24));
    return u32x2{__builtin_amdgcn_perm(b, a, 0x07060302u), __builtin_amdgcn_perm(d, c, 0x07060302u)};
}

__device__ __forceinline__ u32x4 bf16_of_bytes8(u32x2 w) {
    const u32x2 lo = bf16_of_bytes(w.x), hi = bf16_of_bytes(w.y);
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// Tiles over packed sequences of starts[s + 1] - starts[s] times `each` rows.
// With tiles of 2^shift rows, sequence s is given the tile slots from
// (starts[s] * each >> shift) + s up to the next sequence's: at least as many
// as its tiles, and no prefix sum is needed.
// Finds the sequence of slot t with a 64-way search (one load for up to 64
// sequences); the same in every lane of the wave.  Returns the slot's tile
// number within the sequence through *tile.
__device__ __forceinline__ uint32_t sequence_of_slot(const int32_t *starts, uint32_t n_seqs, uint32_t t,
                                                     uint32_t each, uint32_t shift, uint32_t *tile) {
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t lo = 0, n = n_seqs;
    while (n > 1) {
        const uint32_t step = (n + 63u) >> 6;
        const uint32_t at = lane * step;
        bool below = false;
        if (at < n) below = ((uint32_t)starts[lo + at] * each >> shift) + lo + at <= t;
        const uint32_t c = (uint32_t)__builtin_popcountll(__ballot(below));
        const uint32_t skip = (c ? c - 1 : 0) * step;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    *tile = t - (((uint32_t)starts[lo] * each >> shift) + lo);
    return lo;
}

}  // namespace df11
