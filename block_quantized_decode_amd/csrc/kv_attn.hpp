// What the attention kernels over the quantized key/value cache share: codes
// as matrix-core operands, query rows, sequences, outputs.
#pragma once

#include "kv_device.hpp"
#include "kv_plan.hpp"

namespace qbd {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr float kNoKey = -3e38f;  // reference of a row that has seen no key
// A product of a weight and a V scale enters the matrix cores in binary16.
// The reference puts the largest at 2^kLift, and it may grow to 2^kTop
// before the reference moves: near the top of the type's range, so that
// weights far below the largest keep their bits (11 down to 2^-28 of it).
constexpr float kLift = 12.f, kTop = 15.f;

// Scores this large (in log2) are rounded to units of a half and more: neither
// kLift and kTop nor the residue of a fused product fit between two of them.  A
// row whose largest is beyond takes it as its reference, as it is, and moves it
// whenever it grows, and its wave finds the weights' exponents from rounded
// products: the largest weight is 1 (so weights times V scales below 2^-14 lose
// bits there).
constexpr float kFar = 4194304.f;
__device__ __forceinline__ bool is_far(float score) { return fabsf(score) > kFar && score > kNoKey; }

// A query row enters scaled by a power of two to a maximum of 2^14 or more,
// below 2^15, so that its elements keep a binary16 number's 11 bits down to
// 2^-28 of the largest.
constexpr int kQueryTop = 15;

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {  // eight bf16 each
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// The upper halves of two words: two floats cut to bf16.
__device__ __forceinline__ uint32_t uppers(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Two floats as their leading 8 significant bits; a and b keep the rest.
__device__ __forceinline__ uint32_t cut8(float& a, float& b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    a -= __uint_as_float(x & 0xffff0000u);  // exact
    b -= __uint_as_float(y & 0xffff0000u);
    return uppers(x, y);
}

__device__ __forceinline__ h2 as_h2(uint32_t w) { return __builtin_bit_cast(h2, w); }
__device__ __forceinline__ h8 as_h8(h2 a, h2 b, h2 c, h2 d) { return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]}; }

// The binary16 pair (1024, 1024) in a vector register, of a value that the
// compiler does not know, so that the and-or below is one instruction (it takes
// a single scalar operand).  No asm statement here holds an instruction: the
// compiler counts the states that the matrix instructions have to wait for
// between its own instructions alone.
__device__ __forceinline__ uint32_t pair1024() {
    uint32_t v = 0x64006400u;
    asm("" : "+v"(v));
    return v;
}
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t high) { return (w & mask) | high; }

// Nibbles 0 and 4 (low) or 1 and 5 (high) of w as exact q - 8: 0x6400 | n
// is 1024 + n in binary16, and with the nibble four places up 1024 + 16 n.
// k is pair1024().
__device__ __forceinline__ h2 nib_lo(uint32_t w, uint32_t k) { return as_h2(and_or(w, 0x000f000fu, k)) - h2{1032.f16, 1032.f16}; }
__device__ __forceinline__ h2 nib_hi(uint32_t w, uint32_t k) {
    return __builtin_elementwise_fma(as_h2(and_or(w, 0x00f000f0u, k)), h2{0.0625f16, 0.0625f16}, h2{-72.f16, -72.f16});
}
// Bytes I and J of w, code + 128, as exact codes: 0x6400 | u is 1024 + u.
template <int I, int J>
__device__ __forceinline__ h2 bytes_of(uint32_t w) {
    return as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04000400u | I | J << 16)) - h2{1152.f16, 1152.f16};
}

// N words in the widest loads that their number allows (p is aligned to it).
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const void* p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = static_cast<const uint4*>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint2 v = static_cast<const uint2*>(p)[i];
            w[2 * i] = v.x; w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = static_cast<const uint32_t*>(p)[i];
    }
}

// One K row's codes of a lane: group g's four (4-bit) or eight (8-bit)
// bytes of every block.  Operand slots 0 .. 7 of a block: 4-bit elements
// 4g + {0, 2, 1, 3}, then 16 + 4g + {0, 2, 1, 3}; 8-bit elements 8g + 0 .. 7.
template <int BITS, int NB>
struct KCodes {
    uint32_t w[NB * BITS / 4];
    __device__ __forceinline__ void load(const uint8_t* p) { load_words<NB * BITS / 4>(w, p); }
    __device__ __forceinline__ h8 operand(int b, uint32_t k) const {
        if constexpr (BITS == 4) {
            const uint32_t x = w[b];
            return as_h8(nib_lo(x, k), nib_lo(x >> 8, k), nib_hi(x, k), nib_hi(x >> 8, k));
        } else {
            const uint32_t x = w[2 * b] ^ 0x80808080u, y = w[2 * b + 1] ^ 0x80808080u;
            return as_h8(bytes_of<0, 1>(x), bytes_of<2, 3>(x), bytes_of<0, 1>(y), bytes_of<2, 3>(y));
        }
    }
};

// Eight keys of V for the lane's elements i and 16 + i of every block.  Key
// order in a binary16 operand: 0, 2, 1, 3, 4, 6, 5, 7; in a bf16 operand
// 0 .. 7, 4-bit codes times 16.
template <int BITS, int NB>
struct VCodes {
    uint32_t w[NB * BITS / 2];
    __device__ __forceinline__ void load(const uint8_t* p) { load_words<NB * BITS / 2>(w, p); }
    __device__ __forceinline__ h8 operand(int b, int h, uint32_t k) const {
        if constexpr (BITS == 4) {
            const uint32_t x = w[2 * b], y = w[2 * b + 1];
            return h == 0 ? as_h8(nib_lo(x, k), nib_lo(x >> 8, k), nib_lo(y, k), nib_lo(y >> 8, k))
                          : as_h8(nib_hi(x, k), nib_hi(x >> 8, k), nib_hi(y, k), nib_hi(y >> 8, k));
        } else {
            const uint32_t x = w[4 * b + 2 * h] ^ 0x80808080u, y = w[4 * b + 2 * h + 1] ^ 0x80808080u;
            return as_h8(bytes_of<0, 2>(x), bytes_of<1, 3>(x), bytes_of<0, 2>(y), bytes_of<1, 3>(y));
        }
    }
    static __device__ __forceinline__ uint32_t bf(float a, float b) { return uppers(__float_as_uint(a), __float_as_uint(b)); }
    __device__ __forceinline__ u4 operand_bf16(int b, int h) const {
        uint32_t x, y;
        if constexpr (BITS == 4) {
            x = h == 0 ? q4x16_lo(w[2 * b]) : q4x16_hi(w[2 * b]);
            y = h == 0 ? q4x16_lo(w[2 * b + 1]) : q4x16_hi(w[2 * b + 1]);
        } else {
            x = w[4 * b + 2 * h];
            y = w[4 * b + 2 * h + 1];
        }
        return u4{bf(sbyte_f32<0>(x), sbyte_f32<1>(x)), bf(sbyte_f32<2>(x), sbyte_f32<3>(x)),
                  bf(sbyte_f32<0>(y), sbyte_f32<1>(y)), bf(sbyte_f32<2>(y), sbyte_f32<3>(y))};
    }
};

// Scales of a lane group's eight keys, every block.
template <int NB>
struct Scales {
    uint32_t w[4 * NB];  // keys 2i and 2i + 1 of block b at 4b + i
    __device__ __forceinline__ void load(const uint16_t* p) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[b];
            w[4 * b] = v.x; w[4 * b + 1] = v.y; w[4 * b + 2] = v.z; w[4 * b + 3] = v.w;
        }
    }
    __device__ __forceinline__ float at(int b, int j) const { return static_cast<float>(as_h2(w[4 * b + j / 2])[j % 2]); }
};

// Values that are the same in every lane, kept in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(uniform(static_cast<int>(v)))) |
                                static_cast<uint64_t>(static_cast<uint32_t>(uniform(static_cast<int>(v >> 32)))) << 32);
}

// The same value, which the compiler cannot carry over a loop: what follows
// from it is computed where it is used and holds no register elsewhere.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A sequence: its query rows and its keys.
struct Seq {
    int first;  // query row
    int n;      // query rows
    int len;    // keys
};

__device__ __forceinline__ Seq uniform(const Seq& s) { return Seq{uniform(s.first), uniform(s.n), uniform(s.len)}; }

// The tensors are taken at their word no further than the buffers reach.
__device__ __forceinline__ Seq sequence_of(const AttnArgs& a, int b) {
    Seq s;
    if (a.q_starts) {
        const int64_t x = min(static_cast<int64_t>(max(a.q_starts[b], 0)), a.T);
        const int64_t y = min(static_cast<int64_t>(max(a.q_starts[b + 1], 0)), a.T);
        s.first = static_cast<int>(x);
        s.n = static_cast<int>(max<int64_t>(y - x, 0));
    } else {
        s.n = static_cast<int>(a.T / a.batch);
        s.first = b * s.n;
    }
    const int64_t held = a.kv.pages > 0 ? a.table_width << a.kv.page_shift : 0;
    s.len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), held));
    return s;
}

// Four elements of a row as loaded.
template <bool F32>
struct Run4 {
    uint32_t w[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (F32) {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
            w[0] = v.x; w[1] = v.y;
        }
    }
    __device__ __forceinline__ float at(int i, Elem e) const {
        if constexpr (F32) return __uint_as_float(w[i]);
        else if (e == Elem::BF16) return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else return static_cast<float>(as_h2(w[i / 2])[i % 2]);
    }
};

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));

template <bool F32>
__device__ __forceinline__ void store4(void* out, int64_t at, Elem e, f4 v) {
    if constexpr (F32) *reinterpret_cast<f4*>(static_cast<float*>(out) + at) = v;
    else if (e == Elem::BF16) *reinterpret_cast<b4*>(static_cast<__bf16*>(out) + at) = __builtin_convertvector(v, b4);
    else *reinterpret_cast<h4*>(static_cast<_Float16*>(out) + at) = __builtin_convertvector(v, h4);
}

}  // namespace

}  // namespace qbd
