// Writing rows of keys and values into the quantized cache, and reading
// them back: memory-bound both ways.
//
// A wave takes eight rows (lane % 8) and eight pieces of them (lane / 8).  A
// piece is a quarter of a block: elements 4u .. 4u + 3 and 16 + 4u .. + 3,
// which are one word of a 4-bit K row and two of an 8-bit one, and four
// bytes (eight) of the interleaved V.  Eight consecutive slots put a V byte
// of neighbouring lanes side by side, so that even byte accesses touch whole
// 8-byte runs; rows of unrelated slots take the same code.  The lanes of a
// block are four apart by eight, and its maximum is one step inside a
// 16-lane row and one across two.
//
// What bounds them is how much a wave keeps in flight: a lane takes K's and
// V's piece, all its loads are under way before the first is used, and 16-bit
// rows move in 16 bytes.  32768 rows of 8 heads of 128, 4 bits to bf16 (172
// MB): 42 us, 4.1 TB/s, where K or V a lane and 8-byte accesses took 64; 8190
// such rows in bf16 into 8 and 4 bits: 16.7 us where they took 18.4 (both with
// the rows in cache; 18.1 from memory).  1, 2 and 4 pieces a lane when reading
// were level to 4%, 2 when writing 4% slower.
#include "kv_device.hpp"

namespace qbd {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));

template <Elem E> struct Vec4 { using type = f4; };
template <> struct Vec4<Elem::BF16> { using type = b4; };
template <> struct Vec4<Elem::F16> { using type = h4; };

// Where a lane's pieces are, in K and in V.
struct Piece {
    int u, b, head;
    bool live;
};

template <int NB>
__device__ __forceinline__ Piece piece_of(int heads, uint32_t at) {
    const uint32_t block = at >> 2, head = block / NB;
    return Piece{static_cast<int>(at & 3), static_cast<int>(block - head * NB), static_cast<int>(head), head < static_cast<uint32_t>(heads)};
}

// Pieces of K, and of V, that a lane takes, and waves that eight rows take.
constexpr int kWritePieces = 1, kReadPieces = 2;
template <int P>
__host__ __device__ __forceinline__ int64_t group_waves(int heads, int nb) { return (heads * nb * 4 + 8 * P - 1) / (8 * P); }

// 16-bit elements move in 16 bytes a lane: the lanes of pieces u and u + 1
// (u even, eight lanes apart) hold the first halves of both and the second
// halves of both in memory, and trade the half that is the other's.
__device__ __forceinline__ int neighbours_at(int u) { return u & 1 ? 32 + 8 * (u - 1) : 8 * u; }

template <class V>
__device__ __forceinline__ void trade(bool odd, V (&x)[2]) {
    const uint2 lo = __builtin_bit_cast(uint2, x[0]), hi = __builtin_bit_cast(uint2, x[1]);
    uint2 got;
    got.x = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(odd ? lo.x : hi.x), 0x128, 0xf, 0xf, false));  // row_ror:8
    got.y = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(odd ? lo.y : hi.y), 0x128, 0xf, 0xf, false));
    x[0] = __builtin_bit_cast(V, odd ? got : lo);
    x[1] = __builtin_bit_cast(V, odd ? hi : got);
}

template <int NB, Elem E>
__global__ __launch_bounds__(256) void kv_write_kernel(KvView kv, KvRows k, KvRows v, const int64_t* __restrict__ slots, int64_t T) {
    using V = typename Vec4<E>::type;
    const int lane = threadIdx.x & 63;
    const uint32_t per = group_waves<kWritePieces>(kv.heads, NB);
    const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6), group = wave / per;
    const int64_t row = static_cast<int64_t>(group) * 8 + (lane & 7);
    const int64_t slot = row < T ? slots[row] : -1;
    const bool live = slot >= 0 && slot < (kv.pages << kv.page_shift);
    Piece p[kWritePieces];
    alignas(16) V raw[kWritePieces][2][2] = {};
#pragma unroll
    for (int i = 0; i < kWritePieces; ++i) {
        p[i] = piece_of<NB>(kv.heads, ((wave - group * per) * kWritePieces + i) * 8 + (lane >> 3));
        if (live && p[i].live) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const KvRows& src = z ? v : k;
                const int64_t at = row * src.token_stride + p[i].head * src.head_stride + 32 * p[i].b;
                const char* base = static_cast<const char*>(src.p) + at * static_cast<int64_t>(sizeof(V) / 4);
                const int u = p[i].u;
                if constexpr (sizeof(V) == 16) {
                    raw[i][z][0] = *reinterpret_cast<const V*>(base + 16 * u);
                    raw[i][z][1] = *reinterpret_cast<const V*>(base + 64 + 16 * u);
                } else {
                    *reinterpret_cast<uint4*>(raw[i][z]) = *reinterpret_cast<const uint4*>(base + neighbours_at(u));
                }
            }
        }
    }
    const int64_t page = slot >> kv.page_shift;
    const int t = static_cast<int>(slot & ((1 << kv.page_shift) - 1));
#pragma unroll
    for (int i = 0; i < kWritePieces; ++i) {
        const int64_t head_at = (page * kv.heads + p[i].head) << kv.page_shift;  // tokens of heads before it
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int bits = z ? kv.vbits : kv.kbits;
            if constexpr (sizeof(V) == 8) trade(p[i].u & 1, raw[i][z]);
            f4 x[2];
            uint32_t top = 0;  // of the magnitudes' bits: NaN sorts above infinity
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j % 4 == 0) x[j / 4] = __builtin_convertvector(raw[i][z][j / 4], f4);
                top = max(top, __float_as_uint(x[j / 4][j % 4]) & 0x7fffffffu);
            }
            top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 8)));
            top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
            if (!live || !p[i].live) continue;

            const bool bad = top >= 0x7f800000u;
            const _Float16 d = kv_block_scale(__uint_as_float(top), bits);
            const float df = static_cast<float>(d), inv = 1.f / df, levels = static_cast<float>(kv_levels(bits));
            int q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = bad || df == 0.f ? 0 : static_cast<int>(kv_code(x[j / 4][j % 4], df, inv, levels));

            if (p[i].u == 0)
                (z ? kv.vd : kv.kd)[head_at * NB + (t / 8 * NB + p[i].b) * 8 + t % 8] = bad ? 0x7e00 : __builtin_bit_cast(uint16_t, d);
            const int u = p[i].u, b = p[i].b;
            if (bits == 4) {
                uint32_t w = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) w |= static_cast<uint32_t>((q[j] + 8) | (q[4 + j] + 8) << 4) << (8 * j);
                if (z == 0) {
                    *reinterpret_cast<uint32_t*>(kv.kc + (head_at + t) * (16 * NB) + (u * NB + b) * 4) = w;
                } else {
                    uint8_t* o = kv.vc + (head_at + (t & ~7)) * (16 * NB) + (t & 7);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[((4 * u + j) * NB + b) * 8] = static_cast<uint8_t>(w >> (8 * j));
                }
            } else if (z == 0) {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j / 4] |= static_cast<uint32_t>(q[j] & 255) << (8 * (j % 4));
                uint8_t* o = kv.kc + (head_at + t) * (32 * NB) + (u & 1) * 4 + b * 8;
                *reinterpret_cast<uint32_t*>(o + (u >> 1) * NB * 8) = w[0];
                *reinterpret_cast<uint32_t*>(o + (2 + (u >> 1)) * NB * 8) = w[1];
            } else {
                uint8_t* o = kv.vc + (head_at + (t & ~7)) * (32 * NB) + (t & 7);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[(((4 * u + j % 4) * NB + b) * 2 + j / 4) * 8] = static_cast<uint8_t>(q[j]);
            }
        }
    }
}

// BITS of K and of V are the kernel's: what is loaded of a piece stays in
// registers until all loads are under way.
template <int NB, Elem E, int KB, int VB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvView kv, const int64_t* __restrict__ slots, int64_t T,
                                                      void* __restrict__ k, void* __restrict__ v) {
    using V = typename Vec4<E>::type;
    constexpr int P = kReadPieces;
    const int lane = threadIdx.x & 63;
    const uint32_t per = group_waves<P>(kv.heads, NB);
    const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6), group = wave / per;
    const int64_t row = static_cast<int64_t>(group) * 8 + (lane & 7);
    if (row >= T) return;
    const int64_t slot = slots[row];
    const bool live = slot >= 0 && slot < (kv.pages << kv.page_shift);
    const int64_t page = slot >> kv.page_shift;
    const int t = static_cast<int>(slot & ((1 << kv.page_shift) - 1));
    Piece p[P];
    uint32_t kraw[P][KB / 4], vraw[P][VB];
    uint16_t d[P][2];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        p[i] = piece_of<NB>(kv.heads, ((wave - group * per) * P + i) * 8 + (lane >> 3));
#pragma unroll
        for (int j = 0; j < KB / 4; ++j) kraw[i][j] = KB == 4 ? 0x88888888u : 0u;  // zeros, where there is no slot
#pragma unroll
        for (int j = 0; j < VB; ++j) vraw[i][j] = VB == 4 ? 0x88u : 0u;
        d[i][0] = d[i][1] = 0;
        if (!live || !p[i].live) continue;
        const int u = p[i].u, b = p[i].b;
        const int64_t head_at = (page * kv.heads + p[i].head) << kv.page_shift, scale = head_at * NB + (t / 8 * NB + b) * 8 + t % 8;
        const uint8_t* kc = kv.kc + (head_at + t) * (4 * KB * NB);
        if constexpr (KB == 4) {
            kraw[i][0] = *reinterpret_cast<const uint32_t*>(kc + (u * NB + b) * 4);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) kraw[i][h] = *reinterpret_cast<const uint32_t*>(kc + (u & 1) * 4 + b * 8 + (2 * h + (u >> 1)) * NB * 8);
        }
        d[i][0] = kv.kd[scale];
        const uint8_t* vc = kv.vc + (head_at + (t & ~7)) * (4 * VB * NB) + (t & 7);
#pragma unroll
        for (int j = 0; j < VB; ++j)
            vraw[i][j] = VB == 4 ? vc[((4 * u + j) * NB + b) * 8] : vc[(((4 * u + j % 4) * NB + b) * 2 + j / 4) * 8];
        d[i][1] = kv.vd[scale];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (!p[i].live) continue;
        const int u = p[i].u;
        const int64_t at = (row * kv.heads + p[i].head) * (32 * NB) + 32 * p[i].b;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            uint32_t w[2] = {0, 0};  // signed codes; for 4 bits times 16
            if (z == 0) {
#pragma unroll
                for (int h = 0; h < KB / 4; ++h) w[h] = kraw[i][h];
            } else {
#pragma unroll
                for (int j = 0; j < VB; ++j) w[j / 4] |= vraw[i][j] << (8 * (j % 4));
            }
            float f = f16_bits_to_f32(d[i][z]);
            if ((z ? VB : KB) == 4) {
                f *= 0.0625f;  // exact
                w[1] = q4x16_hi(w[0]);
                w[0] = q4x16_lo(w[0]);
            }
            alignas(16) V x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) x[h] = __builtin_convertvector((f4{f * sbyte_f32<0>(w[h]), f * sbyte_f32<1>(w[h]), f * sbyte_f32<2>(w[h]), f * sbyte_f32<3>(w[h])}), V);
            char* to = static_cast<char*>(z ? v : k) + at * static_cast<int64_t>(sizeof(V) / 4);
            if constexpr (sizeof(V) == 16) {
                *reinterpret_cast<V*>(to + 16 * u) = x[0];
                *reinterpret_cast<V*>(to + 64 + 16 * u) = x[1];
            } else {
                trade(u & 1, x);
                *reinterpret_cast<uint4*>(to + neighbours_at(u)) = *reinterpret_cast<const uint4*>(x);
            }
        }
    }
}

// Rows of one launch: a grid holds fewer than 2^32 threads.
inline int64_t launch_rows(int64_t per) { return ((int64_t{1} << 25) / per + 1) * 8; }

template <int NB, Elem E>
hipError_t write_as(const KvView& kv, KvRows k, KvRows v, const int64_t* slots, int64_t T, hipStream_t stream) {
    const int64_t per = group_waves<kWritePieces>(kv.heads, NB), most = launch_rows(per), eb = elem_bytes(E);
    for (; T > 0; T -= most, slots += most) {
        const int64_t n = T < most ? T : most, waves = (n + 7) / 8 * per;
        hipLaunchKernelGGL((kv_write_kernel<NB, E>), dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, stream, kv, k, v, slots, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        k.p = static_cast<const char*>(k.p) + most * k.token_stride * eb;
        v.p = static_cast<const char*>(v.p) + most * v.token_stride * eb;
    }
    return hipSuccess;
}

template <int NB, Elem E, int KB, int VB>
hipError_t read_bits(const KvView& kv, const int64_t* slots, int64_t T, void* k, void* v, hipStream_t stream) {
    const int64_t per = group_waves<kReadPieces>(kv.heads, NB), most = launch_rows(per);
    const int64_t out = most * kv.heads * (32 * NB) * elem_bytes(E);
    for (; T > 0; T -= most, slots += most) {
        const int64_t n = T < most ? T : most, waves = (n + 7) / 8 * per;
        hipLaunchKernelGGL((kv_read_kernel<NB, E, KB, VB>), dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, stream, kv, slots, n, k, v);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        k = static_cast<char*>(k) + out;
        v = static_cast<char*>(v) + out;
    }
    return hipSuccess;
}

template <int NB, Elem E>
hipError_t read_as(const KvView& kv, const int64_t* slots, int64_t T, void* k, void* v, hipStream_t stream) {
    if (kv.kbits == 4) return read_bits<NB, E, 4, 4>(kv, slots, T, k, v, stream);
    return kv.vbits == 8 ? read_bits<NB, E, 8, 8>(kv, slots, T, k, v, stream) : read_bits<NB, E, 8, 4>(kv, slots, T, k, v, stream);
}

template <int NB>
hipError_t write_dim(const KvView& kv, const KvRows& k, const KvRows& v, Elem e, const int64_t* slots, int64_t T, hipStream_t stream) {
    if (e == Elem::F32) return write_as<NB, Elem::F32>(kv, k, v, slots, T, stream);
    if (e == Elem::BF16) return write_as<NB, Elem::BF16>(kv, k, v, slots, T, stream);
    return write_as<NB, Elem::F16>(kv, k, v, slots, T, stream);
}

template <int NB>
hipError_t read_dim(const KvView& kv, const int64_t* slots, int64_t T, Elem e, void* k, void* v, hipStream_t stream) {
    if (e == Elem::F32) return read_as<NB, Elem::F32>(kv, slots, T, k, v, stream);
    if (e == Elem::BF16) return read_as<NB, Elem::BF16>(kv, slots, T, k, v, stream);
    return read_as<NB, Elem::F16>(kv, slots, T, k, v, stream);
}

}  // namespace

hipError_t launch_kv_write(const KvView& kv, const KvRows& k, const KvRows& v, Elem e, const int64_t* slots, int64_t T,
                           hipStream_t stream) {
    switch (kv.dim) {
        case 64: return write_dim<2>(kv, k, v, e, slots, T, stream);
        case 96: return write_dim<3>(kv, k, v, e, slots, T, stream);
        case 128: return write_dim<4>(kv, k, v, e, slots, T, stream);
        case 192: return write_dim<6>(kv, k, v, e, slots, T, stream);
        case 256: return write_dim<8>(kv, k, v, e, slots, T, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_kv_read(const KvView& kv, const int64_t* slots, int64_t T, Elem e, void* k, void* v, hipStream_t stream) {
    switch (kv.dim) {
        case 64: return read_dim<2>(kv, slots, T, e, k, v, stream);
        case 96: return read_dim<3>(kv, slots, T, e, k, v, stream);
        case 128: return read_dim<4>(kv, slots, T, e, k, v, stream);
        case 192: return read_dim<6>(kv, slots, T, e, k, v, stream);
        case 256: return read_dim<8>(kv, slots, T, e, k, v, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace qbd
