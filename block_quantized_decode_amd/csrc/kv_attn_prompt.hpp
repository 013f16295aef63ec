// Attention over the quantized key/value cache for many query rows a cached
// head (prompts and their chunks), 16-bit rows: bound by the matrix cores
// and the softmax beside them.
//
// A workgroup of W waves owns 32 W query rows (token, query head of the group)
// of one cached head, 32 a wave, and walks the keys in tiles of BN.  For each
// tile its threads turn the codes into binary16 elements d * code in LDS, once
// for all rows, while the tile before is being used; the products run on
// v_mfma_f32_32x32x16_f16 as
//   S^T = K Q^T,  O^T = V^T P^T,
// so that a lane holds 16 of a tile's 32 scores of one row, which are the K
// slots 8 (lane / 32) + j of the second product when V's keys are laid out
// in the same order: the weights stay in their lane.
//
// What bounds it is the vector work beside the matrix cores (a weight costs an
// exponential, an element of a tile its expansion) and what a wave cannot
// overlap by itself, as it issues in order.  Hence two waves a SIMD (one alone
// runs its products and its vector work in turn), eight waves on one tile
// where there are rows for them (half the expansion of four: 197 -> 185 us at
// 4096 rows x 8 heads of 8192 keys of 128 elements, 4-bit codes), addresses
// found for 16 tiles at once and the scales looked at by one wave for all
// (185 -> 172 us; now 167, 774 TFLOP/s, 59% of what a large fp16 matrix product
// reaches), and an order laid out by hand:
//   scores of keys 0-31        | the next tile's expansion
//   scores of keys 32-63       | weights of keys 0-31
//   sums over keys 0-31        | weights of keys 32-63
//   sums over keys 32-63
// 64 rows a wave (an LDS operand for two products) needs one wave a SIMD and
// took 218 us.  The reference of a row is a whole number (its moves are
// exact), so weights made before a move are moved with the sums.
//
// Rows of too few workgroups for the card are walked in `parts` runs of
// keys, joined by a second launch.
//
// Roundings (11 bits each): an element d * code, exact in 18 bits, a weight
// relative to its row's running maximum; q is scaled by a power of two as in
// the split kernel.  d * code is a multiple of the type's smallest step, so
// it is exact or good to 11 bits however small.  It overflows where d is above
// 256: such a block enters times 2^-8, block by block, and in a tile that has
// one the products over those blocks are made once more and 255 times their
// result is added (1024 rows of 32 over 8 heads, 8192 keys of 128: 1.6 times as
// long with such a K block in every tile, 1.4 with one of V, 2.1 and 1.8 where
// all are).  What keys that no row sees hold can cost that, but changes no bit.
#pragma once

#include "kv_attn.hpp"

namespace qbd {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f16v mfma32(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// LDS places, in 16-byte chunks of eight elements.  K: a row a key, chunk
// 4b + g holds what lane group g of a K row's codes gives for block b.  V: a
// row an element, chunk 2c + half holds keys 16c + 4 half + {0, 2, 1, 3} and
// 16c + 8 + 4 half + {0, 2, 1, 3}.  The exclusive or spreads 16 rows of one
// chunk, and the 16 chunks that neighbouring lanes write, over the banks.
template <int NB>
__device__ __forceinline__ int k_chunk(int key, int chunk) {
    if constexpr (NB == 4 || NB == 8) return key * (4 * NB) + (chunk ^ ((key & 3) * 4 + (key >> 2 & 3)));
    else if constexpr (NB == 2) return key * 8 + (chunk ^ ((key >> 1 & 1) * 4 + (key >> 2 & 3)));
    else return key * (4 * NB + 1) + chunk;
}
template <int NB>
constexpr int k_row_chunks() { return NB == 3 || NB == 6 ? 4 * NB + 1 : 4 * NB; }

template <int BN>
__device__ __forceinline__ int v_chunk(int d, int chunk) {
    if constexpr (BN == 64) return d * 8 + (chunk ^ ((d >> 1 & 7) ^ (d >> 5 & 3) << 1));
    else return d * 4 + (chunk ^ (d >> 2 & 3));
}

template <int NB, int BN>
struct TileLds {
    u4 k[BN * k_row_chunks<NB>()];
    u4 v[32 * NB * BN / 8];
};

// LDS by its own addresses: an exclusive or on one is one instruction
__device__ __forceinline__ uint32_t lds_place(void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)p));
}
__device__ __forceinline__ u4 lds_read(uint32_t place) {
    return *reinterpret_cast<__attribute__((address_space(3))) const u4*>(static_cast<uintptr_t>(place));
}

// A row in operand order for steps of 16 elements (chunk 2x + half of K's
// order is 4b + g), scaled (kQueryTop); returns the factor of its scores in
// units of log2.
template <int KB, int NB>
__device__ __forceinline__ float load_query(const AttnArgs& a, int64_t at, int half, h8 (&q)[2 * NB]) {
    constexpr int kRun = KB == 4 ? 16 : 4;
    Run4<false> raw[2 * NB][2];
    float top = 0.f;
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
        const int first = 32 * (x / 2) + (KB == 4 ? 4 : 8) * (x % 2 * 2 + half);
        raw[x][0].load(a.q.p, at + first);
        raw[x][1].load(a.q.p, at + first + kRun);
    }
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(raw[x][i / 4].at(i % 4, a.elem)));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const int e = __builtin_amdgcn_frexp_expf(top) - kQueryTop;
    const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[x][j] = static_cast<_Float16>(sign * ldexpf(raw[x][j / 4].at(KB == 4 ? j % 2 * 2 + j % 4 / 2 : j % 4, a.elem), -e));
    }
    // not zero, so that a masked score of minus infinity stays one
    return fmaxf(ldexpf(fabsf(a.scale) * 1.44269504088896340736f, e), 1.17549435e-38f);
}

// What one thread fetches of a tile.  A wave works on one run of 16 keys, or
// two waves do: on half the blocks of K each, and on half the keys of V or
// (more than 128 elements) half its elements.  A lane takes a quarter of a K
// row's blocks and two elements of V, with their scales.  The run lies in one
// page, so its addresses are a scalar base and an offset that never changes.
template <int KB, int VB, int NBT, int Z>
struct Fetch {
    uint32_t k[NBT * KB / 4];
    uint32_t kd[NBT];  // one scale each
    uint32_t v[Z][VB / 2];
    uint32_t vd[Z][4];
};

// Partial results, where the keys of the rows are walked in parts.
struct Prompt {
    int group;     // query heads a cached head
    int parts;
    float* part;   // [workgroups][rows][dim]
    float2* stat;  // [workgroups][rows]: reference, weight total
};

template <int KB, int VB, int NB, int BN, int W>
__global__ __launch_bounds__(64 * W, kv_plan::prompt_groups_a_cu(NB, W) * W / 4) void kv_attn_prompt(AttnArgs a, Prompt pr) {
    constexpr int D = 32 * NB, ROWS = 32 * W, UNITS = BN / 16, STEPS = BN / 32, SPLIT = W / UNITS, NBT = NB / SPLIT;
    constexpr bool kByKeys = SPLIT == 2 && NB <= 4;
    constexpr int Z = kByKeys ? 1 : 2;
    constexpr int krow = D * KB / 8, vrow = D * VB / 8;
    using Lds = TileLds<NB, BN>;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int lane = threadIdx.x & 63, half = lane >> 5, group = pr.group;
    const int wave = uniform(static_cast<int>(threadIdx.x >> 6));
    Lds* buf = reinterpret_cast<Lds*>(smem);
    const int head = blockIdx.x;

    for (int b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const Seq s = uniform(sequence_of(a, b));
    const int total = s.n * group;
    const int row_tiles = (total + ROWS - 1) / ROWS;
    for (int y = blockIdx.y;; y += gridDim.y) {
    // row tiles, the longest first: as many as the grid was planned for in
    // parts, any more whole
    const bool planned = y < static_cast<int>(gridDim.y);
    const int order = planned ? y / pr.parts : gridDim.y / pr.parts + (y - gridDim.y);
    if (order >= row_tiles) break;
    const int parts = planned ? pr.parts : 1, part = planned ? y % pr.parts : 0;
    const int row0 = (row_tiles - 1 - order) * ROWS;
    const int rows = min(ROWS, total - row0);

    // keys that the workgroup's rows see, and its part of them
    const int tok_a = row0 / group, tok_b = (row0 + rows - 1) / group;
    const int end = a.causal ? max(0, min(s.len, s.len - s.n + tok_b + 1)) : s.len;
    const int begin = a.window > 0 ? static_cast<int>(max<int64_t>(static_cast<int64_t>(s.len) - s.n + tok_a - a.window + 1, 0)) & ~(BN - 1) : 0;
    const int tiles = end > begin ? (end - begin + BN - 1) / BN : 0;
    const int first = static_cast<int>(static_cast<int64_t>(tiles) * part / parts);
    const int stop = static_cast<int>(static_cast<int64_t>(tiles) * (part + 1) / parts);

    // the lane's rows, and what all rows of the wave see
    h8 q[2 * NB];
    f16v acc[NB];
    const int row = row0 + min(32 * wave + (lane & 31), rows - 1);
    const int tok = row / group;
    const int64_t pos = static_cast<int64_t>(s.len) - s.n + tok;
    const int hi_r = a.causal ? static_cast<int>(max<int64_t>(pos + 1, 0)) : s.len;
    const int lo_r = a.window > 0 ? static_cast<int>(max<int64_t>(pos - a.window + 1, 0)) : 0;
    const float c = load_query<KB, NB>(a, (s.first + tok) * a.q.token_stride + (head * group + row - tok * group) * a.q.head_stride, half, q);
    float ref = kNoKey, sum = 0.f;
    bool far = false;  // a reference of the wave is
#pragma unroll
    for (int x = 0; x < NB; ++x) {
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[x][i] = 0.f;
    }
    const int tok_f = (row0 + min(32 * wave, rows - 1)) / group, tok_l = (row0 + min(32 * wave + 31, rows - 1)) / group;
    const int hi_all = a.causal ? s.len - s.n + tok_f + 1 : s.len, hi_any = a.causal ? s.len - s.n + tok_l + 1 : s.len;
    const int lo_all = a.window > 0 ? static_cast<int>(max<int64_t>(static_cast<int64_t>(s.len) - s.n + tok_l - a.window + 1, 0)) : 0;
    const int lo_any = a.window > 0 ? static_cast<int>(max<int64_t>(static_cast<int64_t>(s.len) - s.n + tok_f - a.window + 1, 0)) : 0;

    const int32_t* table = a.table + b * a.table_width;
    const int shift = a.kv.page_shift, mask = (1 << shift) - 1;

    // the thread's part of a tile
    const int unit = wave / SPLIT, other = wave % SPLIT;
    const int kkey = lane >> 2, kgrp = lane & 3, kb0 = other * NBT, vz = kByKeys ? other : 0;
    const int vib = (kByKeys ? 0 : other * (16 / SPLIT * NB)) + min(lane, (kByKeys ? 16 : 16 / SPLIT) * NB - 1);  // the rest repeat the last
    const int off_k = kkey * krow + kgrp * (krow / 4) + kb0 * KB;
    const int off_kd = (kkey & 8) * NB + kb0 * 8 + (kkey & 7);
    const int off_v = vib * (2 * VB), off_vd = vib % NB * 8;
    const int lds_k = 16 * k_chunk<NB>(16 * unit + kkey, 4 * kb0 + kgrp);
    const int lds_v = 16 * v_chunk<BN>(32 * (vib % NB) + vib / NB, 2 * unit) + 8 * vz;
    const uint32_t lane_k = lds_place(smem) + 16 * k_chunk<NB>(lane & 31, half);
    const uint32_t lane_v = lds_place(smem) + static_cast<uint32_t>(sizeof(Lds::k)) + 16 * v_chunk<BN>(lane & 31, half);
    const uint32_t magic = pair1024();
    Fetch<KB, VB, NBT, Z> f;

    // Where the runs of 16 keys of the next 64 / UNITS tiles are, a run a lane:
    // tokens of the head before it, or of page 0 when its page is not held.
    constexpr int kRuns = 64 / UNITS;
    int64_t runs = 0;
    uint64_t runs_held = 0;
    auto find_runs = [&](int j) {
        const int t = begin + (j + lane / UNITS) * BN + lane % UNITS * 16;
        int id = t < end && j + lane / UNITS < stop ? table[t >> shift] : -1;
        id = fresh(id);  // waited for here, so that no other tile's loads are
        const bool ok = static_cast<uint32_t>(id) < static_cast<uint64_t>(a.kv.pages);
        runs_held = __ballot(ok);
        runs = ((static_cast<int64_t>(ok ? id : 0) * a.kv.heads + head) << shift) + (t & mask);
    };
    // the wave's run of the tile that is fetched next, and which are held
    int64_t run = 0;
    uint32_t run_held = 0;
    auto find = [&](int n) {  // tile first + n
        if (n % kRuns == 0) find_runs(first + n);
        const int at = n % kRuns * UNITS;
        run_held = static_cast<uint32_t>(runs_held >> at) & ((1u << UNITS) - 1);
        run = static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(runs), at + unit)) |
                                   static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(runs >> 32), at + unit))) << 32);
    };
    uint32_t held_next = 0, held = 0;  // runs of 16 keys that are held
    auto fetch = [&]() {
        held_next = run_held;
        load_words<NBT * KB / 4>(f.k, a.kv.kc + run * krow + off_k);
        const uint16_t* kd = a.kv.kd + run * NB + off_kd;
#pragma unroll
        for (int y = 0; y < NBT; ++y) f.kd[y] = kd[y * 8];
#pragma unroll
        for (int z = 0; z < Z; ++z) {
            load_words<VB / 2>(f.v[z], a.kv.vc + (run + 8 * (z + vz)) * vrow + off_v);
            load_words<4>(f.vd[z], a.kv.vd + (run + 8 * (z + vz)) * NB + off_vd);
        }
    };
    // All scales of a tile are looked at by one wave, three tiles ahead, which
    // leaves for all waves what the tile's use has to know: 1 K scales are
    // above 256, 2 V scales are, 4 a V scale is no number.
    int* const notes = reinterpret_cast<int*>(smem + 2 * sizeof(Lds));
    u4 scan = {0, 0, 0, 0};
    auto look = [&](int n) {
        const int chunk = min(lane & 31, 2 * NB * UNITS - 1), at = n % kRuns * UNITS + chunk / (2 * NB);
        const int64_t from = static_cast<int64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(runs), at)) |
                                                  static_cast<uint64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(runs >> 32), at))) << 32);
        scan = *reinterpret_cast<const u4*>((half ? a.kv.vd : a.kv.kd) + from * NB + chunk % (2 * NB) * 8);
    };
    auto note = [&](int n) {
        int flags = 0;
        if (__any(((scan[0] | scan[1] | scan[2] | scan[3]) & 0x40004000u) != 0)) {  // a scale of 2 or more
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(scan[i] & 0x7fffu, scan[i] >> 16 & 0x7fffu));
            const uint64_t big = __ballot(top > 0x5c00u), nan = __ballot(top >= 0x7c00u);
            flags = (static_cast<uint32_t>(big) != 0 ? 1 : 0) | (big >> 32 != 0 ? 2 : 0) | (nan >> 32 != 0 ? 4 : 0);
        }
        if (lane == 0) notes[n & 3] = flags;
    };
    // The fetched scales made fit, before their tile is expanded: those above
    // 256 times 2^-8, none for a V key that is not there or is no number.
    int flags_next = 0;
    auto large = [](uint32_t d) { return (d & 0x7fffu) > 0x5c00u; };  // a NaN too
    auto adjust = [&](int j) {
        flags_next = uniform(notes[(j - first) & 3]);
        if (flags_next & 1) {
#pragma unroll
            for (int y = 0; y < NBT; ++y) f.kd[y] = large(f.kd[y]) ? __builtin_bit_cast(uint16_t, static_cast<_Float16>(as_h2(f.kd[y])[0] * 0.00390625f16)) : f.kd[y];
        }
        const int t = begin + j * BN + 16 * unit;
        const bool ok = held_next >> unit & 1;
        if (!ok || t + 16 > end || (flags_next & 4)) {
#pragma unroll
            for (int i = 0; i < 4 * Z; ++i) {
                const int key = t + 8 * vz + 2 * i;
                uint32_t& w = f.vd[i / 4][i % 4];
                const bool x = ok && key < end && (w & 0x7c00u) != 0x7c00u;
                const bool y = ok && key + 1 < end && (w & 0x7c000000u) != 0x7c000000u;
                w &= (x ? 0xffffu : 0u) | (y ? 0xffff0000u : 0u);
            }
        }
        if (flags_next & 2) {
#pragma unroll
            for (int i = 0; i < 4 * Z; ++i) {
                uint32_t& w = f.vd[i / 4][i % 4];
                const uint32_t less = __builtin_bit_cast(uint32_t, as_h2(w) * h2{0.00390625f16, 0.00390625f16});
                w = ((large(w) ? less : w) & 0xffffu) | ((large(w >> 16) ? less : w) & 0xffff0000u);
            }
        }
        held = held_next;
    };
    // codes to elements in LDS, in kPieces pieces: NBT of K, then two keys'
    // halves by two elements of V
    constexpr int kPieces = NBT + 2 * Z;
    auto expand = [&](Lds& o, int piece) {
        char* base = reinterpret_cast<char*>(&o);
        if (piece < NBT) {
            KCodes<KB, 1> kc;
#pragma unroll
            for (int i = 0; i < KB / 4; ++i) kc.w[i] = f.k[KB / 4 * piece + i];
            const _Float16 d = as_h2(f.kd[piece])[0];
            char* to = base;
            if constexpr (NB == 3 || NB == 6) to += lds_k + 64 * piece;
            else to += lds_k ^ (64 * piece);  // the block is bits 6 and up of the place, under the exclusive or
            *reinterpret_cast<u4*>(to) = __builtin_bit_cast(u4, kc.operand(0, magic) * d);
            return;
        }
        const int z = (piece - NBT) % Z, h = (piece - NBT) / Z;
        VCodes<VB, 1> vc;
#pragma unroll
        for (int i = 0; i < VB / 2; ++i) vc.w[i] = f.v[z][i];
        const h8 x = vc.operand(0, h, magic);
        h2 e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the operand's pairs: keys 0, 2; 1, 3; 4, 6; 5, 7
            const h2 sc = as_h2(__builtin_amdgcn_perm(f.vd[z][i / 2 * 2 + 1], f.vd[z][i / 2 * 2], i % 2 ? 0x07060302u : 0x05040100u));
            e[i] = h2{x[2 * i], x[2 * i + 1]} * sc;
        }
        char* to = base + sizeof(Lds::k) + 16 * h * (2 * BN) + 8 * z;  // element 16h + i: the same exclusive or
        *reinterpret_cast<uint2*>(to + lds_v) = make_uint2(__builtin_bit_cast(uint32_t, e[0]), __builtin_bit_cast(uint32_t, e[1]));
        *reinterpret_cast<uint2*>(to + (lds_v ^ 16)) = make_uint2(__builtin_bit_cast(uint32_t, e[2]), __builtin_bit_cast(uint32_t, e[3]));
    };
    auto expand_all = [&](Lds& o) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) expand(o, i);
    };

    int held_lds = 0;
    const int count = stop - first;
    if (count > 0) {
        find(0);
        fetch();
        if (wave < 3) {
            look(wave);
            note(wave);
        }
        __syncthreads();
        adjust(first);
        expand_all(buf[0]);
        held_lds = held;
        find(1);
        if (count > 1) fetch();
        find(2);
    }
    // in the midst of tile first + n: the tile after the next is fetched
    auto ahead = [&](int n) {
        if (n + 2 < count) fetch();
        if (n + 3 < count) {
            find(n + 3);
            if ((n + 3) % W == wave) look(n + 3);
        }
    };
    for (int j = first; j < stop; ++j) {
        __syncthreads();
        const int flags = flags_next;
        const int held_now = held_lds, n = j - first;
        if (n > 0 && (n + 2) % W == wave) note(n + 2);
        if (j + 1 < stop) {
            adjust(j + 1);
            held_lds = held;
        }
        Lds& out = buf[(j + 1 - first) & 1];
        const int t0 = begin + j * BN;
        if (t0 >= hi_any || t0 + BN <= lo_any) {  // not seen by this wave
            expand_all(out);
            ahead(n);
            continue;
        }
        const bool masked = held_now != (1 << UNITS) - 1 || t0 + BN > min(hi_all, s.len) || t0 < lo_all;
        f16v sc[STEPS];
        h8 p[UNITS];
        // places of the lane's operands: the chunk number is under an
        // exclusive or, all else is an offset
        const uint32_t at = static_cast<uint32_t>(n & 1) * static_cast<uint32_t>(sizeof(Lds));
        const uint32_t at_k = at + lane_k, at_v = at + lane_v;
        auto k_operand = [&](int n, int x) {
            const uint32_t place = NB == 3 || NB == 6 ? at_k + 32 * x : at_k ^ (32 * x);
            return __builtin_bit_cast(h8, lds_read(place + 32 * n * 16 * k_row_chunks<NB>()));
        };
        auto v_operand = [&](int i) {
            const int x = i % NB, y = i / NB;
            const uint32_t place = at_v ^ (32 * (BN == 64 ? y ^ (x & 3) : y));
            return __builtin_bit_cast(h8, lds_read(place + 32 * x * 2 * BN));
        };
        // (a tile with notes) which of its keys have a scale in block x that
        // asks(d) is about: a key a lane
        auto keys_where = [&](const uint16_t* scales, int x, auto asks) {
            const int u = min(lane / 16, UNITS - 1), t = t0 + 16 * u + lane % 16;
            const int64_t page = t < end ? table[t >> shift] : -1;
            const bool ok = lane < BN && page >= 0 && page < a.kv.pages;
            const int64_t at = (((ok ? page : 0) * a.kv.heads + head) << shift) + (t & mask);
            const uint32_t d = ok ? scales[(at & ~int64_t{7}) * NB + 8 * x + (at & 7)] : 0;
            return __ballot(asks(d));
        };
        // scores of step n, work(x) between the products
        auto score = [&](int n, auto work) {
            h8 next[2] = {k_operand(n, 0), k_operand(n, 1)};
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[n][i] = 0.f;
#pragma unroll
            for (int x = 0; x < 2 * NB; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                const h8 cur = next[x & 1];
                sc[n] = mfma32(cur, q[x], sc[n]);
                if (x + 2 < 2 * NB) next[x & 1] = k_operand(n, x + 2);
                work(x);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        float by = c, less = 0.f;  // the exponent of a weight is its score times by, less this
        // masks, and a reference that the step's scores fit; the weights of
        // `made` steps before it in this tile move with it
        auto settle = [&](int n, int made) {
            if (flags & 1) {  // blocks of K that entered times 2^-8
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    const uint32_t keys = static_cast<uint32_t>(keys_where(a.kv.kd, x, large) >> (32 * n));
                    if (keys == 0) continue;
                    f16v part;
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[i] = 0.f;
                    part = mfma32(k_operand(n, 2 * x), q[2 * x], part);
                    part = mfma32(k_operand(n, 2 * x + 1), q[2 * x + 1], part);
                    const uint32_t mine = keys >> (4 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i) sc[n][i] = mine >> (8 * (i / 4) + i % 4) & 1 ? fmaf(255.f, part[i], sc[n][i]) : sc[n][i];
                }
            }
            if (masked) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int k = 32 * n + 8 * (i / 4) + 4 * half + i % 4;
                    const bool see = t0 + k < min(hi_r, s.len) && t0 + k >= lo_r && (held_now >> (2 * n + i / 8) & 1);
                    sc[n][i] = see ? sc[n][i] : -INFINITY;
                }
            }
            float top = sc[n][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, sc[n][i]);
            const float mark = top * c;
            by = c;
            less = ref;
            if (__any(mark > ref + kTop) || far) {
                const float score = fmaxf(mark, __shfl_xor(mark, 32));
                const float best = fmaxf(ref, is_far(score) ? score : ceilf(score) - kLift);
                const float z = __builtin_amdgcn_exp2f(ref - best);
                ref = less = best;
                sum *= z;
#pragma unroll
                for (int x = 0; x < NB; ++x) acc[x] *= z;
#pragma unroll
                for (int u = 0; u < 2 * made; ++u) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[u][i] = static_cast<_Float16>(static_cast<float>(p[u][i]) * z);
                }
                far |= __any(is_far(best));
                if (far) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) sc[n][i] = sc[n][i] * by - less;
                    by = 1.f;
                    less = 0.f;
                }
            }
        };
        // weights of scores 2i and 2i + 1 of step n as the second product
        // takes them: keys r and r + 2 of a run of four
        auto weigh = [&](int n, int i) {
            const int at = i / 2 * 4 + i % 2;
            h2 w;
#pragma unroll
            for (int z = 0; z < 2; ++z) w[z] = static_cast<_Float16>(__builtin_amdgcn_exp2f(fmaf(sc[n][at + 2 * z], by, -less)));
            // pinned here: left to itself the compiler moves this to where the
            // weights are used, out from between the products
            w = as_h2(static_cast<uint32_t>(fresh(static_cast<int>(__builtin_bit_cast(uint32_t, w)))));
            p[2 * n + i / 4][i % 4 * 2] = w[0];
            p[2 * n + i / 4][i % 4 * 2 + 1] = w[1];
            sum = __builtin_amdgcn_fdot2(w, h2{1.f16, 1.f16}, sum, false);
        };
        // weights of step n in 2 NB pieces
        auto weigh_piece = [&](int n, int x) {
#pragma unroll
            for (int i = x * 8 / (2 * NB); i < (x + 1) * 8 / (2 * NB); ++i) weigh(n, i);
        };
        // sums over step n
        auto add = [&](int n, auto work) {
            h8 next[2] = {v_operand(2 * n * NB), v_operand(2 * n * NB + 1)};
#pragma unroll
            for (int x = 0; x < 2 * NB; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                const int i = 2 * n * NB + x;
                const h8 cur = next[x & 1];
                acc[i % NB] = mfma32(cur, p[i / NB], acc[i % NB]);
                if (x + 2 < 2 * NB) next[x & 1] = v_operand(i + 2);
                work(x);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto nothing = [](int) {};

        // (after the last tile the expansion is of no use, and nothing reads it)
        score(0, [&](int x) {
#pragma unroll
            for (int i = x * kPieces / (2 * NB); i < (x + 1) * kPieces / (2 * NB); ++i) expand(out, i);
        });
        ahead(n);
        settle(0, 0);
        if constexpr (STEPS == 2) {
            score(1, [&](int x) { weigh_piece(0, x); });
            settle(1, 1);
            add(0, [&](int x) { weigh_piece(1, x); });
            add(1, nothing);
        } else {
#pragma unroll
            for (int x = 0; x < 2 * NB; ++x) weigh_piece(0, x);
            add(0, nothing);
        }
        if (flags & 2) {  // blocks of V that entered times 2^-8
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                const uint64_t keys = keys_where(a.kv.vd, x, [&](uint32_t d) { return large(d) && (d & 0x7c00) != 0x7c00; });
                if (keys == 0) continue;
                f16v part;
#pragma unroll
                for (int i = 0; i < 16; ++i) part[i] = 0.f;
#pragma unroll
                for (int u = 0; u < UNITS; ++u) {
                    const uint32_t mine = static_cast<uint32_t>(keys >> (16 * u)) >> (4 * half);
                    h8 w = p[u];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = mine >> (8 * (i / 4) + i / 2 % 2 + 2 * (i % 2)) & 1 ? w[i] : 0.f16;
                    part = mfma32(v_operand(u * NB + x), w, part);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[x][i] = fmaf(255.f, part[i], acc[x][i]);
            }
        }
        if (flags & 4) {  // a V scale that is no number spoils the rows that see it
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                const uint64_t bad = keys_where(a.kv.vd, x, [](uint32_t d) { return (d & 0x7c00) == 0x7c00; });
                const int lo = min(max(lo_r - t0, 0), BN), hi = min(max(min(hi_r, s.len) - t0, 0), BN);
                const uint64_t below = hi >= 64 ? ~uint64_t{0} : (uint64_t{1} << hi) - 1;
                const uint64_t seen = lo >= 64 ? 0 : below & ~((uint64_t{1} << lo) - 1);
                if (bad & seen) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[x][i] = __builtin_nanf("");
                }
            }
        }
    }

    sum += __shfl_xor(sum, 32);
    const int at_row = 32 * wave + (lane & 31);
    if (at_row < rows && parts > 1) {
        const int64_t slot = ((static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * ROWS + at_row;
        float* to = pr.part + slot * D + 4 * half;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f4*>(to + 32 * x + 8 * i) = f4{acc[x][4 * i], acc[x][4 * i + 1], acc[x][4 * i + 2], acc[x][4 * i + 3]};
        }
        if (half == 0) pr.stat[slot] = make_float2(ref, sum);
    } else if (at_row < rows) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t at = ((static_cast<int64_t>(s.first) + tok) * a.qheads + head * group + (row - tok * group)) * D + 4 * half;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store4<false>(a.out, at + 32 * x + 8 * i, a.elem,
                              f4{acc[x][4 * i] * inv, acc[x][4 * i + 1] * inv, acc[x][4 * i + 2] * inv, acc[x][4 * i + 3] * inv});
        }
    }
    __syncthreads();  // LDS is free for the next rows
    }
    }
}

// Adds the parts: a workgroup takes 32 rows.
template <int NB, int ROWS>
__global__ __launch_bounds__(256) void kv_attn_prompt_join(AttnArgs a, Prompt pr, int grid_y) {
    constexpr int D = 32 * NB, LANES = D / 4;
    const int head = blockIdx.x, b = blockIdx.z;
    const Seq s = uniform(sequence_of(a, b));
    const int total = s.n * pr.group, row_tiles = (total + ROWS - 1) / ROWS;
    const int y = blockIdx.y / (ROWS / 32), rt = row_tiles - 1 - y;
    if (rt < 0) return;
    for (int e = threadIdx.x; e < 32 * LANES; e += 256) {
        const int at_row = blockIdx.y % (ROWS / 32) * 32 + e / LANES, d = e % LANES * 4, row = rt * ROWS + at_row;
        if (row >= total) break;
        float best = kNoKey, sum = 0.f;
        f4 o = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < pr.parts; ++p) {
            const int64_t slot = ((static_cast<int64_t>(b) * grid_y + y * pr.parts + p) * gridDim.x + head) * ROWS + at_row;
            const float2 st = pr.stat[slot];
            const f4 x = *reinterpret_cast<const f4*>(pr.part + slot * D + d);
            const float top = fmaxf(best, st.x);
            const float f = __builtin_amdgcn_exp2f(best - top), h = __builtin_amdgcn_exp2f(st.x - top);
            best = top;
            sum = fmaf(sum, f, h * st.y);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = fmaf(o[i], f, h * x[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = sum == 0.f ? 0.f : o[i] / sum;
        const int tok = row / pr.group;
        store4<false>(a.out, ((static_cast<int64_t>(s.first) + tok) * a.qheads + head * pr.group + (row - tok * pr.group)) * D + d, a.elem, o);
    }
}

template <int KB, int VB, int NB, int W>
hipError_t run_prompt(const AttnArgs& a, const kv_plan::PromptPlan& plan, hipStream_t stream) {
    constexpr int BN = NB <= 4 ? 64 : 32;
    constexpr size_t lds = 2 * sizeof(TileLds<NB, BN>) + 16;
    if constexpr (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&kv_attn_prompt<KB, VB, NB, BN, W>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return e;
    }
    const unsigned y = static_cast<unsigned>(plan.row_tiles * plan.parts < 65535 ? plan.row_tiles * plan.parts : 65535);
    const unsigned z = a.batch < 65535 ? a.batch : 65535;
    Prompt pr{a.qheads / a.kv.heads, plan.parts, static_cast<float*>(a.work), nullptr};
    pr.stat = reinterpret_cast<float2*>(pr.part + static_cast<int64_t>(a.kv.heads) * y * z * 32 * W * 32 * NB);
    hipLaunchKernelGGL((kv_attn_prompt<KB, VB, NB, BN, W>), dim3(a.kv.heads, y, z), dim3(64 * W), lds, stream, a, pr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || plan.parts == 1) return e;
    hipLaunchKernelGGL((kv_attn_prompt_join<NB, 32 * W>), dim3(a.kv.heads, static_cast<unsigned>(plan.row_tiles * W), z), dim3(256), 0, stream, a, pr,
                       static_cast<int>(y));
    return hipGetLastError();
}

template <int KB, int VB, int NB>
hipError_t prompt_rows(const AttnArgs& a, hipStream_t stream) {
    const kv_plan::PromptPlan plan = kv_plan::prompt_plan(32 * NB, a.kv.heads, a.qheads, a.batch, a.T, a.max_q, a.max_len, a.window);
    if constexpr (NB == 2 || NB == 4) {
        if (plan.rows == 256) return run_prompt<KB, VB, NB, 8>(a, plan, stream);
    }
    return run_prompt<KB, VB, NB, 4>(a, plan, stream);
}

template <int NB>
hipError_t attn_prompt(const AttnArgs& a, hipStream_t stream) {
    if (a.kv.kbits == 4) return prompt_rows<4, 4, NB>(a, stream);
    return a.kv.vbits == 8 ? prompt_rows<8, 8, NB>(a, stream) : prompt_rows<8, 4, NB>(a, stream);
}

}  // namespace

}  // namespace qbd
