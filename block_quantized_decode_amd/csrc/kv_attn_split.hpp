// Attention over the quantized key/value cache for few query rows a cached
// head (single tokens, drafted blocks): the keys of a sequence are split
// over waves and workgroups, and the parts joined.
//
// For query row q and the keys t it sees, with c = scale * log2(e),
//   out = sum_t 2^(c q.k_t - R) v_t / sum_t 2^(c q.k_t - R),
// any R; partial sums over disjoint keys with their own R add after a
// factor 2^(R_i - R).
//
// A wave walks tiles of 32 keys for 16 rows (RT times; once is fastest,
// kv_plan.hpp), all in registers:
//   S^T = K Q^T   A = K codes (16 keys x 32 elements of a block), B = q
//   O^T = V^T W   A = V codes (16 elements x 32 keys), B = the weights
// on v_mfma_f32_16x16x32_f16.  The codes, integers of at most 127, are exact
// in binary16, so the block scales stay outside: a K scale multiplies the
// fp32 dot of its block, a V scale the weight of its key (once per block).
// In the 16 x 16 result a lane holds one row (lane % 16) and four keys
// 4 (lane / 16) + r of each half tile; with key 8 (m / 4) + 4 half + m % 4
// at row m of the half's A operand, a lane group's eight scores are the
// eight consecutive keys 8 (lane / 16) .. + 7, which are its K slots of the
// second product: the weights never leave their lane.  The cache stores V
// by eight keys so that this operand is one load as well.
//
// Roundings: q is scaled by a power of two (kQueryTop) and rounded to
// binary16, exact for bf16 and f16 elements down to 2^-28 of the row's
// largest; f32 rows add a second binary16 for the remainder (22 bits, down to
// 2^-17).  A weight times its V scale is rounded to binary16 (11 bits: as
// coarse as an f16 output, whose error is a third above one rounding alone);
// for f32 outputs it enters exactly, as three bf16 parts of 8 bits, so that a
// sum keeps its precision however far its weights lie below the largest.
// With binary16 the reference R of a row counts the largest V scale in, so
// that these products use the type's range whatever the size of the values.
// R only moves when a tile passes it by 2^(kTop - kLift), so most tiles
// rescale nothing.
//
// Bound by memory over long histories: 131001 keys of 8 heads of 128 in 4 bits
// (151 MB) take 40.7 us with the join; by the slope over the length (65536 to
// 262144 keys, cold) it reads 4.8 to 5.2 TB/s, where a plain read reaches 6.0,
// on a fixed 13 us (the start of a workgroup: lengths, table, queries, first
// tile; the join's launch).  64 sequences of up to 8192 keys (73 MB) take 30
// us, 24 with a window of 2048 and heads of 256 (82 MB) 28.1 us.  fp32 rows
// are bound by the vector work of their exact splits: four prompts of up to
// 997 tokens, 14 over 2 heads of 64, 52.2 us.  A sequence's items all walk the
// same keys: those after a causal row tile's last row or before its first row's
// window are computed and masked, about half of the tiles of such prompts.
#pragma once

#include <type_traits>

#include "kv_attn.hpp"

namespace qbd {
namespace {

// A sequence's keys in tiles, and its items.
struct Work : Seq {
    int begin;   // first key of its first tile
    int tiles;
    int items;   // row tiles * cached heads
};

__device__ __forceinline__ Work uniform(const Work& s) {
    Work r;
    static_cast<Seq&>(r) = uniform(static_cast<const Seq&>(s));
    r.begin = uniform(s.begin);
    r.tiles = uniform(s.tiles);
    r.items = uniform(s.items);
    return r;
}

struct Split {
    int group;     // query heads a cached head
    int direct;    // one workgroup an item
    int groups;    // workgroups that share the items otherwise
    float* part;   // [2 * groups][rows][dim]
    float2* stat;  // [2 * groups][rows]: reference, weight total
    struct Cut* cut;  // [2 * groups]
};

// An item that shares' ends cut, as each of its workgroups notes it: parts
// w0 .. w1 hold its sums, the first in slot 2 w0 + 1, the others in 2 w.
struct Cut {
    int w0, w1;  // w0 < 0: no item
    int first;   // the sequence's first query row
    int row0, rows, head;
    int pad[2];
};

template <int RT>
__device__ __forceinline__ Work sequence(const AttnArgs& a, const Split& sp, int b) {
    Work s;
    static_cast<Seq&>(s) = sequence_of(a, b);
    // the keys that the first row sees begin here
    const int64_t lo = a.window > 0 ? static_cast<int64_t>(s.len) - s.n + 1 - a.window : 0;
    s.begin = static_cast<int>(max<int64_t>(lo, 0)) & ~(kv_plan::kTile - 1);
    s.tiles = s.len > s.begin ? (s.len - s.begin + kv_plan::kTile - 1) / kv_plan::kTile : 0;
    s.items = static_cast<int>((static_cast<int64_t>(s.n) * sp.group + 16 * RT - 1) / (16 * RT)) * a.kv.heads;
    return s;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(v), lane))) |
                                static_cast<uint64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(v >> 32), lane))) << 32);
}

__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
        const int64_t o = shfl64(v, lane >= k ? lane - k : lane);
        if (lane >= k) v += o;
    }
    return v;
}

template <int RT>
__device__ __forceinline__ int64_t cost_of(const AttnArgs& a, const Split& sp, int b) {
    const Work s = sequence<RT>(a, sp, b);
    return static_cast<int64_t>(s.items) * (s.tiles + kv_plan::kItemCost);
}

// Cost of all items, and of those before sequence `want`.  Every wave does
// this for itself, 64 sequences at a time.
template <int RT>
__device__ __forceinline__ int64_t total_cost(const AttnArgs& a, const Split& sp, int lane) {
    int64_t sum = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) sum += b0 + lane < a.batch ? cost_of<RT>(a, sp, b0 + lane) : 0;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) sum += shfl64(sum, lane ^ k);
    return sum;
}

// The few-items split: every item in equal parts of at most `most` tiles, a
// workgroup each.
struct Parts {
    int most;    // tiles a part; 0: too many items for it
    int before;  // parts of the sequences before the one found
};

__device__ __forceinline__ int parts_of(const Work& s, int most) { return s.tiles > most ? (s.tiles + most - 1) / most : 1; }

template <int RT>
__device__ __forceinline__ Parts plan_parts(const AttnArgs& a, const Split& sp, int lane) {
    float sum[2] = {0.f, 0.f};  // tiles and items
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        if (b0 + lane < a.batch) {
            const Work s = sequence<RT>(a, sp, b0 + lane);
            sum[0] += static_cast<float>(s.items) * static_cast<float>(s.tiles);
            sum[1] += static_cast<float>(s.items);
        }
    }
    wave_reduce<2>(sum);
    const float tiles = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum[0]), reduced_lane<2>(0)));
    const float items = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum[0]), reduced_lane<2>(1)));
    Parts p{0, 0};
    if (2.f * items > static_cast<float>(sp.groups)) return p;
    // the shortest of a few part lengths whose parts do not outnumber the
    // workgroups: the even share, 1/8 and 3/8 more, and one that always fits
    const float groups = static_cast<float>(sp.groups), even = tiles * 1.00001f / groups;
    const int most[3] = {max(kv_plan::kMinPart, static_cast<int>(even) + 1), max(kv_plan::kMinPart, static_cast<int>(even * 1.125f) + 1),
                         max(kv_plan::kMinPart, static_cast<int>(even * 1.375f) + 1)};
    float count[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        if (b0 + lane < a.batch) {
            const Work s = sequence<RT>(a, sp, b0 + lane);
#pragma unroll
            for (int i = 0; i < 3; ++i) count[i] += static_cast<float>(s.items) * static_cast<float>(parts_of(s, most[i]));
        }
    }
    wave_reduce<4>(count);
    p.most = max(kv_plan::kMinPart, static_cast<int>(tiles * 1.00001f / (groups - items)) + 1);
#pragma unroll
    for (int i = 2; i >= 0; --i) {
        const float n = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(count[0]), reduced_lane<4>(i)));
        if (n <= groups) p.most = min(p.most, most[i]);
    }
    return p;
}

// The sequence that holds part w, or -1.
template <int RT>
__device__ __forceinline__ int find_part(const AttnArgs& a, const Split& sp, int lane, int w, Parts& p) {
    p.before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        int v = 0;
        if (b0 + lane < a.batch) {
            const Work s = sequence<RT>(a, sp, b0 + lane);
            v = s.items * parts_of(s, p.most);
        }
        int inc = v;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            const int o = __shfl_up(inc, k);
            inc += lane >= k ? o : 0;
        }
        const uint64_t past = __ballot(p.before + inc <= w);
        if (past != ~uint64_t{0}) {
            const int k = __builtin_ctzll(~past);
            p.before += __builtin_amdgcn_readlane(inc - v, k);
            return b0 + k;
        }
        p.before += __builtin_amdgcn_readlane(inc, 63);
    }
    return -1;
}

// The sequence that holds cost position `at` (below the total), and the
// cost before it.
template <int RT>
__device__ __forceinline__ int find_sequence(const AttnArgs& a, const Split& sp, int lane, int64_t at, int64_t& before) {
    before = 0;
    for (int b0 = 0;; b0 += 64) {
        const int64_t v = b0 + lane < a.batch ? cost_of<RT>(a, sp, b0 + lane) : 0;
        const int64_t inc = wave_scan(v, lane) + before;
        const uint64_t past = __ballot(inc <= at);
        if (past != ~uint64_t{0}) {
            const int k = __builtin_ctzll(~past);
            before = shfl64(inc - v, k);
            return b0 + k;
        }
        before = shfl64(inc, 63);
    }
}



// A lane's part of a query row in operand order, scaled (kQueryTop).  The
// codes that it meets are the exact ones: entered with
// an offset (fewer instructions) they make a block's dot the difference of two
// larger sums, whose fp32 roundings were up to some hundred times the dot's own
// where a block's codes are small (an outlier beside them, queries with a mean).
template <int KB, int NB, bool SPLIT>
struct Query {
    static constexpr int kRun1 = KB == 4 ? 16 : 4;  // a slot's eight elements are two runs of four
    Run4<SPLIT> raw[NB][2];
    h8 hi[NB];
    h8 lo[SPLIT ? NB : 1];
    float c;  // a score in units of log2
    __device__ __forceinline__ void fetch(const AttnArgs& a, int64_t at, int g) {
        const int first = KB == 4 ? 4 * g : 8 * g;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            raw[b][0].load(a.q.p, at + 32 * b + first);
            raw[b][1].load(a.q.p, at + 32 * b + first + kRun1);
        }
    }
    __device__ __forceinline__ void ready(const AttnArgs& a) {
        float top = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(raw[b][i / 4].at(i % 4, a.elem)));
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const int e = __builtin_amdgcn_frexp_expf(top) - kQueryTop;
        const float sign = a.scale < 0.f ? -1.f : 1.f;
        c = ldexpf(fabsf(a.scale) * 1.44269504088896340736f, e);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = sign * ldexpf(raw[b][j / 4].at(KB == 4 ? j % 2 * 2 + j % 4 / 2 : j % 4, a.elem), -e);
                hi[b][j] = static_cast<_Float16>(y);
                if constexpr (SPLIT) lo[b][j] = static_cast<_Float16>(y - static_cast<float>(hi[b][j]));
            }
        }
    }
};

// p0 times half H of d0 and p1 times half H of d1, rounded to binary16 (the
// sum with zero lets the compiler take one mixed-precision instruction each).
template <int H>
__device__ __forceinline__ h2 weigh_pair(float p0, float p1, uint32_t d0, uint32_t d1) {
    return h2{static_cast<_Float16>(__builtin_fmaf(p0, static_cast<float>(as_h2(d0)[H]), 0.f)),
              static_cast<_Float16>(__builtin_fmaf(p1, static_cast<float>(as_h2(d1)[H]), 0.f))};
}

template <int KB, int VB, int NB, int RT, bool SPLIT>
__global__ __launch_bounds__(256, kv_plan::split_groups_a_cu(KB, VB, NB, RT)) void kv_attn_split(AttnArgs a, Split sp) {
    constexpr int D = 32 * NB, ROWS = 16 * RT, LDW = D + 4;
    __shared__ float acc_s[4][ROWS][LDW];
    __shared__ float2 stat_s[4][ROWS];
    const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x >> 6));
    const int64_t w = blockIdx.x;
    constexpr int krow = D * KB / 8, vrow = D * VB / 8;
    const uint32_t magic = pair1024();

    // this workgroup's place in the row of items
    Work s;
    int b = 0, item = 0;
    Parts parts{0, 0};
    kv_plan::Part run{0, 0};
    int cut0 = 0, cut1 = 0;                  // workgroups of the item's parts
    int64_t share = 0, start = 0, stop = 0;  // cost positions: of the item, of the share's end
    if (sp.direct) {
        b = blockIdx.y;
        s = uniform(sequence<RT>(a, sp, b));
        item = blockIdx.x;
    } else {
        if (threadIdx.x == 0) sp.cut[2 * w].w0 = sp.cut[2 * w + 1].w0 = -1;
        parts = plan_parts<RT>(a, sp, lane);
        if (parts.most > 0) {
            b = find_part<RT>(a, sp, lane, static_cast<int>(w), parts);
            if (b < 0) return;
            s = uniform(sequence<RT>(a, sp, b));
            const int count = parts_of(s, parts.most), at = static_cast<int>(w) - parts.before;
            item = uniform(at / count);
            const int i = at - item * count;
            cut0 = static_cast<int>(w) - i;
            cut1 = cut0 + count - 1;
            run.begin = uniform(static_cast<int>(static_cast<int64_t>(s.tiles) * i / count));
            run.end = uniform(static_cast<int>(static_cast<int64_t>(s.tiles) * (i + 1) / count));
        } else {
            const int64_t total = uniform(total_cost<RT>(a, sp, lane));
            share = kv_plan::share_of(total, sp.groups);
            const int64_t at = w * share;
            if (at >= total) return;
            stop = min(at + share, total);
            int64_t before;
            b = uniform(find_sequence<RT>(a, sp, lane, at, before));
            before = uniform(before);
            s = uniform(sequence<RT>(a, sp, b));
            const int64_t off = at - before;
            const int cost = s.tiles + kv_plan::kItemCost;
            item = uniform(off >> 32 ? static_cast<int>(off / cost) : static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(cost)));
            start = before + static_cast<int64_t>(item) * cost;
        }
    }

    for (;;) {
        // the next segment: an item and a run of its tiles
        bool own = true;  // the item starts here
        if (sp.direct) {
            if (item >= s.items) break;
            run = {0, s.tiles};
        } else if (parts.most == 0) {
            if (start >= stop) break;
            while (item >= s.items) {  // sequences without rows have no items
                s = uniform(sequence<RT>(a, sp, ++b));
                item = 0;
            }
            run = kv_plan::part_of(start, s.tiles, w, share);
            own = start >= w * share;
            cut0 = static_cast<int>((start + kv_plan::kItemCost) / share);
            cut1 = static_cast<int>((start + kv_plan::kItemCost + s.tiles - 1) / share);
        }
        const bool whole = run.begin == 0 && run.end == s.tiles;
        if (run.end > run.begin || (own && s.tiles == 0)) {
            const int m = fresh(lane) & 15, g = fresh(lane) >> 4;
            const int head = uniform(item % a.kv.heads);
            const int row0 = uniform(item / a.kv.heads * ROWS);
            const int rows = min(ROWS, s.n * sp.group - row0);

            const int32_t* table = a.table + b * a.table_width;
            const int shift = a.kv.page_shift, mask = (1 << shift) - 1;
            // page numbers of the wave's next 64 tiles, one tile a lane
            int ids[2];
            auto fetch_ids = [&](int tile) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t t = s.begin + (static_cast<int64_t>(tile) + 4 * lane) * 32 + 16 * h;
                    ids[h] = t < s.len && tile + 4 * lane < run.end ? table[t >> shift] : -1;
                }
            };
            int tile = run.begin + wave, slot = 0;
            if (tile < run.end) fetch_ids(tile);

            Query<KB, NB, SPLIT> q[RT];
            float ref[RT], sum[RT];
            f4 acc[RT][NB][2];
            int lo_r[RT], hi_r[RT];  // keys that the lane's row sees
            bool far = false;        // a reference of the wave is
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = row0 + min(16 * r + m, rows - 1);
                const int tok = row / sp.group;
                q[r].fetch(a, (s.first + tok) * a.q.token_stride + (head * sp.group + row - tok * sp.group) * a.q.head_stride, g);
                const int64_t pos = static_cast<int64_t>(s.len) - s.n + tok;
                hi_r[r] = a.causal ? static_cast<int>(pos + 1) : s.len;
                lo_r[r] = a.window > 0 ? static_cast<int>(max<int64_t>(pos - a.window + 1, 0)) : 0;
                ref[r] = kNoKey;
                sum[r] = 0.f;
#pragma unroll
                for (int x = 0; x < NB; ++x) acc[r][x][0] = acc[r][x][1] = f4{0.f, 0.f, 0.f, 0.f};
            }
            // a tile with its last key below hi_all and its first at or
            // above lo_all needs no mask
            const int first_tok = row0 / sp.group, last_tok = (row0 + rows - 1) / sp.group;
            const int hi_all = a.causal ? s.len - s.n + first_tok + 1 : s.len;
            const int lo_all = a.window > 0 ? static_cast<int>(max<int64_t>(static_cast<int64_t>(s.len) - s.n + last_tok - a.window + 1, 0)) : 0;

            // where a tile's two halves lie in the planes (in tokens of a
            // head), and which of them are held
            struct Place {
                int64_t at[2];
                int held;
            };
            auto place = [&](int tile, int slot) {
                Place pl;
                pl.held = 0;
                const int t = s.begin + 32 * tile;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int id = __builtin_amdgcn_readlane(ids[h], slot);
                    const bool ok = static_cast<uint32_t>(id) < static_cast<uint64_t>(a.kv.pages);
                    pl.held |= ok << h;
                    id = ok ? id : 0;
                    pl.at[h] = ((static_cast<int64_t>(id) * a.kv.heads + head) << shift) + ((t + 16 * h) & mask);
                }
                return pl;
            };
            KCodes<KB, NB> k[2];
            VCodes<VB, NB> v;
            Scales<NB> kd, vd;
            auto load_k = [&](const Place& pl) {
                const uint8_t* p0 = a.kv.kc + pl.at[0] * krow;
                const uint8_t* p1 = a.kv.kc + pl.at[1] * krow;
                const uint8_t* p = (m < 8 ? p0 : p1) + ((8 * (m / 4 & 1) + (m & 3)) * krow + g * (krow / 4));
                k[0].load(p);
                k[1].load(p + 4 * krow);
                const uint16_t* d0 = a.kv.kd + pl.at[0] * NB;
                const uint16_t* d1 = a.kv.kd + pl.at[1] * NB;
                kd.load((g < 2 ? d0 : d1) + 8 * NB * (g & 1));
            };
            auto load_v = [&](const Place& pl) {
                const uint16_t* d0 = a.kv.vd + pl.at[0] * NB;
                const uint16_t* d1 = a.kv.vd + pl.at[1] * NB;
                vd.load((g < 2 ? d0 : d1) + 8 * NB * (g & 1));
                const uint8_t* p0 = a.kv.vc + pl.at[0] * vrow;
                const uint8_t* p1 = a.kv.vc + pl.at[1] * vrow;
                v.load((g < 2 ? p0 : p1) + (8 * vrow * (g & 1) + m * (vrow / 2)));
            };
            // one tile; with MORE the next one's K is under way from the end
            // of this one's scores, its V from the end of this one's sums
            auto use_tile = [&](auto more, const Place& here, const Place& next) {
                constexpr bool MORE = decltype(more)::value;
                const int t0 = s.begin + 32 * tile;
                const bool masked = here.held != 3 || t0 + 32 > hi_all || t0 < lo_all;
                const int tg = t0 + 8 * g;
                const bool mine = here.held >> (g >> 1) & 1;
                float sc[RT][8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int y = 0; y < NB; ++y) {
                        const h8 kop = k[h].operand(y, magic);
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            f4 d = {0.f, 0.f, 0.f, 0.f};
                            if constexpr (SPLIT) d = mfma(kop, q[r].lo[y], d);
                            d = mfma(kop, q[r].hi[y], d);
#pragma unroll
                            for (int j = 0; j < 4; ++j) sc[r][4 * h + j] = fmaf(kd.at(y, 4 * h + j), d[j], y == 0 ? 0.f : sc[r][4 * h + j]);
                        }
                    }
                }
                if constexpr (MORE) load_k(next);
                uint32_t seen[RT];
                if (masked) {
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        seen[r] = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const bool see = mine && tg + j < min(hi_r[r], s.len) && tg + j >= lo_r[r];
                            seen[r] |= static_cast<uint32_t>(see) << j;
                            sc[r][j] = see ? sc[r][j] : -INFINITY;
                        }
                    }
                    if constexpr (!SPLIT) {  // scales of keys that the lane's rows do not see may hold anything
                        uint32_t any = 0;
#pragma unroll
                        for (int r = 0; r < RT; ++r) any |= seen[r];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t keep = any >> (2 * j) & 1 ? 0xffffu : 0u;
                            keep |= any >> (2 * j + 1) & 1 ? 0xffff0000u : 0u;
#pragma unroll
                            for (int y = 0; y < NB; ++y) vd.w[4 * y + j] &= keep;
                        }
                    }
                }
                float lb = 0.f;  // largest V scale of the lane's keys, in log2
                if constexpr (!SPLIT) {
                    h2 big = as_h2(vd.w[0]);
#pragma unroll
                    for (int j = 1; j < 4 * NB; ++j) big = __builtin_elementwise_max(big, as_h2(vd.w[j]));
                    lb = static_cast<float>(__builtin_amdgcn_frexp_expf(fmaxf(static_cast<float>(big[0]), static_cast<float>(big[1]))));
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float top = sc[r][0];
#pragma unroll
                    for (int j = 1; j < 8; ++j) top = fmaxf(top, sc[r][j]);
                    const float mark = fmaf(top, q[r].c, lb);
                    float by = q[r].c, less = ref[r];
                    if (__any(mark > ref[r] + kTop) || far) {
                        float best = fmaxf(mark, __shfl_xor(mark, 16)), score = top * q[r].c;
                        best = fmaxf(best, __shfl_xor(best, 32)) - kLift;
                        score = fmaxf(score, __shfl_xor(score, 16));
                        score = fmaxf(score, __shfl_xor(score, 32));
                        best = fmaxf(ref[r], is_far(score) ? score : best);
                        const float f = __builtin_amdgcn_exp2f(ref[r] - best);
                        ref[r] = less = best;
                        sum[r] *= f;
#pragma unroll
                        for (int y = 0; y < NB; ++y) {
                            acc[r][y][0] *= f;
                            acc[r][y][1] *= f;
                        }
                        far |= __any(is_far(best));
                        if (far) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) sc[r][j] = sc[r][j] * by - less;
                            by = 1.f;
                            less = 0.f;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) sc[r][j] = __builtin_amdgcn_exp2f(fmaf(sc[r][j], by, -less));
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) sc[r][j] = seen[r] >> j & 1 ? sc[r][j] : 0.f;
                    }
                    sum[r] += ((sc[r][0] + sc[r][1]) + (sc[r][2] + sc[r][3])) + ((sc[r][4] + sc[r][5]) + (sc[r][6] + sc[r][7]));
                }
#pragma unroll
                for (int y = 0; y < NB; ++y) {
                    if constexpr (SPLIT) {
                        const u4 v0 = v.operand_bf16(y, 0), v1 = v.operand_bf16(y, 1);
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            float x[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = sc[r][j] * vd.at(y, j);
                            if (masked) {  // a NaN scale of a key that another row sees
#pragma unroll
                                for (int j = 0; j < 8; ++j) x[j] = seen[r] >> j & 1 ? x[j] : 0.f;
                            }
                            u4 part[3];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) part[z][j] = cut8(x[2 * j], x[2 * j + 1]);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) part[2][j] = uppers(__float_as_uint(x[2 * j]), __float_as_uint(x[2 * j + 1]));
#pragma unroll
                            for (int z = 2; z >= 0; --z) {
                                acc[r][y][0] = mfma(v0, part[z], acc[r][y][0]);
                                acc[r][y][1] = mfma(v1, part[z], acc[r][y][1]);
                            }
                        }
                    } else {
                        const h8 v0 = v.operand(y, 0, magic), v1 = v.operand(y, 1, magic);
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const uint32_t* dv = vd.w + 4 * y;
                            const float* p = sc[r];
                            h8 x = as_h8(weigh_pair<0>(p[0], p[2], dv[0], dv[1]), weigh_pair<1>(p[1], p[3], dv[0], dv[1]),
                                         weigh_pair<0>(p[4], p[6], dv[2], dv[3]), weigh_pair<1>(p[5], p[7], dv[2], dv[3]));
                            if (RT > 1 && masked) {  // a NaN scale of a key that another of the lane's rows sees
                                constexpr int order[8] = {0, 2, 1, 3, 4, 6, 5, 7};
#pragma unroll
                                for (int j = 0; j < 8; ++j) x[j] = seen[r] >> order[j] & 1 ? x[j] : 0.f16;
                            }
                            acc[r][y][0] = mfma(v0, x, acc[r][y][0]);
                            acc[r][y][1] = mfma(v1, x, acc[r][y][1]);
                        }
                    }
                }
                if constexpr (MORE) load_v(next);
            };
            if (tile < run.end) {
                Place here = place(tile, 0);
                load_k(here);
                load_v(here);
#pragma unroll
                for (int r = 0; r < RT; ++r) q[r].ready(a);
                while (tile + 4 < run.end) {
                    if (++slot == 64) {
                        fetch_ids(tile + 4);
                        // waited for here, so that no other tile's loads are
                        ids[0] = fresh(ids[0]);
                        ids[1] = fresh(ids[1]);
                        slot = 0;
                    }
                    const Place next = place(tile + 4, slot);
                    use_tile(std::true_type{}, here, next);
                    here = next;
                    tile += 4;
                }
                use_tile(std::false_type{}, here, here);
            }

            // join the four waves
            __syncthreads();  // the last segment's reads of LDS are done
            const int tid = fresh(threadIdx.x);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                sum[r] += __shfl_xor(sum[r], 16);
                sum[r] += __shfl_xor(sum[r], 32);
                if constexpr (SPLIT && VB == 4) sum[r] *= 16.f;  // as the bf16 codes are
                if (g == 0) stat_s[wave][16 * r + m] = make_float2(ref[r], sum[r]);
#pragma unroll
                for (int z = 0; z < NB; ++z) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) *reinterpret_cast<f4*>(&acc_s[wave][16 * r + m][32 * z + 16 * h + 4 * g]) = acc[r][z][h];
                }
            }
            __syncthreads();
            for (int e = tid; e < rows * (D / 4); e += 256) {
                const int row = e / (D / 4), d = e % (D / 4) * 4;
                float2 st[4];
                float best = kNoKey;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    st[k] = stat_s[k][row];
                    best = fmaxf(best, st[k].x);
                }
                float total = 0.f;
                f4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f = __builtin_amdgcn_exp2f(st[k].x - best);
                    total = fmaf(f, st[k].y, total);
                    const f4 z = *reinterpret_cast<const f4*>(&acc_s[k][row][d]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = fmaf(f, z[i], o[i]);
                }
                if (whole) {
                    const int r = row0 + row, tok = r / sp.group;
                    const int64_t at = ((static_cast<int64_t>(s.first) + tok) * a.qheads + head * sp.group + (r - tok * sp.group)) * D + d;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = total == 0.f ? 0.f : o[i] / total;
                    store4<SPLIT>(a.out, at, a.elem, o);
                } else {
                    const int64_t slot_at = (2 * w + (run.begin == 0)) * ROWS + row;
                    *reinterpret_cast<f4*>(sp.part + slot_at * D + d) = o;
                    if (d == 0) sp.stat[slot_at] = make_float2(best, total);
                }
            }
            if (!whole && threadIdx.x == 0) sp.cut[2 * w + (run.begin == 0)] = Cut{cut0, cut1, s.first, row0, rows, head, {0, 0}};
        }
        if (parts.most > 0) break;
        if (sp.direct) {
            item += gridDim.x;
        } else {
            start += s.tiles + kv_plan::kItemCost;
            ++item;
        }
    }
}

// Joins the parts of the items that shares' ends cut.  Every workgroup that
// noted such an item takes an equal piece of its elements; a thread sums four
// elements over a part of the parts.
template <int NB, int RT>
__global__ __launch_bounds__(256) void kv_attn_join(AttnArgs a, Split sp) {
    constexpr int D = 32 * NB, ROWS = 16 * RT, LANES = D / 4;
    const int w = blockIdx.x;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const Cut cut = sp.cut[2 * w + z];
        if (cut.w0 < 0) continue;
        const int parts = cut.w1 - cut.w0 + 1, all = cut.rows * LANES;
        const int lo = static_cast<int>(static_cast<int64_t>(all) * (w - cut.w0) / parts);
        const int n = static_cast<int>(static_cast<int64_t>(all) * (w - cut.w0 + 1) / parts) - lo;
        int ways = 1;  // threads on one place
        while (ways < 64 && ways < parts && 2 * ways * n <= 256) ways *= 2;
        const int way = threadIdx.x & (ways - 1);
        for (int e0 = 0; e0 < n; e0 += 256 / ways) {
            const int e = lo + min(e0 + static_cast<int>(threadIdx.x) / ways, n - 1);
            const int row = e / LANES, d = e % LANES * 4;
            float best = kNoKey, sum = 0.f;
            f4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int p = way; p < parts; p += ways) {
                const int64_t at = static_cast<int64_t>(2 * (cut.w0 + p) + (p == 0)) * ROWS + row;
                const float2 st = sp.stat[at];
                const f4 x = *reinterpret_cast<const f4*>(sp.part + at * D + d);
                const float top = fmaxf(best, st.x);
                const float f = __builtin_amdgcn_exp2f(best - top), h = __builtin_amdgcn_exp2f(st.x - top);
                best = top;
                sum = fmaf(sum, f, h * st.y);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fmaf(o[i], f, h * x[i]);
            }
            for (int k = 1; k < ways; k *= 2) {
                const float other = __shfl_xor(best, k);
                const float top = fmaxf(best, other);
                const float f = __builtin_amdgcn_exp2f(best - top), h = __builtin_amdgcn_exp2f(other - top);
                best = top;
                sum = fmaf(sum, f, h * __shfl_xor(sum, k));
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fmaf(o[i], f, h * __shfl_xor(o[i], k));
            }
            if (way == 0 && e0 + static_cast<int>(threadIdx.x) / ways < n) {
                const int r = cut.row0 + row, tok = r / sp.group;
                const int64_t at = ((static_cast<int64_t>(cut.first) + tok) * a.qheads + cut.head * sp.group + (r - tok * sp.group)) * D + d;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = sum == 0.f ? 0.f : o[i] / sum;
                if (a.elem == Elem::F32) store4<true>(a.out, at, a.elem, o);
                else store4<false>(a.out, at, a.elem, o);
            }
        }
    }
}

template <int KB, int VB, int NB, int RT, bool SPLIT>
hipError_t run(const AttnArgs& a, hipStream_t stream) {
    Split sp{};
    sp.group = a.qheads / a.kv.heads;
    const int64_t rows = kv_plan::most_rows(sp.group, a.T, a.max_q);
    const int64_t tiles = (rows + 16 * RT - 1) / (16 * RT);
    sp.direct = kv_plan::direct(32 * NB, kv_plan::most_keys(a.T, a.max_q, a.max_len, a.window),
                               kv_plan::split_items(a.kv.heads, a.qheads, a.batch, a.T, a.max_q), a.batch);
    if (sp.direct) {
        const int64_t items = tiles * a.kv.heads;
        hipLaunchKernelGGL((kv_attn_split<KB, VB, NB, RT, SPLIT>), dim3(static_cast<unsigned>(items < 65535 ? items : 65535), a.batch), dim3(256), 0,
                           stream, a, sp);
        return hipGetLastError();
    }
    sp.groups = 256 * kv_plan::split_groups_a_cu(KB, VB, NB, RT);
    sp.part = static_cast<float*>(a.work);
    sp.stat = reinterpret_cast<float2*>(sp.part + int64_t{2} * sp.groups * 16 * RT * 32 * NB);
    sp.cut = reinterpret_cast<Cut*>(sp.stat + int64_t{2} * sp.groups * 16 * RT);
    hipLaunchKernelGGL((kv_attn_split<KB, VB, NB, RT, SPLIT>), dim3(sp.groups), dim3(256), 0, stream, a, sp);
    hipLaunchKernelGGL((kv_attn_join<NB, RT>), dim3(sp.groups), dim3(256), 0, stream, a, sp);
    return hipGetLastError();
}

template <int NB, bool SPLIT>
hipError_t by_bits(const AttnArgs& a, hipStream_t stream) {
    if (a.kv.kbits == 4) return run<4, 4, NB, kv_plan::kRowTiles, SPLIT>(a, stream);
    return a.kv.vbits == 8 ? run<8, 8, NB, kv_plan::kRowTiles, SPLIT>(a, stream) : run<8, 4, NB, kv_plan::kRowTiles, SPLIT>(a, stream);
}

template <int NB>
hipError_t attn_split(const AttnArgs& a, hipStream_t stream) {
    return a.elem == Elem::F32 ? by_bits<NB, true>(a, stream) : by_bits<NB, false>(a, stream);
}

}  // namespace

}  // namespace qbd
