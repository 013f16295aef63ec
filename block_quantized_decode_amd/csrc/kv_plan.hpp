// Host-side rules of the quantized key/value cache: accepted shapes and the
// split of the attention's work.  Plain C++, shared by the C-ABI layer, the
// kernels and the host checks.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define QBD_HD __host__ __device__
#else
#define QBD_HD
#endif

namespace qbd {
namespace kv_plan {

constexpr bool page_ok(int64_t page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }
constexpr bool dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }
constexpr bool bits_ok(int k, int v) { return (k == 4 && v == 4) || (k == 8 && v == 8) || (k == 8 && v == 4); }

// ---- split attention (kv_attn_split.hip)
//
// An item is one cached head of one sequence with up to 16 * RT of its query
// rows; its keys are walked in tiles of 32.  The grid fits the card at once,
// and its workgroups find their work from the lengths on the device, so that
// ragged batches balance without the host knowing them:
// - few items (at most half the workgroups): each in equal parts, one a
//   workgroup, about as many as there are workgroups, of kMinPart tiles and
//   more (one a wave);
// - more: all items in a row, each with kItemCost tiles of overhead before
//   its own, are cut into equal shares of at least kMinShare tiles.
// Measured, us, one query row of four heads a cached head, 8 cached heads of
// 128 elements in 4 bits, sequences x keys: parts of 1, 4, 16 tiles 14.2,
// 11.6, 14.2 (1 x 2000) and 15.5, 15.2, 14.9 (8 x 1500); a cost of 0, 8, 24
// tiles 134, 80, 83 (64 x 1 .. 8192) and 71, 25, 25 (64 x 1 .. 1024); shares
// of 4, 16, 64 tiles and more 24, 24, 39 (64 x 1000).
constexpr int kTile = 32;
constexpr int kItemCost = 8;
constexpr int kMinShare = 16;
constexpr int kMinPart = 4;

// Rows of an item: tiles of 16 that a wave keeps at once.  Two were slower
// throughout, by their registers (8 heads of 128, 4 bits, 8 x 5000 keys, one
// tile / two, as the kernel then was: 20 rows 29.7 / 31.3, 40 rows 42.7 / 47.0,
// 80 rows 57.2 / 71.6).
constexpr int kRowTiles = 1;

// Workgroups of four waves that a CU holds, by the registers of a wave: its
// sums, queries (with the second parts of fp32 rows), a tile of codes and
// scales, and what the work on them takes (found by compiling): three within 168, two
// within 256, else one.
QBD_HD constexpr int split_groups_a_cu(int kbits, int vbits, int nb, int rt) {
    const int kept = 16 * nb * rt + nb * (kbits / 2 + vbits / 2 + 8) + 90 + 25 * (rt - 1);
    return kept <= 165 ? 3 : kept <= 240 && nb <= 4 ? 2 : 1;
}
constexpr int kMaxSplitGroups = 256 * 3;

// Cost of all items over the workgroups.
QBD_HD constexpr int64_t share_of(int64_t total, int groups) {
    const int64_t s = (total + groups - 1) / groups;
    return s > kMinShare ? s : kMinShare;
}

// The tiles of an item (cost positions start + kItemCost ...) that fall in
// the share [w * share, (w + 1) * share).
struct Part {
    int begin, end;
};
QBD_HD constexpr Part part_of(int64_t start, int tiles, int64_t w, int64_t share) {
    const int64_t b = w * share - start - kItemCost, e = b + share;
    return Part{static_cast<int>(b < 0 ? 0 : b > tiles ? tiles : b), static_cast<int>(e < 0 ? 0 : e > tiles ? tiles : e)};
}

// The most tokens and, with the lengths and a window's, the most keys that a
// sequence's rows walk; 0: not known.
constexpr int64_t most_tokens(int64_t T, int64_t max_q) { return max_q > 0 && max_q < T ? max_q : T; }
constexpr int64_t most_keys(int64_t T, int64_t max_q, int64_t max_len, int64_t window) {
    const int64_t n = most_tokens(T, max_q);
    return window > 0 && (max_len == 0 || (window < max_len && n < max_len - window)) && window < INT64_MAX - n ? window + n : max_len;
}

// The most rows of one cached head in a sequence, as far as the host knows.
constexpr int64_t most_rows(int64_t group, int64_t T, int64_t max_q) {
    return group * most_tokens(T, max_q);
}

// The most items of all sequences.
constexpr double split_items(int heads, int qheads, int64_t batch, int64_t T, int64_t max_q) {
    const int64_t group = qheads / heads, rows = most_rows(group, T, max_q), tile = 16 * kRowTiles;
    const double each = static_cast<double>((rows + tile - 1) / tile) * batch, all = static_cast<double>(group * T / tile) + batch;
    return heads * (each < all ? each : all);
}

// Short sequences, and longer ones where they are many: one workgroup an item
// with no second launch.  Measured as above, so / split: 1 x 500 8.9 / 11.4,
// 64 x 500 13.7 / 17.1; 1 x 1000 12.3 / 11.4, 8 x 1000 12.8 / 14.7, 64 x
// 1 .. 1000 16.9 / 25.0; 16 x 2000 20.7 / 19.0, 32 x 2000 21.4 / 24.8, 128 x
// 1 .. 2000 39.6 / 47.2; 64 x 1 .. 4000 43.8 / 42.3.  Heads of 256 elements
// (4 cached, 8- and 4-bit): 16 x 1000 19.4 / 16.0, 64 x 1000 22.1 / 26.0.
constexpr bool direct(int dim, int64_t keys, double items, int64_t batch) {
    return keys > 0 && batch <= 65535 && (keys <= 512 || (keys <= 1024 && items >= (dim > 128 ? 256 : 64)) || (keys <= 2048 && items >= 256));
}

// ---- prompt attention (kv_attn_prompt.hpp)
//
// A workgroup takes 256 rows of a cached head (64 and 128 elements) or 128,
// and one run of their keys: eight waves that share a tile expand half as much
// a row as four (kv_attn_prompt.hpp has both sides).  Fewer workgroups than
// three quarters of what the card holds leave CUs idle: their keys are walked
// in parts.
struct PromptPlan {
    int rows;           // a workgroup; 0: the split kernel's work
    int64_t row_tiles;  // of a sequence's head, at most
    int parts;
};

// Workgroups that a CU holds (registers).
QBD_HD constexpr int prompt_groups_a_cu(int nb, int waves) {
    return waves == 4 && nb <= 3 ? 2 : 1;
}

// Which kernel: this one has a start (some 30 us at 128 elements) and wants
// full tiles of rows, the split kernel's time grows with rows x keys from the
// first.  Measured, this one / the split kernel, 4-bit codes of 128 elements,
// rows x cached heads of all sequences:
//    8192 keys    64 x 32  56 / 41    96 x 32  56 / 63    512 x 8  60 / 62    4096 x 8  171 / 404
//    2048 keys   512 x 8   37 / 21  1024 x 8   41 / 32    256 x 32 43 / 32     512 x 32  47 / 58
//     512 keys  2048 x 8   32 / 25   512 x 32  33 / 24   1024 x 32 32 / 44
//   16384 keys   256 x 8   79 / 61    96 x 32  82 / 105   512 x 8  77 / 106
// so it takes over where rows x heads x (keys + 1300) pass 40 million, and
// near that for the other sizes and codes (256 elements: 1024 x 8 over 2048
// keys 65 / 65, 512 x 8 over 8192 103 / 108; 192 elements: 1024 x 8 over 2048
// 52 / 43; 64 elements, 8-bit: 512 x 8 over 8192 38 / 42).  A length that the
// host does not know counts as 16384 keys; a window as its keys and the rows',
// but never as more than the length would without it, so that the workspace,
// whose size is asked without the window, holds whatever it chooses.
// The sequences' rows together are no more than the tokens', and without a
// bound on a sequence's their average has to be a prompt's.
constexpr int kPromptRows = 96;
constexpr double kPromptWork = 40e6;
constexpr int64_t kPromptKeys = 32768;  // longer counts as this
constexpr int kPromptPart = 512;  // keys of a part, at least

constexpr PromptPlan prompt_plan(int dim, int heads, int qheads, int64_t batch, int64_t T, int64_t max_q, int64_t max_len,
                                 int64_t window) {
    const int64_t rows = most_rows(qheads / heads, T, max_q);
    const int64_t known = most_keys(T, max_q, max_len, window), most_counted = max_len > 0 ? kPromptKeys : kPromptKeys / 2;
    const int64_t keys = known == 0 || known > most_counted ? most_counted : known;
    const double all = static_cast<double>(qheads / heads) * T, each = static_cast<double>(rows) * batch;
    if (rows < kPromptRows || (max_q == 0 && all < static_cast<double>(kPromptRows) * batch)) return PromptPlan{0, 0, 1};
    if ((each < all ? each : all) * heads * (keys + 1300) < kPromptWork) return PromptPlan{0, 0, 1};
    const int take = (dim == 64 || dim == 128) && rows > 128 ? 256 : 128;
    const int64_t tiles = (rows + take - 1) / take, fill = 256 * prompt_groups_a_cu(dim / 32, take / 32);
    const double groups = static_cast<double>(tiles) * heads * batch;
    const int64_t most = keys < 2 * kPromptPart ? 1 : keys / kPromptPart;
    int64_t parts = groups >= 3 * fill / 4 ? 1 : static_cast<int64_t>(fill / groups);
    if (parts > most) parts = most;
    return PromptPlan{take, tiles, static_cast<int>(parts)};
}

// Partial results: for each part of a prompt's rows, or for each workgroup of
// the split kernel two slots (the item that its share cuts at the start, and
// the one it cuts at the end) of 16 * RT rows: dim sums, a reference and a
// weight total a row, a note of each item.  The size is asked for without a
// window (0), under which a call never takes more: fewer keys make neither
// more parts nor a second launch.
constexpr int64_t work_bytes(int dim, int heads, int qheads, int64_t batch, int64_t T, int64_t max_q, int64_t max_len,
                             int64_t window = 0) {
    const PromptPlan plan = prompt_plan(dim, heads, qheads, batch, T, max_q, max_len, window);
    const int64_t prompt = plan.parts > 1 ? plan.row_tiles * plan.parts * heads * batch * plan.rows * (dim + 2) * 4 : 0;
    const int64_t rows = 16 * kRowTiles;
    const bool once = direct(dim, most_keys(T, max_q, max_len, window), split_items(heads, qheads, batch, T, max_q), batch);
    const int64_t split = once ? 0 : 2 * kMaxSplitGroups * (rows * (dim + 2) * 4 + 32);
    return prompt > split ? prompt : split;
}

}  // namespace kv_plan
}  // namespace qbd
