// Host-side checks of what a kv_attention call launches against the workspace
// that it was asked to bring, built with the cache's C-ABI layer (kv_api.cpp)
// under AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_kv_plan_sanitized.py, with stand-ins for the HIP runtime and the
// launchers.  The first argument names the check.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../block_quantized_decode_amd/csrc/kv.hpp"
#include "../../block_quantized_decode_amd/csrc/kv_plan.hpp"
#include "../../include/qbd.h"

namespace {
int g_calls = 0;
qbd::AttnArgs g_attn;
}  // namespace

extern "C" hipError_t hipGetDevice(int* dev) {
    *dev = 0;
    return hipSuccess;
}
extern "C" hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
    std::memset(p, 0, sizeof(*p));
    std::strncpy(p->gcnArchName, "gfx950", sizeof(p->gcnArchName) - 1);
    return hipSuccess;
}
extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

namespace qbd {
hipError_t launch_kv_write(const KvView&, const KvRows&, const KvRows&, Elem, const int64_t*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_read(const KvView&, const int64_t*, int64_t, Elem, void*, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_attention(const AttnArgs& a, hipStream_t) {
    g_attn = a;
    ++g_calls;
    return hipSuccess;
}
}  // namespace qbd

namespace {

int g_failures = 0;

template <typename T = void>
T* fake(int i) {
    return reinterpret_cast<T*>((uintptr_t{1} << 40) * static_cast<uintptr_t>(i + 1));
}

struct Shape {
    int64_t dim, heads, group, batch, T, max_q, max_len, window;
};

// One call of 16-bit rows with the workspace that its sizes ask for.
int attend(const Shape& s, int64_t& need) {
    const qbd_kv_cache c = {fake(0), fake(1), fake(2), fake(3), 64, s.heads, 64, s.dim, 4, 4};
    const int64_t qheads = s.heads * s.group;
    need = kv_attention_work_bytes(&c, s.batch, s.T, qheads, s.max_q, s.max_len);
    return kv_attention(&c, fake(4), QBD_BF16, qheads * s.dim, s.dim, fake<int32_t>(5), 64, fake<int32_t>(6), fake<int32_t>(7), s.batch, s.T,
                        qheads, s.max_q, s.max_len, 1, s.window, 0.125f, fake(8), need ? fake(9) : nullptr, need, nullptr);
}

// Bytes of the workspace that the launchers write for these arguments.
int64_t taken(const qbd::AttnArgs& a) {
    using namespace qbd::kv_plan;
    const PromptPlan p = prompt_plan(a.kv.dim, a.kv.heads, a.qheads, a.batch, a.T, a.max_q, a.max_len, a.window);
    if (p.rows) return p.parts > 1 ? p.row_tiles * p.parts * a.kv.heads * a.batch * p.rows * (a.kv.dim + 2) * 4 : 0;
    if (direct(a.kv.dim, most_keys(a.T, a.max_q, a.max_len, a.window), split_items(a.kv.heads, a.qheads, a.batch, a.T, a.max_q), a.batch)) return 0;
    return 2 * kMaxSplitGroups * (16 * kRowTiles * (a.kv.dim + 2) * 4 + 32);
}

// Whatever its window, a call fits the workspace that was asked for without it.
void check_window_workspace() {
    int in_parts = 0, bad = 0;
    for (int64_t dim : {64, 96, 128, 192, 256})
        for (int64_t heads : {1, 2, 4, 8})
            for (int64_t group : {1, 4, 7})
                for (int64_t batch : {1, 3, 16})
                    for (int64_t T : {40, 64, 100, 333, 1200, 2048})
                        for (int64_t max_q : {0, 64, 1200})
                            for (int64_t max_len : {0, 20000, 100000})
                                for (int64_t window : {int64_t{1}, int64_t{4096}, int64_t{16000}, int64_t{16384}, int64_t{17000}, int64_t{20000},
                                                       int64_t{32000}, int64_t{32768}, int64_t{65536}, int64_t{1} << 20, int64_t{1} << 40}) {
                                    const Shape s = {dim, heads, group, batch, T, max_q, max_len, window};
                                    int64_t need = 0;
                                    const int calls = g_calls, st = attend(s, need);
                                    if (st != QBD_OK || g_calls != calls + 1) {
                                        ++bad;
                                        continue;
                                    }
                                    const int64_t bytes = taken(g_attn);
                                    in_parts += bytes > 0;
                                    if (bytes > need) {
                                        if (bad++ < 5)
                                            std::fprintf(stderr, "dim %lld heads %lld group %lld batch %lld T %lld max_q %lld max_len %lld window %lld: %lld bytes of %lld\n",
                                                         (long long)dim, (long long)heads, (long long)group, (long long)batch, (long long)T, (long long)max_q,
                                                         (long long)max_len, (long long)window, (long long)bytes, (long long)need);
                                    }
                                }
    if (bad) std::fprintf(stderr, "%d calls refused or past their workspace\n", bad);
    g_failures += bad + (in_parts == 0);
}

// A row's window is found as position - window in 64 bits, for rows as far
// before the first key as a call's sizes allow.
void check_window_range() {
    for (int64_t window : {int64_t{1} << 31, int64_t{1} << 62, INT64_MAX - (int64_t{1} << 31), INT64_MAX - 1, INT64_MAX}) {
        int64_t need = 0;
        if (attend({64, 2, 4, 1, 100, 0, 5000, window}, need) != QBD_OK) ++g_failures;
        const int64_t lowest = int64_t{0} - ((int64_t{1} << 31) - (int64_t{1} << 20));
        int64_t first = 0;
        if (__builtin_sub_overflow(lowest, g_attn.window, &first)) {
            std::fprintf(stderr, "window %lld reaches the kernels as %lld\n", (long long)window, (long long)g_attn.window);
            ++g_failures;
        }
        if (g_attn.window < int64_t{1} << 31) ++g_failures;  // no position is out of it
    }
}

// The rows of one cached head (tokens times query heads of its group) are
// counted in 32 bits.
void check_row_count() {
    const int64_t most = (int64_t{1} << 31) - (int64_t{1} << 20);
    int64_t need = 0;
    for (int64_t group : {1, 2, 64})
        for (int64_t T : {most / group, most / group + 1, (int64_t{1} << 32) / group}) {
            if (T > most) continue;
            const int calls = g_calls, st = attend({64, 1, group, 1, T, 0, 5000, 0}, need);
            const bool fits = group * T <= most;
            if (fits != (st == QBD_OK) || (!fits && (st != QBD_ERR_SHAPE || g_calls != calls))) {
                std::fprintf(stderr, "group %lld T %lld: status %d\n", (long long)group, (long long)T, st);
                ++g_failures;
            }
        }
}

// Without a bound on a sequence's rows the tokens of all are shared among
// them: a batch of single tokens is not taken for prompts, prompts still are.
void check_unknown_rows() {
    using namespace qbd::kv_plan;
    auto rows = [](const Shape& s) {
        int64_t need = 0;
        if (attend(s, need) != QBD_OK) ++g_failures;
        return prompt_plan(g_attn.kv.dim, g_attn.kv.heads, g_attn.qheads, g_attn.batch, g_attn.T, g_attn.max_q, g_attn.max_len, g_attn.window).rows;
    };
    for (int64_t dim : {64, 128, 256})
        for (int64_t heads : {1, 8})
            for (int64_t group : {1, 4, 7})
                for (int64_t max_len : {0, 500, 8192, 100000}) {
                    for (int64_t batch : {1, 32, 64, 256, 4096})
                        for (int64_t each : {1, 8}) {
                            const Shape s = {dim, heads, group, batch, batch * each, 0, max_len, 0};
                            if (each * group < kPromptRows && rows(s) != 0) {
                                std::fprintf(stderr, "%lld x %lld tokens of %lld over %lld heads, max_len %lld: taken for prompts\n", (long long)batch,
                                             (long long)each, (long long)(heads * group), (long long)heads, (long long)max_len);
                                ++g_failures;
                            }
                        }
                    // the same answer as with the bound, where the sequences are alike
                    for (int64_t batch : {1, 4, 16})
                        for (int64_t each : {100, 600, 2000})
                            if ((rows({dim, heads, group, batch, batch * each, 0, max_len, 0}) > 0) !=
                                (rows({dim, heads, group, batch, batch * each, each, max_len, 0}) > 0)) {
                                std::fprintf(stderr, "%lld x %lld tokens: not what the bound gives\n", (long long)batch, (long long)each);
                                ++g_failures;
                            }
                }
}

}  // namespace

int main(int argc, char** argv) {
    const char* which = argc > 1 ? argv[1] : "";
    if (!std::strcmp(which, "window_workspace")) check_window_workspace();
    else if (!std::strcmp(which, "window_range")) check_window_range();
    else if (!std::strcmp(which, "row_count")) check_row_count();
    else if (!std::strcmp(which, "unknown_rows")) check_unknown_rows();
    else return 2;
    if (g_failures) return 1;
    std::printf("%s passed\n", which);
    return 0;
}
