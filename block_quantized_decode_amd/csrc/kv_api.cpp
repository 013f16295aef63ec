// C ABI of the quantized key/value cache: host-side validation, then the
// launchers.  Every check runs before the first HIP call.
#include <cmath>
#include <cstdint>

#include "../../include/qbd.h"
#include "check.hpp"
#include "kv.hpp"
#include "kv_plan.hpp"

namespace {

using qbd::check::aligned;
using qbd::check::check_device;
using qbd::check::kMaxDim;
using qbd::check::kMaxPlane;
using qbd::check::launched;
using qbd::check::overlaps;
using qbd::check::Span;

struct Planes {
    Span s[4];  // kc, kd, vc, vd
};

// The cache's shape; fills the kernels' view and the planes' spans.
int check_cache(const qbd_kv_cache* c, qbd::KvView& kv, Planes& pl) {
    if (!c) return QBD_ERR_NULL;
    if (c->pages < 0 || c->heads <= 0 || c->pages > kMaxDim || c->heads > 65535) return QBD_ERR_SHAPE;
    if (!qbd::kv_plan::page_ok(c->page) || !qbd::kv_plan::dim_ok(c->dim)) return QBD_ERR_SHAPE;
    if (!qbd::kv_plan::bits_ok(c->kbits, c->vbits)) return QBD_ERR_SHAPE;
    const int64_t rows = c->heads * c->page;  // below 2^26
    if (c->pages > 0 && rows * c->dim > kMaxPlane / c->pages) return QBD_ERR_SHAPE;
    if (c->pages > 0) {
        if (!c->kc || !c->kd || !c->vc || !c->vd) return QBD_ERR_NULL;
        if (!aligned(c->kc, 16) || !aligned(c->kd, 16) || !aligned(c->vc, 16) || !aligned(c->vd, 16)) return QBD_ERR_ALIGN;
    }
    const int64_t tokens = rows * c->pages;
    pl.s[0] = {c->kc, tokens * c->dim * c->kbits / 8};
    pl.s[1] = {c->kd, tokens * (c->dim / 32) * 2};
    pl.s[2] = {c->vc, tokens * c->dim * c->vbits / 8};
    pl.s[3] = {c->vd, tokens * (c->dim / 32) * 2};
    int shift = 0;
    while ((int64_t{1} << shift) < c->page) ++shift;
    kv = qbd::KvView{static_cast<uint8_t*>(c->kc), static_cast<uint16_t*>(c->kd), static_cast<uint8_t*>(c->vc),
                     static_cast<uint16_t*>(c->vd), c->pages, static_cast<int>(c->heads), shift,
                     static_cast<int>(c->dim), c->kbits, c->vbits};
    return QBD_OK;
}

bool elem_ok(int dtype) { return dtype == QBD_F32 || dtype == QBD_BF16 || dtype == QBD_F16; }

// T strided rows of `heads` heads: strides of 0 or more, in 16-byte steps.
int check_rows(int64_t T, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride, int64_t eb) {
    if (token_stride < 0 || head_stride < 0 || token_stride > kMaxPlane / 4 || head_stride > kMaxPlane / 4) return QBD_ERR_SHAPE;
    if (T > 1 && token_stride > kMaxPlane / 4 / (T - 1)) return QBD_ERR_SHAPE;
    if (heads > 1 && head_stride > kMaxPlane / 4 / (heads - 1)) return QBD_ERR_SHAPE;
    if (token_stride * eb % 16 != 0 || head_stride * eb % 16 != 0) return QBD_ERR_ALIGN;
    return QBD_OK;
}

Span rows_span(const void* p, int64_t T, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride, int64_t eb) {
    return {p, ((T - 1) * token_stride + (heads - 1) * head_stride + dim) * eb};
}

}  // namespace

extern "C" {

int kv_cache_write(const qbd_kv_cache* cache, const void* k, const void* v, int dtype, int64_t k_token_stride,
                   int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                   int64_t T, qbd_stream_t stream) {
    qbd::KvView kv;
    Planes pl;
    int st = check_cache(cache, kv, pl);
    if (st != QBD_OK) return st;
    if (!elem_ok(dtype) || T < 0 || T > kMaxDim) return QBD_ERR_SHAPE;
    if (T > 0 && int64_t{kv.heads} * kv.dim > kMaxPlane / 4 / T) return QBD_ERR_SHAPE;
    if (T == 0 || kv.pages == 0) return QBD_OK;
    const auto elem = static_cast<qbd::Elem>(dtype);
    const int64_t eb = qbd::elem_bytes(elem);
    if (!k || !v || !slots) return QBD_ERR_NULL;
    if ((st = check_rows(T, kv.heads, kv.dim, k_token_stride, k_head_stride, eb)) != QBD_OK) return st;
    if ((st = check_rows(T, kv.heads, kv.dim, v_token_stride, v_head_stride, eb)) != QBD_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return QBD_ERR_ALIGN;
    const Span ins[3] = {rows_span(k, T, kv.heads, kv.dim, k_token_stride, k_head_stride, eb),
                         rows_span(v, T, kv.heads, kv.dim, v_token_stride, v_head_stride, eb), {slots, T * 8}};
    for (int i = 0; i < 4; ++i) {
        for (const Span& in : ins) {
            if (overlaps(pl.s[i], in)) return QBD_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j) {
            if (overlaps(pl.s[i], pl.s[j])) return QBD_ERR_ALIAS;
        }
    }
    st = check_device();
    if (st != QBD_OK) return st;
    return launched(qbd::launch_kv_write(kv, {k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}, elem,
                                         slots, T, reinterpret_cast<hipStream_t>(stream)));
}

int kv_cache_read(const qbd_kv_cache* cache, const int64_t* slots, int64_t T, int dtype, void* k, void* v,
                  qbd_stream_t stream) {
    qbd::KvView kv;
    Planes pl;
    int st = check_cache(cache, kv, pl);
    if (st != QBD_OK) return st;
    if (!elem_ok(dtype) || T < 0 || T > kMaxDim) return QBD_ERR_SHAPE;
    if (T > 0 && int64_t{kv.heads} * kv.dim > kMaxPlane / 4 / T) return QBD_ERR_SHAPE;
    if (T == 0) return QBD_OK;
    const auto elem = static_cast<qbd::Elem>(dtype);
    if (!k || !v || !slots) return QBD_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return QBD_ERR_ALIGN;
    const int64_t bytes = T * kv.heads * kv.dim * qbd::elem_bytes(elem);
    const Span outs[2] = {{k, bytes}, {v, bytes}};
    if (overlaps(outs[0], outs[1])) return QBD_ERR_ALIAS;
    for (const Span& o : outs) {
        if (overlaps(o, {slots, T * 8})) return QBD_ERR_ALIAS;
        for (const Span& p : pl.s) {
            if (overlaps(o, p)) return QBD_ERR_ALIAS;
        }
    }
    st = check_device();
    if (st != QBD_OK) return st;
    return launched(qbd::launch_kv_read(kv, slots, T, elem, k, v, reinterpret_cast<hipStream_t>(stream)));
}

int64_t kv_attention_work_bytes(const qbd_kv_cache* cache, int64_t batch, int64_t T, int64_t qheads, int64_t max_q,
                                int64_t max_len) {
    qbd::KvView kv;
    Planes pl;
    if (!cache || batch <= 0 || batch > kMaxDim || T <= 0 || T > kMaxDim || qheads <= 0 || qheads > 65535) return 0;
    qbd_kv_cache shape = *cache;
    shape.pages = 0;  // the planes are not looked at
    if (check_cache(&shape, kv, pl) != QBD_OK || qheads % kv.heads != 0) return 0;
    return qbd::kv_plan::work_bytes(kv.dim, kv.heads, static_cast<int>(qheads), batch, T, max_q, max_len);
}

int kv_attention(const qbd_kv_cache* cache, const void* q, int dtype, int64_t q_token_stride, int64_t q_head_stride,
                 const int32_t* table, int64_t table_width, const int32_t* lens, const int32_t* q_starts, int64_t batch,
                 int64_t T, int64_t qheads, int64_t max_q, int64_t max_len, int causal, int64_t window, float scale,
                 void* out, void* work, int64_t work_bytes, qbd_stream_t stream) {
    qbd::KvView kv;
    Planes pl;
    int st = check_cache(cache, kv, pl);
    if (st != QBD_OK) return st;
    if (!elem_ok(dtype) || batch < 0 || batch > kMaxDim || T < 0 || T > kMaxDim) return QBD_ERR_SHAPE;
    if (qheads <= 0 || qheads > 65535 || qheads % kv.heads != 0) return QBD_ERR_SHAPE;
    if (table_width < 0 || table_width > kMaxDim || max_q < 0 || max_len < 0 || window < 0 || work_bytes < 0) return QBD_ERR_SHAPE;
    if (table_width > kMaxDim >> kv.page_shift) return QBD_ERR_SHAPE;  // positions are 32-bit
    if (batch > 0 && table_width > kMaxPlane / 4 / batch) return QBD_ERR_SHAPE;
    if (window > int64_t{1} << 31) window = int64_t{1} << 31;  // positions lie below it: the kernels subtract a window from them
    if ((window > 0 && !causal) || !std::isfinite(scale)) return QBD_ERR_SHAPE;
    if (T > 0 && qheads * kv.dim > kMaxPlane / 4 / T) return QBD_ERR_SHAPE;
    if (T > 0 && qheads / kv.heads > kMaxDim / T) return QBD_ERR_SHAPE;  // rows of a cached head are 32-bit
    if (T > 0 && (batch == 0 || (!q_starts && T % batch != 0))) return QBD_ERR_SHAPE;
    if (T == 0) return QBD_OK;
    const auto elem = static_cast<qbd::Elem>(dtype);
    const int64_t eb = qbd::elem_bytes(elem);
    if (!q || !out || !lens || (table_width > 0 && !table)) return QBD_ERR_NULL;
    if ((st = check_rows(T, qheads, kv.dim, q_token_stride, q_head_stride, eb)) != QBD_OK) return st;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_starts, 4)) return QBD_ERR_ALIGN;
    // the size that was asked for, or what this launch takes should that be more
    const int64_t asked = qbd::kv_plan::work_bytes(kv.dim, kv.heads, static_cast<int>(qheads), batch, T, max_q, max_len);
    const int64_t taken = qbd::kv_plan::work_bytes(kv.dim, kv.heads, static_cast<int>(qheads), batch, T, max_q, max_len, window);
    const int64_t need = taken > asked ? taken : asked;
    if (need > 0) {
        if (!work || work_bytes < need) return QBD_ERR_WORK;
        if (!aligned(work, 256)) return QBD_ERR_ALIGN;
    }
    const Span outs[2] = {{out, T * qheads * kv.dim * eb}, {work, need}};
    const Span ins[8] = {rows_span(q, T, qheads, kv.dim, q_token_stride, q_head_stride, eb), {table, batch * table_width * 4},
                         {lens, batch * 4}, {q_starts, q_starts ? (batch + 1) * 4 : 0}, pl.s[0], pl.s[1], pl.s[2], pl.s[3]};
    if (overlaps(outs[0], outs[1])) return QBD_ERR_ALIAS;
    for (const Span& o : outs) {
        for (const Span& in : ins) {
            if (overlaps(o, in)) return QBD_ERR_ALIAS;
        }
    }
    st = check_device();
    if (st != QBD_OK) return st;
    qbd::AttnArgs a{};
    a.kv = kv;
    a.q = {q, q_token_stride, q_head_stride};
    a.elem = elem;
    a.table = table;
    a.table_width = table_width;
    a.lens = lens;
    a.q_starts = q_starts;
    a.batch = static_cast<int>(batch);
    a.T = T;
    a.qheads = static_cast<int>(qheads);
    a.max_q = max_q;
    a.max_len = max_len;
    a.causal = causal != 0;
    a.window = window;
    a.scale = scale;
    a.out = out;
    a.work = work;
    return launched(qbd::launch_kv_attention(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
