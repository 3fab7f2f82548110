// ds_lm_api.cpp -- the C ABI of the language-model rows: embedding rows,
// normed and rotated q/k rows and token log probabilities, forward and
// gradient.  Arguments are checked here before anything is launched.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <new>
#include <vector>

#include <cuda_runtime.h>

#include "ds.h"
#include "ds_host.h"
#include "ds_lm.h"

namespace {

using namespace ds;

constexpr int64_t kMaxLd = int64_t(1) << 40;

ds_status launched(int e)
{
    if (e != 0) {
        char buf[96];
        std::snprintf(buf, sizeof(buf), "kernel launch failed (cudaError %d)", e);
        return fail(DS_ERR_CUDA, buf);
    }
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return DS_OK;
}

bool dtype_ok(ds_dtype d) { return d == DS_F32 || d == DS_BF16; }
int size_of(ds_dtype d) { return d == DS_BF16 ? 2 : 4; }

// A vector of n values.
ds_status check_vector(const void *p, int64_t n, int align, const char *name, int i)
{
    if (n == 0)
        return DS_OK;
    if (!p)
        return fail(DS_ERR_INVALID_ARG, where((std::string(name) + " is NULL").c_str(), i));
    if (!aligned(p, align))
        return fail(DS_ERR_ALIGNMENT, where((std::string(name) + " is not aligned").c_str(), i));
    return DS_OK;
}

// -------------------------------------------------------- embedding rows --

constexpr int64_t kMaxTokens = int64_t(1) << 30;

// What both directions check of a segment.
ds_status check_embed(const ds_eseg &s, int i)
{
    if (s.tokens < 0 || s.tokens > kMaxTokens)
        return fail(DS_ERR_INVALID_ARG, where("tokens outside [0, 2^30]", i));
    if (s.vocab < 1 || s.vocab > kMaxCols)
        return fail(DS_ERR_INVALID_ARG, where("vocab outside [1, 2^31 - 1]", i));
    if (s.cols < 1 || s.cols > kMaxCols)
        return fail(DS_ERR_INVALID_ARG, where("cols outside [1, 2^31 - 1]", i));
    if (!std::isfinite(s.radius))
        return fail(DS_ERR_INVALID_ARG, where("radius is not finite", i));
    if (s.gain && !s.unit)
        return fail(DS_ERR_INVALID_ARG, where("gain needs unit = 1", i));
    if (s.gain && !aligned(s.gain, 4))
        return fail(DS_ERR_ALIGNMENT, where("gain is not 4-byte aligned", i));
    return check_vector(s.ids, s.tokens, s.ids_i64 ? 8 : 4, "ids", i);
}

ds_status check_ld(int64_t ld, int64_t cols, const char *name, int i)
{
    if (ld < cols || ld > kMaxLd)
        return fail(DS_ERR_INVALID_ARG, where((std::string(name) + " below cols (or too large)").c_str(), i));
    return DS_OK;
}

// What a call only reads of a segment.
void embed_inputs(const ds_eseg &s, int i, ds_dtype w_dtype, bool w, std::vector<Span> &spans)
{
    if (s.tokens > 0)
        spans.push_back(span_of(s.ids, 1, s.tokens, s.tokens, s.ids_i64 ? 8 : 4, i, 0, -1));
    if (w)
        spans.push_back(span_rows(s.w, s.vocab, s.cols, s.ld, size_of(w_dtype), i, 0, -1));
    if (s.unit && s.gain) {
        const int64_t n = s.gain_scalar ? 1 : s.vocab;
        spans.push_back(span_of(s.gain, 1, n, n, 4, i, 0, -1));
    }
}

ds_status run_embed(const ds_eseg *segs, int nseg, ds_dtype w_dtype, ds_dtype out_dtype, float eps, void *stream)
{
    g_last_error.clear();
    if (ds_status s = check_common(nseg, segs, eps, stream))
        return s;
    if (!dtype_ok(w_dtype) || !dtype_ok(out_dtype))
        return fail(DS_ERR_UNSUPPORTED_DTYPE, "w_dtype and out_dtype must be DS_F32 or DS_BF16");
    std::vector<Span> spans;
    for (int i = 0; i < nseg; ++i) {
        const ds_eseg &s = segs[i];
        if (ds_status st = check_embed(s, i))
            return st;
        if (ds_status st = check_ld(s.ld, s.cols, "ld", i))
            return st;
        if (ds_status st = check_ld(s.ld_y, s.cols, "ld_y", i))
            return st;
        if (s.tokens == 0)
            continue;
        if (ds_status st = check_matrix(s.w, s.vocab, s.ld, size_of(w_dtype), "w", i))
            return st;
        if (ds_status st = check_matrix(s.y, s.tokens, s.ld_y, size_of(out_dtype), "y", i))
            return st;
        embed_inputs(s, i, w_dtype, true, spans);
        spans.push_back(span_rows(s.y, s.tokens, s.cols, s.ld_y, size_of(out_dtype), i, 1, -1));
    }
    if (ds_status st = check_overlaps(spans))
        return st;
    static thread_local EParams<kLmSegs> params;
    for (int cls = 0; cls < 8; ++cls) { // one launch per class present
        int n = 0;
        int64_t units = 0;
        auto flush = [&]() -> ds_status {
            if (n == 0)
                return DS_OK;
            params.nseg = n;
            params.unit_start[n] = units;
            params.eps = eps;
            const ds_status st =
                launched(launch_embed(w_dtype == DS_BF16, out_dtype == DS_BF16, cls, params, units, stream));
            n = 0;
            units = 0;
            return st;
        };
        for (int i = 0; i < nseg; ++i) {
            const ds_eseg &s = segs[i];
            if (s.tokens == 0 || embed_class(s.cols) != cls)
                continue;
            if (n == kLmSegs || units + s.tokens > 0x7fffffff)
                if (ds_status st = flush())
                    return st;
            ESegK &k = params.seg[n];
            k = ESegK{};
            k.w = s.w;
            k.ids = s.ids;
            k.gain = s.unit ? s.gain : nullptr;
            k.y = s.y;
            k.tokens = s.tokens;
            k.vocab = s.vocab;
            k.ld = s.ld;
            k.ld_y = s.ld_y;
            k.cols = static_cast<int32_t>(s.cols);
            k.nu = static_cast<int32_t>((s.cols + 7) / 8);
            k.radius = s.radius;
            k.unit = s.unit;
            k.gain_scalar = s.gain_scalar;
            k.ids_i64 = s.ids_i64;
            params.unit_start[n] = units;
            units += s.tokens;
            ++n;
        }
        if (ds_status st = flush())
            return st;
    }
    return DS_OK;
}

// The gradient's workspace, in order; every part starts on 256 bytes.
struct EmbedWs {
    int64_t named_ld, line_ld, nlines;
    uint64_t items, list, order, nitems, named, arrived, lines, bytes;
};

EmbedWs embed_ws(int64_t tokens, int64_t vocab, int64_t cols)
{
    auto up = [](uint64_t b) { return (b + 255) / 256 * 256; };
    EmbedWs w{};
    const int64_t rows = (vocab + kEmbedBuckets - 1) / kEmbedBuckets;
    w.named_ld = (rows + 31) / 32;
    w.line_ld = (cols + 7) / 8 * 8;
    // only rows of more than 2^l tokens have partial sums
    const int64_t least = int64_t(1) << embed_l(cols);
    const uint64_t lines = tokens > least ? 2 * ((tokens + least - 1) / least) : 0;
    w.nlines = lines;
    w.items = 0;
    w.list = w.items + up(16 * tokens);
    w.order = w.list + up(8 * tokens);
    w.nitems = w.order + up(4 * tokens);
    w.named = w.nitems + up(8 * kEmbedBuckets);
    w.arrived = w.named + up(4 * kEmbedBuckets * w.named_ld);
    w.lines = w.arrived + up(8 * lines);
    w.bytes = w.lines + up(4 * lines * w.line_ld);
    return w;
}

constexpr int64_t kEmbedGradCols = 16384;
constexpr int64_t kEmbedGradVocab = int64_t(kEmbedBuckets) * kEmbedMaxRows;

uint64_t embed_ws_bytes(int64_t tokens, int64_t vocab, int64_t cols)
{
    if (tokens < 0 || tokens > kMaxTokens || vocab < 1 || vocab > kEmbedGradVocab || cols < 1 || cols > kEmbedGradCols)
        return 0;
    return embed_ws(tokens, vocab, cols).bytes;
}

ds_status run_embed_grad(const ds_eseg *segs, int nseg, ds_dtype w_dtype, ds_dtype dy_dtype, float eps, void *ws,
                         uint64_t ws_bytes, void *stream)
{
    g_last_error.clear();
    if (ds_status s = check_common(nseg, segs, eps, stream))
        return s;
    if (!dtype_ok(w_dtype) || !dtype_ok(dy_dtype))
        return fail(DS_ERR_UNSUPPORTED_DTYPE, "w_dtype and dy_dtype must be DS_F32 or DS_BF16");
    std::vector<Span> spans;
    uint64_t need = 0;
    auto idle = [](const ds_eseg &s) { return s.tokens == 0 && s.accumulate; };
    for (int i = 0; i < nseg; ++i) {
        const ds_eseg &s = segs[i];
        if (ds_status st = check_embed(s, i))
            return st;
        if (s.vocab > kEmbedGradVocab)
            return fail(DS_ERR_INVALID_ARG, where("vocab above 5242880 (the gradient counts a row's tokens on chip)", i));
        if (s.cols > kEmbedGradCols)
            return fail(DS_ERR_INVALID_ARG, where("cols above 16384 (the gradient holds a row in registers)", i));
        if (s.unit)
            if (ds_status st = check_ld(s.ld, s.cols, "ld", i))
                return st;
        if (ds_status st = check_ld(s.ld_y, s.cols, "ld_y", i))
            return st;
        if (ds_status st = check_ld(s.ld_g, s.cols, "ld_g", i))
            return st;
        if (idle(s))
            continue;
        if (ds_status st = check_matrix(s.grad_w, s.vocab, s.ld_g, 4, "grad_w", i))
            return st;
        if (s.unit)
            if (ds_status st = check_matrix(s.w, s.vocab, s.ld, size_of(w_dtype), "w", i))
                return st;
        if (ds_status st = check_matrix(s.dy, s.tokens, s.ld_y, size_of(dy_dtype), "dy", i))
            return st;
        embed_inputs(s, i, w_dtype, s.unit != 0, spans);
        if (s.tokens > 0)
            spans.push_back(span_rows(s.dy, s.tokens, s.cols, s.ld_y, size_of(dy_dtype), i, 0, -1));
        spans.push_back(span_rows(s.grad_w, s.vocab, s.cols, s.ld_g, 4, i, 1, -1));
        if (s.gain) {
            const int64_t n = s.vocab + (s.gain_scalar ? 1 : 0);
            if (ds_status st = check_vector(s.grad_g, n, 4, "grad_g", i))
                return st;
            spans.push_back(span_of(s.grad_g, 1, n, n, 4, i, 1, -1));
        }
        need = std::max(need, embed_ws_bytes(s.tokens, s.vocab, s.cols));
    }
    if (need > 0) {
        if (!ws || !aligned(ws, 256))
            return fail(ws ? DS_ERR_ALIGNMENT : DS_ERR_INVALID_ARG, "workspace NULL or not 256-byte aligned");
        if (ws_bytes < need)
            return fail(DS_ERR_INVALID_ARG, "workspace smaller than ds_embed_rows_backward_workspace(tokens, vocab, cols)");
        const uintptr_t lo = reinterpret_cast<uintptr_t>(ws);
        spans.push_back({lo, lo + need, -1, 1, -1});
    }
    if (ds_status st = check_overlaps(spans))
        return st;
    char *base = static_cast<char *>(ws);
    for (int i = 0; i < nseg; ++i) { // one after another: they share the workspace
        const ds_eseg &s = segs[i];
        if (idle(s))
            continue;
        const EmbedWs w = embed_ws(s.tokens, s.vocab, s.cols);
        EGroupParams g{};
        g.ids = s.ids;
        g.tokens = s.tokens;
        g.vocab = s.vocab;
        g.named_ld = w.named_ld;
        g.order = reinterpret_cast<int32_t *>(base + w.order);
        g.list = reinterpret_cast<int2 *>(base + w.list);
        g.items = reinterpret_cast<int4 *>(base + w.items);
        g.nitems = reinterpret_cast<int2 *>(base + w.nitems);
        g.named = reinterpret_cast<uint32_t *>(base + w.named);
        g.arrived = reinterpret_cast<int32_t *>(base + w.arrived);
        g.ids_i64 = s.ids_i64;
        g.lines = w.nlines;
        g.l = embed_l(s.cols);
        if (ds_status st = launched(launch_embed_group(g, stream)))
            return st;
        EGradParams p{};
        p.w = s.w;
        p.dy = s.dy;
        p.gain = s.gain;
        p.grad_w = s.grad_w;
        p.grad_g = s.gain ? s.grad_g : nullptr;
        p.order = g.order;
        p.items = g.items;
        p.nitems = g.nitems;
        p.named = g.named;
        p.arrived = g.arrived;
        p.lines = reinterpret_cast<float *>(base + w.lines);
        p.vocab = s.vocab;
        p.ld = s.ld;
        p.ld_y = s.ld_y;
        p.ld_g = s.ld_g;
        p.named_ld = w.named_ld;
        p.line_ld = w.line_ld;
        p.cols = static_cast<int32_t>(s.cols);
        p.radius = s.radius;
        p.eps = eps;
        p.unit = s.unit;
        p.gain_scalar = s.gain_scalar;
        p.accumulate = s.accumulate;
        p.nlines = w.nlines;
        p.l = g.l;
        p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
        if (ds_status st = launched(launch_embed_reduce(w_dtype == DS_BF16, dy_dtype == DS_BF16, embed_class(s.cols), p,
                                                        sm_count(), stream)))
            return st;
        if (s.gain && s.gain_scalar) { // dL/dg of the one gain: the rows' parts in a fixed order
            static thread_local GainSumParams sums;
            sums.nseg = 1;
            sums.seg[0] = {s.grad_g, s.vocab};
            if (ds_status st = launched(launch_gain_sums(sums, stream)))
                return st;
        }
    }
    return DS_OK;
}

// ------------------------------------------- normed and rotated q/k rows --

ds_status check_heads(int64_t rows, int32_t D, int32_t rot, int32_t hq, int32_t hk, const int32_t *pos,
                      const float *inv, int i)
{
    if (rows < 0 || rows > kMaxLd)
        return fail(DS_ERR_INVALID_ARG, where("rows outside [0, 2^40]", i));
    if (D < 16 || D > kNormMaxDim || D % 16)
        return fail(DS_ERR_INVALID_ARG, where("head_dim must be a multiple of 16 in [16, 512]", i));
    if (rot < 0 || rot > D || rot % 16)
        return fail(DS_ERR_INVALID_ARG, where("rot_dim must be a multiple of 16 in [0, head_dim]", i));
    if (hq < 0 || hk < 0 || hq + hk < 1 || hq > 4096 || hk > 4096)
        return fail(DS_ERR_INVALID_ARG, where("hq, hk must be in [0, 4096] with hq + hk >= 1", i));
    if (rows > 0 && rot > 0) {
        if (ds_status st = check_vector(pos, rows, 4, "pos", i))
            return st;
        if (ds_status st = check_vector(inv, rot / 2, 4, "inv_freq", i))
            return st;
    }
    return DS_OK;
}

ds_status check_weight(const float *w, int32_t D, const char *name, int i, std::vector<Span> &spans)
{
    if (!w)
        return DS_OK;
    if (!aligned(w, 16))
        return fail(DS_ERR_ALIGNMENT, where((std::string(name) + " is not 16-byte aligned").c_str(), i));
    spans.push_back(span_of(w, 1, D, D, 4, i, 0, -1));
    return DS_OK;
}

// A matrix of whole heads.
ds_status check_rows(const void *p, int64_t rows, int64_t cols, int64_t ld, int esize, const char *name, int i)
{
    if (ld < cols || ld > kMaxLd)
        return fail(DS_ERR_INVALID_ARG, where((std::string(name) + ": leading dimension below its heads (or too large)").c_str(), i));
    return check_matrix(p, rows, ld, esize, name, i);
}

// How a row's heads are dealt to lanes and warps.  A row is split over
// several warps where there are fewer rows than warps on the device (the
// values do not depend on it).
template <class K>
void deal_heads(K &k, bool v, bool mean, float eps, int64_t total_rows)
{
    int lp = 1;
    while (lp * 16 < k.D)
        lp *= 2;
    const int hw = 32 / lp;
    k.lp = lp;
    k.nq = (k.hq + hw - 1) / hw;
    k.nk = (k.hk + hw - 1) / hw;
    k.tpr = k.nq + k.nk + (v ? k.nk : 0);
    const int64_t warps = int64_t(sm_count()) * qkn_blocks_per_sm() * qkn_warps();
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(k.tpr, warps / std::max<int64_t>(1, total_rows)));
    k.tpp = static_cast<int32_t>((k.tpr + want - 1) / want);
    k.parts = (k.tpr + k.tpp - 1) / k.tpp;
    k.eps = mean ? eps * static_cast<float>(k.D) : eps;
    k.post = mean ? std::sqrt(static_cast<float>(k.D)) : 1.f;
}

ds_status run_qkn(const ds_qnseg *segs, int nseg, ds_dtype dtype, float eps, void *stream)
{
    g_last_error.clear();
    if (ds_status s = check_common(nseg, segs, eps, stream))
        return s;
    if (!dtype_ok(dtype))
        return fail(DS_ERR_UNSUPPORTED_DTYPE, "dtype must be DS_F32 or DS_BF16");
    const int es = size_of(dtype);
    std::vector<Span> spans;
    int64_t total_rows = 0;
    if (!std::isfinite(eps * kNormMaxDim))
        return fail(DS_ERR_INVALID_ARG, "eps too large");
    for (int i = 0; i < nseg; ++i) {
        const ds_qnseg &s = segs[i];
        if (ds_status st = check_heads(s.rows, s.head_dim, s.rot_dim, s.hq, s.hk, s.pos, s.inv_freq, i))
            return st;
        if (s.v && s.hk == 0)
            return fail(DS_ERR_INVALID_ARG, where("v needs hk >= 1", i));
        if (s.rows == 0)
            continue;
        total_rows += s.rows;
        const int64_t wq = int64_t(s.hq) * s.head_dim, wk = int64_t(s.hk) * s.head_dim;
        if (s.rot_dim > 0) {
            spans.push_back(span_of(s.pos, 1, s.rows, s.rows, 4, i, 0, -1));
            spans.push_back(span_of(s.inv_freq, 1, s.rot_dim / 2, s.rot_dim / 2, 4, i, 0, -1));
        }
        if (s.hq > 0) {
            if (ds_status st = check_rows(s.q, s.rows, wq, s.ld_q, es, "q", i))
                return st;
            if (ds_status st = check_rows(s.q_out, s.rows, wq, s.ld_qo, es, "q_out", i))
                return st;
            if (ds_status st = check_weight(s.wq, s.head_dim, "wq", i, spans))
                return st;
            spans.push_back(span_rows(s.q, s.rows, wq, s.ld_q, es, i, 0, 3 * i));
            spans.push_back(span_rows(s.q_out, s.rows, wq, s.ld_qo, es, i, 1, 3 * i));
        }
        if (s.hk > 0) {
            if (s.cache_rows < 1 || s.cache_rows > kMaxLd || (!s.slot && s.cache_rows < s.rows))
                return fail(DS_ERR_INVALID_ARG, where("cache_rows below rows (no slot) or outside [1, 2^40]", i));
            if (s.slot) {
                if (ds_status st = check_vector(s.slot, s.rows, 4, "slot", i))
                    return st;
                spans.push_back(span_of(s.slot, 1, s.rows, s.rows, 4, i, 0, -1));
            }
            if (ds_status st = check_rows(s.k, s.rows, wk, s.ld_kv, es, "k", i))
                return st;
            if (ds_status st = check_rows(s.k_cache, s.cache_rows, wk, s.ld_cache, es, "k_cache", i))
                return st;
            if (ds_status st = check_weight(s.wk, s.head_dim, "wk", i, spans))
                return st;
            // in place only row for row (no slots) over the same matrix
            const int key_k = s.slot ? -1 : 3 * i + 1, key_v = s.slot ? -1 : 3 * i + 2;
            spans.push_back(span_rows(s.k, s.rows, wk, s.ld_kv, es, i, 0, key_k));
            spans.push_back(span_rows(s.k_cache, s.cache_rows, wk, s.ld_cache, es, i, 1, key_k));
            if (s.v) {
                if (ds_status st = check_rows(s.v, s.rows, wk, s.ld_kv, es, "v", i))
                    return st;
                if (ds_status st = check_rows(s.v_cache, s.cache_rows, wk, s.ld_cache, es, "v_cache", i))
                    return st;
                spans.push_back(span_rows(s.v, s.rows, wk, s.ld_kv, es, i, 0, key_v));
                spans.push_back(span_rows(s.v_cache, s.cache_rows, wk, s.ld_cache, es, i, 1, key_v));
            }
        }
    }
    if (ds_status st = check_overlaps(spans))
        return st;
    static thread_local QNParams<kLmSegs> params;
    for (int style = 0; style < 2; ++style) { // one launch per pairing present
        int n = 0;
        int64_t units = 0;
        auto flush = [&]() -> ds_status {
            if (n == 0)
                return DS_OK;
            params.nseg = n;
            params.unit_start[n] = units;
            const ds_status st = launched(launch_qkn(dtype == DS_BF16, style != 0, params, units, sm_count(), stream));
            n = 0;
            units = 0;
            return st;
        };
        for (int i = 0; i < nseg; ++i) {
            const ds_qnseg &s = segs[i];
            if (s.rows == 0 || (s.interleaved != 0) != (style != 0))
                continue;
            if (n == kLmSegs)
                if (ds_status st = flush())
                    return st;
            QNSegK &k = params.seg[n];
            k = QNSegK{};
            k.q = s.q;
            k.k = s.k;
            k.v = s.v;
            k.q_out = s.q_out;
            k.k_cache = s.k_cache;
            k.v_cache = s.v_cache;
            k.wq = s.wq;
            k.wk = s.wk;
            k.inv = s.inv_freq;
            k.pos = s.pos;
            k.slot = s.hk > 0 ? s.slot : nullptr;
            k.rows = s.rows;
            k.cache_rows = s.cache_rows;
            k.ld_q = s.ld_q;
            k.ld_kv = s.ld_kv;
            k.ld_qo = s.ld_qo;
            k.ld_cache = s.ld_cache;
            k.D = s.head_dim;
            k.rot = s.rot_dim;
            k.hq = s.hq;
            k.hk = s.hk;
            deal_heads(k, s.v != nullptr, s.mean != 0, eps, total_rows);
            params.unit_start[n] = units;
            units += s.rows * k.parts;
            ++n;
        }
        if (ds_status st = flush())
            return st;
    }
    return DS_OK;
}

uint64_t qkn_ws_bytes(int64_t head_dim)
{
    if (head_dim < 16 || head_dim > kNormMaxDim || head_dim % 16)
        return 0;
    return static_cast<uint64_t>(sm_count()) * qkn_blocks_per_sm() * 2 * static_cast<uint64_t>(head_dim) * 4;
}

ds_status run_qkn_grad(const ds_qngseg *segs, int nseg, ds_dtype dtype, ds_dtype grad_dtype, float eps, float *dwq,
                       float *dwk, void *ws, uint64_t ws_bytes, void *stream)
{
    g_last_error.clear();
    if (ds_status s = check_common(nseg, segs, eps, stream))
        return s;
    if (!dtype_ok(dtype) || !dtype_ok(grad_dtype))
        return fail(DS_ERR_UNSUPPORTED_DTYPE, "dtype and grad_dtype must be DS_F32 or DS_BF16");
    const int es = size_of(dtype), gs = size_of(grad_dtype);
    const bool want = (dwq || dwk) && nseg > 0;
    std::vector<Span> spans;
    int64_t total_rows = 0;
    if (!std::isfinite(eps * kNormMaxDim))
        return fail(DS_ERR_INVALID_ARG, "eps too large");
    for (int i = 0; i < nseg; ++i) {
        const ds_qngseg &s = segs[i];
        if (ds_status st = check_heads(s.rows, s.head_dim, s.rot_dim, s.hq, s.hk, s.pos, s.inv_freq, i))
            return st;
        if (want && (s.head_dim != segs[0].head_dim || s.rot_dim != segs[0].rot_dim ||
                     (s.interleaved != 0) != (segs[0].interleaved != 0) || (dwq && s.wq != segs[0].wq) ||
                     (dwk && s.wk != segs[0].wk)))
            return fail(DS_ERR_INVALID_ARG, where("dwq and dwk need one weight and one head layout", i));
        if (s.rows == 0)
            continue;
        total_rows += s.rows;
        const int64_t wq = int64_t(s.hq) * s.head_dim, wk = int64_t(s.hk) * s.head_dim;
        if (s.rot_dim > 0) {
            spans.push_back(span_of(s.pos, 1, s.rows, s.rows, 4, i, 0, -1));
            spans.push_back(span_of(s.inv_freq, 1, s.rot_dim / 2, s.rot_dim / 2, 4, i, 0, -1));
        }
        struct Side {
            int32_t heads;
            const void *x, *dy;
            void *dx;
            const float *w;
            int64_t ld, ld_dy, ld_dx, cols;
            const char *names[4];
        };
        const Side sides[2] = {{s.hq, s.q, s.dq_out, s.dq, s.wq, s.ld_q, s.ld_dqo, s.ld_dq, wq, {"q", "dq_out", "dq", "wq"}},
                               {s.hk, s.k, s.dk_out, s.dk, s.wk, s.ld_kv, s.ld_dko, s.ld_dk, wk, {"k", "dk_out", "dk", "wk"}}};
        for (int h = 0; h < 2; ++h) {
            const Side &d = sides[h];
            if (d.heads == 0)
                continue;
            if (ds_status st = check_rows(d.x, s.rows, d.cols, d.ld, es, d.names[0], i))
                return st;
            if (ds_status st = check_rows(d.dy, s.rows, d.cols, d.ld_dy, es, d.names[1], i))
                return st;
            if (ds_status st = check_rows(d.dx, s.rows, d.cols, d.ld_dx, gs, d.names[2], i))
                return st;
            if (ds_status st = check_weight(d.w, s.head_dim, d.names[3], i, spans))
                return st;
            // dx may be exactly dy
            spans.push_back(span_rows(d.x, s.rows, d.cols, d.ld, es, i, 0, -1));
            spans.push_back(span_rows(d.dy, s.rows, d.cols, d.ld_dy, es, i, 0, 2 * i + h));
            spans.push_back(span_rows(d.dx, s.rows, d.cols, d.ld_dx, gs, i, 1, 2 * i + h));
        }
    }
    const int32_t D = want ? segs[0].head_dim : 0;
    if (want) {
        if ((dwq && !aligned(dwq, 4)) || (dwk && !aligned(dwk, 4)))
            return fail(DS_ERR_ALIGNMENT, "dwq or dwk is not 4-byte aligned");
        if (nseg > kLmSegs)
            return fail(DS_ERR_INVALID_ARG, "dwq and dwk: at most 8 segments");
        for (float *d : {dwq, dwk})
            if (d)
                spans.push_back(span_of(d, 1, D, D, 4, -2, 1, -1));
        if (total_rows > 0) {
            if (!ws || !aligned(ws, 256))
                return fail(ws ? DS_ERR_ALIGNMENT : DS_ERR_INVALID_ARG, "workspace NULL or not 256-byte aligned");
            if (ws_bytes < qkn_ws_bytes(D))
                return fail(DS_ERR_INVALID_ARG, "workspace smaller than ds_qk_norm_rows_backward_workspace(head_dim)");
            const uintptr_t lo = reinterpret_cast<uintptr_t>(ws);
            spans.push_back({lo, lo + qkn_ws_bytes(D), -3, 1, -1});
        }
    }
    if (ds_status st = check_overlaps(spans))
        return st;
    if (want && total_rows == 0) { // no rows: both are zero
        for (float *d : {dwq, dwk})
            if (d && cudaMemsetAsync(d, 0, static_cast<size_t>(D) * 4, static_cast<cudaStream_t>(stream)) != cudaSuccess)
                return fail(DS_ERR_CUDA, "cudaMemsetAsync failed");
        return DS_OK;
    }
    static thread_local QNGParams<kLmSegs> params;
    for (int style = 0; style < 2; ++style) {
        int n = 0;
        int64_t units = 0;
        auto flush = [&]() -> ds_status {
            if (n == 0)
                return DS_OK;
            params.nseg = n;
            params.unit_start[n] = units;
            params.ws = want ? static_cast<float *>(ws) : nullptr;
            int grid = 0;
            ds_status st = launched(launch_qkn_grad(dtype == DS_BF16, grad_dtype == DS_BF16, style != 0, params, units,
                                                    sm_count(), &grid, stream));
            if (st == DS_OK && want)
                st = launched(launch_qkn_dw(params.ws, grid, D, dwq, dwk, stream));
            n = 0;
            units = 0;
            return st;
        };
        for (int i = 0; i < nseg; ++i) {
            const ds_qngseg &s = segs[i];
            if (s.rows == 0 || (s.interleaved != 0) != (style != 0))
                continue;
            if (n == kLmSegs)
                if (ds_status st = flush())
                    return st;
            QNGSegK &k = params.seg[n];
            k = QNGSegK{};
            k.q = s.q;
            k.k = s.k;
            k.dqo = s.dq_out;
            k.dko = s.dk_out;
            k.dq = s.dq;
            k.dk = s.dk;
            k.wq = s.wq;
            k.wk = s.wk;
            k.inv = s.inv_freq;
            k.pos = s.pos;
            k.rows = s.rows;
            k.ld_q = s.ld_q;
            k.ld_kv = s.ld_kv;
            k.ld_dqo = s.ld_dqo;
            k.ld_dko = s.ld_dko;
            k.ld_dq = s.ld_dq;
            k.ld_dk = s.ld_dk;
            k.D = s.head_dim;
            k.rot = s.rot_dim;
            k.hq = s.hq;
            k.hk = s.hk;
            deal_heads(k, false, s.mean != 0, eps, total_rows);
            params.unit_start[n] = units;
            units += s.rows * k.parts;
            ++n;
        }
        if (ds_status st = flush())
            return st;
    }
    return DS_OK;
}

// ------------------------------------------------ token log probabilities --

constexpr int kMaxTop = 32;
constexpr int64_t kLogpCols = int64_t(1) << 30;

ds_status check_logits(const ds_lseg &s, int es, int i)
{
    if (ds_status st = check_shape(s.rows, s.cols, s.ld, i))
        return st;
    if (s.cols > kLogpCols)
        return fail(DS_ERR_INVALID_ARG, where("cols above 2^30", i));
    if (!(s.scale > 0.f) || !std::isfinite(s.scale) || !std::isfinite(s.scale * 1.5f))
        return fail(DS_ERR_INVALID_ARG, where("scale must be finite and > 0", i));
    return check_matrix(s.x, s.rows, s.ld, es, "x", i);
}

// A vector of one fp32 per row: read (role 0) or written (1); NULL is allowed.
ds_status row_vector(const float *v, int64_t rows, const char *name, int i, int role, std::vector<Span> &spans)
{
    if (!v)
        return DS_OK;
    if (!aligned(v, 4))
        return fail(DS_ERR_ALIGNMENT, where((std::string(name) + " is not aligned").c_str(), i));
    spans.push_back(span_of(v, 1, rows, rows, 4, i, role, -1));
    return DS_OK;
}

LSegK lseg_rows(const ds_lseg &s, int64_t r0, int64_t nr, int es, int gs)
{
    auto at = [&](auto *p, int64_t n) { return p ? p + n : p; };
    LSegK k{};
    k.x = static_cast<const char *>(s.x) + r0 * s.ld * es;
    k.ids = at(static_cast<const char *>(s.ids), r0 * (s.ids_i64 ? 8 : 4));
    k.logp = at(s.logp, r0);
    k.lse = at(s.lse, r0);
    k.entropy = at(s.entropy, r0);
    k.top_id = at(s.top_id, r0 * s.top_k);
    k.top_logp = at(s.top_logp, r0 * s.top_k);
    k.dlogp = at(s.dlogp, r0);
    k.dentropy = at(s.dentropy, r0);
    k.dlse = at(s.dlse, r0);
    k.dx = at(static_cast<char *>(s.dx), r0 * s.ld_d * gs);
    k.rows = nr;
    k.ld = s.ld;
    k.ld_d = s.ld_d;
    k.cols = static_cast<int32_t>(s.cols);
    k.top = s.top_k;
    k.ids_i64 = s.ids_i64;
    k.scale = s.scale;
    return k;
}

ds_status run_logp(const ds_lseg *segs, int nseg, ds_dtype dtype, void *stream)
{
    g_last_error.clear();
    if (ds_status s = check_common(nseg, segs, 0.f, stream))
        return s;
    if (!dtype_ok(dtype))
        return fail(DS_ERR_UNSUPPORTED_DTYPE, "dtype must be DS_F32 or DS_BF16");
    const int es = size_of(dtype);
    std::vector<Span> spans;
    int64_t total_rows = 0;
    for (int i = 0; i < nseg; ++i) {
        const ds_lseg &s = segs[i];
        if (ds_status st = check_logits(s, es, i))
            return st;
        if (s.top_k < 0 || s.top_k > kMaxTop || s.top_k > s.cols)
            return fail(DS_ERR_INVALID_ARG, where("top_k outside [0, 32] or above cols", i));
        if (s.rows == 0)
            continue;
        total_rows += s.rows;
        if (s.logp)
            if (ds_status st = check_vector(s.ids, s.rows, s.ids_i64 ? 8 : 4, "ids", i))
                return st;
        if (!s.logp && !s.lse && !s.entropy && !s.top_k)
            return fail(DS_ERR_INVALID_ARG, where("nothing to compute", i));
        spans.push_back(span_rows(s.x, s.rows, s.cols, s.ld, es, i, 0, -1));
        if (s.logp)
            spans.push_back(span_of(s.ids, 1, s.rows, s.rows, s.ids_i64 ? 8 : 4, i, 0, -1));
        if (ds_status st = row_vector(s.logp, s.rows, "logp", i, 1, spans))
            return st;
        if (ds_status st = row_vector(s.lse, s.rows, "lse", i, 1, spans))
            return st;
        if (ds_status st = row_vector(s.entropy, s.rows, "entropy", i, 1, spans))
            return st;
        if (s.top_k > 0) {
            if (ds_status st = check_vector(s.top_id, s.rows, 4, "top_id", i))
                return st;
            spans.push_back(span_of(s.top_id, s.rows, s.top_k, s.top_k, 4, i, 1, -1));
            if (ds_status st = row_vector(s.top_logp, s.rows * s.top_k, "top_logp", i, 1, spans))
                return st;
        }
    }
    if (ds_status st = check_overlaps(spans))
        return st;
    // A cluster of CTAs per row while the rows leave SMs without one and the
    // row has a step for each (131,072 logits in fp32, one row: 8 CTAs).
    auto cluster = [&](const ds_lseg &s) {
        const int64_t steps = logp_steps(dtype == DS_BF16, s.cols), sms = sm_count();
        int cl = 1;
        if (logp_class(s.cols) == 1)
            while (cl < 8 && 2 * cl <= steps && total_rows * cl * 2 <= 2 * sms)
                cl *= 2;
        return cl;
    };
    static thread_local LParams<kLmSegs> params;
    std::vector<char> done(static_cast<size_t>(nseg), 0);
    for (int first = 0; first < nseg; ++first) { // one launch per class, cluster and set of outputs present
        if (done[first] || segs[first].rows == 0)
            continue;
        const ds_lseg &f = segs[first];
        const int cls = logp_class(f.cols), cl = cluster(f);
        const bool top = f.top_k > 0, ent = f.entropy != nullptr;
        int n = 0;
        int64_t units = 0;
        auto flush = [&]() -> ds_status {
            if (n == 0)
                return DS_OK;
            params.nseg = n;
            params.unit_start[n] = units;
            params.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
            const ds_status st = launched(launch_logp(dtype == DS_BF16, cls, cl, top, ent, params, units, sm_count(), stream));
            n = 0;
            units = 0;
            return st;
        };
        const int64_t cap = 0x7fffffff / cl;
        for (int i = first; i < nseg; ++i) {
            const ds_lseg &s = segs[i];
            if (done[i] || s.rows == 0 || logp_class(s.cols) != cls || cluster(s) != cl || (s.top_k > 0) != top ||
                (s.entropy != nullptr) != ent)
                continue;
            done[i] = 1;
            for (int64_t r0 = 0; r0 < s.rows;) {
                if (n == kLmSegs || units == cap)
                    if (ds_status st = flush())
                        return st;
                const int64_t nr = std::min(s.rows - r0, cap - units);
                params.seg[n] = lseg_rows(s, r0, nr, es, 0);
                params.seg[n].ids = s.logp ? params.seg[n].ids : nullptr;
                params.unit_start[n] = units;
                units += nr;
                ++n;
                r0 += nr;
            }
        }
        if (ds_status st = flush())
            return st;
    }
    return DS_OK;
}

ds_status run_logp_grad(const ds_lseg *segs, int nseg, ds_dtype dtype, ds_dtype grad_dtype, void *stream)
{
    g_last_error.clear();
    if (ds_status s = check_common(nseg, segs, 0.f, stream))
        return s;
    if (!dtype_ok(dtype) || !dtype_ok(grad_dtype))
        return fail(DS_ERR_UNSUPPORTED_DTYPE, "dtype and grad_dtype must be DS_F32 or DS_BF16");
    const int es = size_of(dtype), gs = size_of(grad_dtype);
    std::vector<Span> spans;
    for (int i = 0; i < nseg; ++i) {
        const ds_lseg &s = segs[i];
        if (ds_status st = check_logits(s, es, i))
            return st;
        if (s.ld_d < s.cols || s.ld_d > kMaxLd)
            return fail(DS_ERR_INVALID_ARG, where("ld_d below cols (or too large)", i));
        if (s.rows == 0)
            continue;
        if (ds_status st = check_matrix(s.dx, s.rows, s.ld_d, gs, "dx", i))
            return st;
        if (!s.lse)
            return fail(DS_ERR_INVALID_ARG, where("lse is NULL", i));
        if (s.dentropy && !s.entropy)
            return fail(DS_ERR_INVALID_ARG, where("dentropy needs entropy", i));
        if (s.dlogp) {
            if (ds_status st = check_vector(s.ids, s.rows, s.ids_i64 ? 8 : 4, "ids", i))
                return st;
            spans.push_back(span_of(s.ids, 1, s.rows, s.rows, s.ids_i64 ? 8 : 4, i, 0, -1));
        }
        // dx may be exactly x
        spans.push_back(span_rows(s.x, s.rows, s.cols, s.ld, es, i, 0, i));
        spans.push_back(span_rows(s.dx, s.rows, s.cols, s.ld_d, gs, i, 1, i));
        if (ds_status st = row_vector(s.lse, s.rows, "lse", i, 0, spans))
            return st;
        if (s.dentropy)
            if (ds_status st = row_vector(s.entropy, s.rows, "entropy", i, 0, spans))
                return st;
        if (ds_status st = row_vector(s.dlogp, s.rows, "dlogp", i, 0, spans))
            return st;
        if (ds_status st = row_vector(s.dentropy, s.rows, "dentropy", i, 0, spans))
            return st;
        if (ds_status st = row_vector(s.dlse, s.rows, "dlse", i, 0, spans))
            return st;
    }
    if (ds_status st = check_overlaps(spans))
        return st;
    static thread_local LParams<kLmSegs> params;
    int n = 0;
    int64_t units = 0;
    auto flush = [&]() -> ds_status {
        if (n == 0)
            return DS_OK;
        params.nseg = n;
        params.unit_start[n] = units;
        const ds_status st =
            launched(launch_logp_grad(dtype == DS_BF16, grad_dtype == DS_BF16, params, units, stream));
        n = 0;
        units = 0;
        return st;
    };
    for (int i = 0; i < nseg; ++i) {
        const ds_lseg &s = segs[i];
        const int64_t parts = logp_grad_parts(s.cols);
        for (int64_t r0 = 0; r0 < s.rows;) {
            if (n == kLmSegs || units + parts > 0x7fffffff)
                if (ds_status st = flush())
                    return st;
            const int64_t nr = std::min(s.rows - r0, (0x7fffffff - units) / parts);
            params.seg[n] = lseg_rows(s, r0, nr, es, gs);
            params.unit_start[n] = units;
            units += nr * parts;
            ++n;
            r0 += nr;
        }
    }
    return flush();
}

// A call whose checks find no host memory (they list every buffer of the segments,
// a few MB for DS_MAX_SEGMENTS): an error, as no exception may leave a C function.
template <class F>
ds_status guarded(F call)
{
    try {
        return call();
    } catch (const std::bad_alloc &) {
        try {
            return fail(DS_ERR_TOO_MANY_SEGMENTS, "no host memory to check the segments");
        } catch (const std::bad_alloc &) {
            return DS_ERR_TOO_MANY_SEGMENTS;
        }
    }
}

} // namespace

extern "C" {

ds_status ds_embed_rows(const ds_eseg *segs, int nseg, ds_dtype w_dtype, ds_dtype out_dtype, float eps, ds_stream stream)
{
    return guarded([&] { return run_embed(segs, nseg, w_dtype, out_dtype, eps, stream); });
}

uint64_t ds_embed_rows_backward_workspace(int64_t tokens, int64_t vocab, int64_t cols)
{
    return embed_ws_bytes(tokens, vocab, cols);
}

ds_status ds_embed_rows_backward(const ds_eseg *segs, int nseg, ds_dtype w_dtype, ds_dtype dy_dtype, float eps,
                                 void *workspace, uint64_t workspace_bytes, ds_stream stream)
{
    return guarded([&] { return run_embed_grad(segs, nseg, w_dtype, dy_dtype, eps, workspace, workspace_bytes, stream); });
}

ds_status ds_qk_norm_rows(const ds_qnseg *segs, int nseg, ds_dtype dtype, float eps, ds_stream stream)
{
    return guarded([&] { return run_qkn(segs, nseg, dtype, eps, stream); });
}

uint64_t ds_qk_norm_rows_backward_workspace(int64_t head_dim) { return qkn_ws_bytes(head_dim); }

ds_status ds_qk_norm_rows_backward(const ds_qngseg *segs, int nseg, ds_dtype dtype, ds_dtype grad_dtype, float eps,
                                   float *dwq, float *dwk, void *workspace, uint64_t workspace_bytes, ds_stream stream)
{
    return guarded([&] { return run_qkn_grad(segs, nseg, dtype, grad_dtype, eps, dwq, dwk, workspace, workspace_bytes, stream); });
}

ds_status ds_logp_rows(const ds_lseg *segs, int nseg, ds_dtype dtype, ds_stream stream)
{
    return guarded([&] { return run_logp(segs, nseg, dtype, stream); });
}

ds_status ds_logp_rows_backward(const ds_lseg *segs, int nseg, ds_dtype dtype, ds_dtype grad_dtype, ds_stream stream)
{
    return guarded([&] { return run_logp_grad(segs, nseg, dtype, grad_dtype, stream); });
}

} // extern "C"
