// ds_lm.h -- structures and launchers of the language-model rows (embedding
// rows, normed and rotated q/k rows, token log probabilities), shared by the
// host side (ds_lm_api.cpp) and the kernels.  Not part of the public ABI.
#pragma once

#include <vector_types.h>

#include "ds_internal.h"

namespace ds {

// Segments of one launch.  Most calls have one: kernels with N = 1 find their
// fields at fixed places of the parameter block (a table in the block costs
// an indexed constant load per field: 54.7 -> 52.0 us on 16,384 embedding rows).
constexpr int kLmSegs = 8;

// Embedding rows (ds_embed.cu).
struct ESegK {
    const void *w, *ids;
    const float *gain;
    void *y;
    int64_t tokens, vocab;
    int64_t ld, ld_y;
    int32_t cols, nu; // nu: octets per row
    float radius;
    int32_t unit, gain_scalar, ids_i64;
};
template <int N>
struct EParams {
    ESegK seg[N];
    int64_t unit_start[N + 1]; // prefix sums of tokens
    int32_t nseg;
    float eps;
};
// Their gradient: the rows of the table are dealt to 128 lists by row mod
// 128, counted in shared memory (kEmbedMaxRows rows a list).
constexpr int kEmbedBuckets = 128;
constexpr int kEmbedMaxRows = 40960;
// Tokens of one row summed in one go (a chunk): 2^l, or so many that a row has at
// most 128 chunks (a multiple of 2^l).  8 where a warp takes a chunk (rows of at
// most 1024 columns), 32 where a block does.
DS_HD constexpr int embed_l(int64_t cols) { return cols <= 1024 ? 3 : 5; }
DS_HD constexpr int embed_chunk(int n, int l)
{
    const int c = (((n + 127) >> 7) + (1 << l) - 1) >> l << l;
    return c > (1 << l) ? c : 1 << l;
}
// The workspace line of a chunk that starts at place `start` of the token
// list, among rows of several chunks: two chunks that start within the same 2^l
// places are the last chunk of one row and the first of the next.
DS_HD constexpr int64_t embed_line(int64_t start, bool first, int l) { return 2 * (start >> l) + (first ? 1 : 0); }
constexpr int kEmbedJoin = 8; // chunks, then sums of chunks, that are joined at once
struct EGroupParams {
    const void *ids;
    int64_t tokens, vocab, named_ld;
    int32_t *order;   // [tokens] the tokens, row by row
    int2 *list;       // [tokens] scratch: (row of the list, token)
    int4 *items;      // [tokens] (row, place of its first token, its tokens, chunk)
    int2 *nitems;     // [128] (place of the list's first item, its items)
    uint32_t *named;  // [128][named_ld] one bit per row: some token names it
    int32_t *arrived; // [2][lines] chunks done, at the line of their first; groups of chunks done
    int64_t lines;
    int32_t ids_i64;
    int32_t l;        // embed_l
};
struct EGradParams {
    const void *w, *dy;
    const float *gain;
    float *grad_w, *grad_g;
    const int32_t *order;
    const int4 *items;
    const int2 *nitems;
    const uint32_t *named;
    int32_t *arrived;
    float *lines; // partial sums of the rows with several chunks
    int64_t nlines;
    int64_t vocab, ld, ld_y, ld_g, named_ld, line_ld;
    int32_t cols;
    float radius, eps;
    int32_t unit, gain_scalar, accumulate, l;
    int32_t stage, stages, per_stage; // set by the launcher: the ring's bytes a stage, stages, tokens a stage
    uint64_t wait_limit_ns;
};
constexpr int kEmbedStages = 6;             // most stages of the ring
constexpr int kEmbedSlots = 16;             // most slots of a warp's ring
constexpr int kEmbedZeros = 8192;           // bytes of zeros that bulk copies write from
constexpr int kEmbedSmemMax = 220 * 1024;   // dynamic shared memory of k_embed_reduce
// Embedding rows (ds_embed.cu): a class by the row length; units: tokens.
int embed_class(int64_t cols);
int launch_embed(bool w_bf16, bool y_bf16, int cls, const EParams<kLmSegs> &p, int64_t units, void *stream);
int launch_embed_group(const EGroupParams &p, void *stream);
int launch_embed_reduce(bool w_bf16, bool dy_bf16, int cls, const EGradParams &p, int sms, void *stream);

// Normed and rotated q and k rows (ds_qkn.cu).
constexpr int kNormMaxDim = 512;
struct QNSegK {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    const float *wq, *wk, *inv;
    const int32_t *pos, *slot;
    int64_t rows, cache_rows, ld_q, ld_kv, ld_qo, ld_cache;
    int32_t D, rot, hq, hk;
    int32_t lp;           // lanes per head (a power of two, >= D / 16)
    int32_t nq, nk, tpr;  // groups of 32 / lp heads of q and of k; groups per row
    int32_t parts, tpp;   // warps per row, groups per warp
    float eps, post;      // n = sqrt(sum x^2 + eps) / post
};
template <int N>
struct QNParams {
    QNSegK seg[N];
    int64_t unit_start[N + 1]; // prefix sums of rows x parts
    int32_t nseg;
};
struct QNGSegK {
    const void *q, *k, *dqo, *dko;
    void *dq, *dk;
    const float *wq, *wk, *inv;
    const int32_t *pos;
    int64_t rows, ld_q, ld_kv, ld_dqo, ld_dko, ld_dq, ld_dk;
    int32_t D, rot, hq, hk;
    int32_t lp, nq, nk, tpr, parts, tpp;
    float eps, post;
};
template <int N>
struct QNGParams {
    QNGSegK seg[N];
    int64_t unit_start[N + 1];
    float *ws; // [grid][2][D] the blocks' sums for dwq and dwk (NULL: not wanted)
    int32_t nseg;
};
int launch_qkn(bool bf16, bool neighbours, const QNParams<kLmSegs> &p, int64_t units, int sms, void *stream);
int launch_qkn_grad(bool bf16, bool grad_bf16, bool neighbours, const QNGParams<kLmSegs> &p, int64_t units, int sms, int *blocks,
                    void *stream); // *blocks: lines of p.ws that are written
int qkn_blocks_per_sm(); // of either direction's grid, of qkn_warps() warps each
int qkn_warps();
int launch_qkn_dw(const float *ws, int lines, int D, float *dwq, float *dwk, void *stream);

// The one segment of a launch as a parameter block of its own.
template <template <int> class P>
inline P<1> only_segment(const P<kLmSegs> &p)
{
    P<1> o;
    o.seg[0] = p.seg[0];
    o.unit_start[0] = p.unit_start[0];
    o.unit_start[1] = p.unit_start[1];
    o.nseg = 1;
    return o;
}

// Token log probabilities (ds_logp.cu).
struct LSegK {
    const void *x, *ids;
    float *logp, *lse, *entropy; // the gradient reads lse and entropy
    int32_t *top_id;
    float *top_logp;
    const float *dlogp, *dentropy, *dlse;
    void *dx;
    int64_t rows, ld, ld_d;
    int32_t cols, top, ids_i64;
    float scale;
};
template <int N>
struct LParams {
    LSegK seg[N];
    int64_t unit_start[N + 1];       // prefix sums of rows (gradient: of parts of rows)
    int32_t nseg;
    uint64_t wait_limit_ns;          // bound of every device-side wait
};
// A class by the row length (1: may be split over a cluster of cl CTAs), the
// steps of a row of class 1.
int logp_class(int64_t cols);
int64_t logp_steps(bool bf16, int64_t cols);
int launch_logp(bool bf16, int cls, int cl, bool top, bool ent, const LParams<kLmSegs> &p, int64_t units, int sms, void *stream);
int64_t logp_grad_parts(int64_t cols); // blocks of a row
int launch_logp_grad(bool bf16, bool grad_bf16, const LParams<kLmSegs> &p, int64_t units, void *stream);

} // namespace ds
