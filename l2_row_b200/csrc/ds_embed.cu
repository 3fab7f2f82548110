// ds_embed.cu -- embedding rows on sm_100a: the rows of a table that a list of
// tokens names, scaled (y = radius w) or brought to their radius on the way
// (y = g radius w / sqrt(sum w^2 + eps), so that the table itself need not be
// normalized to be read), and their gradient.
//
// The forward is bound by memory: ids, every named row once (a repeated one
// comes from L2) and y.  A team of threads takes a token and holds its row in
// registers between the sum of squares and the store.
//
// The gradient of row v is G_v = sum of dy over the tokens that name v, then
// radius G_v, or through the unit row
//     grad_g = radius (w . G) / n,   grad_w = (g radius / n) (G - w (w . G) / n^2).
// Two launches:
//   k_embed_group  lists the tokens of every row in the tokens' order, without
//                  atomics on memory and without a wait between CTAs: CTA b of
//                  128 owns the rows v = b (mod 128).  It reads all ids (they
//                  stay in L2), counts its own and those of the CTAs below it
//                  -- which gives the place of its list -- and writes the
//                  list in a second read.  Rows are dealt by v mod 128
//                  because the frequent tokens of a vocabulary sit together.
//   k_embed_reduce takes the rows in chunks of 32 tokens, a block each, or (rows
//                  of at most 1024 columns) of 8, a warp each; more where that
//                  would be over 128 chunks.  A chunk is summed in fp32 and the
//                  row finished; the chunks of a longer row leave partial sums
//                  in the workspace, joined in order, in eights, by whoever
//                  comes last.  Rows without a token are zeroed beside the sums.
// The sum of a row depends on its own tokens alone, in their order, so it is
// the same on every run.
#include <algorithm>

#include <cuda_runtime.h>

#include "ds_device.cuh"
#include "ds_lm.cuh"

namespace ds {

namespace {

// ---------------------------------------------------------------- forward --

// A team of T threads takes a token and holds its row as K octets per thread
// (octet k T + lane).  K = 0: the row is read twice instead of held.
template <class WT, class YT, int T, int K, int N>
__global__ void __launch_bounds__(T < 128 ? 128 : T, K <= 4 ? 2048 / (T < 128 ? 128 : T) : 4) k_embed(const __grid_constant__ EParams<N> p)
{
    constexpr int kTeams = (T < 128 ? 128 : T) / T;
    constexpr int KK = K > 0 ? K : 1;
    __shared__ float scratch[kTeams][4 * (T / 32)];
    const int team = threadIdx.x / T, lane = threadIdx.x % T;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kTeams + team;
    if (unit >= p.unit_start[p.nseg])
        return;
    const int si = N == 1 ? 0 : find_segment(p, unit);
    const ESegK &sg = p.seg[si];
    const int64_t t = unit - p.unit_start[si];
    const int64_t id = load_id(sg.ids, sg.ids_i64, t);
    const int nu = sg.nu, cols = sg.cols;
    const bool named = id >= 0 && id < sg.vocab;
    const WT *w = static_cast<const WT *>(sg.w) + (named ? id * sg.ld : 0);
    Raw8<WT> row[KK];
    if constexpr (K > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            row[k].load(w + 8 * (k * T + lane), named ? cols - 8 * (k * T + lane) : 0);
    }
    const float g = named && sg.unit && sg.gain ? __ldg(sg.gain + (sg.gain_scalar ? 0 : id)) : 1.f;
    if (id >= sg.vocab && lane == 0)
        raise_device_error(DS_ERR_INVALID_ARG, kSiteEmbedId);
    YT *y = static_cast<YT *>(sg.y) + t * sg.ld_y;
    float v[KK][8];
    if constexpr (K > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[k][i] = row[k].get(i);
    }
    float f = named ? g * sg.radius : 0.f, pre = 1.f;
    if (named && sg.unit) { // uniform in the team
        TeamRed<T> red(scratch[team]);
        float S[1] = {0.f};
        auto each = [&](auto &&fn) {
            if constexpr (K > 0) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        fn(v[k][i]);
            } else {
                for (int o = lane; o < nu; o += T) {
                    load8(w + 8 * o, v[0], cols - 8 * o);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        fn(v[0][i]);
                }
            }
        };
        each([&](float a) { S[0] = fmaf(a, a, S[0]); });
        red.sum(S);
        const RowScale rs = row_scale(S[0], p.eps, red, each);
        f *= rs.inv;
        pre = rs.pre;
    }
    if constexpr (K > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int o = k * T + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[k][i] = (v[k][i] * pre) * f;
            store8(y + 8 * o, v[k], cols - 8 * o);
        }
    } else {
        for (int o = lane; o < nu; o += T) {
            load8(w + 8 * o, v[0], named ? cols - 8 * o : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[0][i] = (v[0][i] * pre) * f;
            store8(y + 8 * o, v[0], cols - 8 * o);
        }
    }
}

// --------------------------------------------------------------- grouping --

constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kPer = 4;             // consecutive ids of a lane
constexpr int kSpan = 32 * kPer;    // of a warp
constexpr int kList = 8192;         // matches that shared memory holds
constexpr int kGroupSmemFixed = kList * 8;

__device__ __forceinline__ void load_ids(const void *ids, int i64, int64_t at, int64_t n, bool vec, int64_t (&v)[kPer])
{
    if (at + kPer <= n && vec) {
        if (i64) {
            const longlong2 a = __ldg(reinterpret_cast<const longlong2 *>(static_cast<const int64_t *>(ids) + at));
            const longlong2 b = __ldg(reinterpret_cast<const longlong2 *>(static_cast<const int64_t *>(ids) + at) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        } else {
            const int4 a = __ldg(reinterpret_cast<const int4 *>(static_cast<const int32_t *>(ids) + at));
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        v[i] = at + i < n ? load_id(ids, i64, at + i) : -1;
}

// Inclusive scan of two counts over the block (packed: tokens low, items high).
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *warp_tot, uint64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += n;
    }
    if (lane == 31)
        warp_tot[warp] = v;
    __syncthreads();
    uint64_t w = warp_tot[lane]; // kGroupWarps = 32: a warp total per lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t n = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o)
            w += n;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const uint64_t below = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    __syncthreads();
    return v + (warp > 0 ? below : 0);
}

// Each warp takes a span of consecutive ids, so that the order of the tokens is
// kept without barriers: lanes by ballots, warps by a scan of their counts.
__global__ void __launch_bounds__(kGroupThreads) k_embed_group(const __grid_constant__ EGroupParams p)
{
    extern __shared__ __align__(128) unsigned char dyn[]; // (every kernel of the file declares it alike)
    int *cnt = reinterpret_cast<int *>(dyn + kGroupSmemFixed); // tokens of each row, then the next place
    __shared__ uint64_t warp_tot[kGroupWarps];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int64_t T = p.tokens;
    const int R = static_cast<int>((p.vocab - b + kEmbedBuckets - 1) / kEmbedBuckets); // rows b, b + 128, ...
    const bool vec = (reinterpret_cast<uintptr_t>(p.ids) & 15) == 0;
    const int64_t span = (T + kGroupWarps * kSpan - 1) / (kGroupWarps * kSpan) * kSpan;
    const int64_t from = min(T, warp * span), to = min(T, from + span);

    for (int r = tid; r < R; r += kGroupThreads)
        cnt[r] = 0;
    __syncthreads();
    // count this CTA's tokens by row, and those of the CTAs below
    uint64_t low = 0, hits = 0;
#pragma unroll 4
    for (int64_t at = from + lane * kPer; at < to; at += kSpan) {
        int64_t v[kPer];
        load_ids(p.ids, p.ids_i64, at, to, vec, v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int bucket = static_cast<int>(v[i] & (kEmbedBuckets - 1));
            if (v[i] >= p.vocab) {
                if (b == 0)
                    raise_device_error(DS_ERR_INVALID_ARG, kSiteEmbedId);
            } else if (v[i] >= 0) {
                low += bucket < b;
                if (bucket == b) {
                    ++hits;
                    atomicAdd(&cnt[v[i] / kEmbedBuckets], 1);
                }
            }
        }
    }
    uint64_t all; // (the scan's barriers also close the counting)
    const uint64_t upto = block_scan((low << 32) | hits, warp_tot, all); // both below 2^31
    const int base = static_cast<int>(all >> 32), matches = static_cast<int>(all & 0xffffffffu);
    // this warp's first match in the list: the scan up to lane 0, without it
    const int first = static_cast<int>((__shfl_sync(0xffffffffu, upto, 0) & 0xffffffffu)) -
                      static_cast<int>(__shfl_sync(0xffffffffu, hits, 0));

    // rows' places, their items and the map of named rows
    uint64_t run = 0; // tokens (low) and items (high) of the rows before
    const int words = (R + 31) / 32;
    for (int r0 = 0; r0 < R; r0 += kGroupThreads) {
        const int r = r0 + tid;
        const int n = r < R ? cnt[r] : 0;
        const int ch = embed_chunk(n, p.l), nch = n ? (n + ch - 1) / ch : 0;
        uint64_t tot;
        const uint64_t incl = run + block_scan((static_cast<uint64_t>(nch) << 32) | static_cast<uint32_t>(n), warp_tot, tot);
        run += tot;
        const uint32_t named = __ballot_sync(0xffffffffu, n > 0);
        if (lane == 0 && r / 32 < words)
            p.named[static_cast<int64_t>(b) * p.named_ld + r / 32] = named;
        if (n > 0) {
            const int start = base + static_cast<int>(incl & 0xffffffffu) - n;
            const int item0 = base + static_cast<int>(incl >> 32) - nch;
            for (int c = 0; c < nch; ++c)
                p.items[item0 + c] = make_int4(r * kEmbedBuckets + b, start, n, c);
            if (nch > 1) {
                for (int c = 0; c < nch; c += kEmbedJoin)
                    p.arrived[embed_line(start + c * ch, c == 0, p.l)] = 0;
                p.arrived[p.lines + embed_line(start, true, p.l)] = 0;
            }
            cnt[r] = start;
        }
    }
    if (tid == 0)
        p.nitems[b] = make_int2(base, static_cast<int>(run >> 32));

    // (row of this CTA, token) in the tokens' order
    int2 *list = matches <= kList ? reinterpret_cast<int2 *>(dyn) : p.list + base;
    int next = first;
#pragma unroll 4
    for (int64_t at0 = from; at0 < to; at0 += kSpan) {
        const int64_t at = at0 + lane * kPer;
        int64_t v[kPer];
        load_ids(p.ids, p.ids_i64, at, to, vec, v);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!(v[i] >= 0 && v[i] < p.vocab && static_cast<int>(v[i] & (kEmbedBuckets - 1)) == b))
                v[i] = -1;
            mine += v[i] >= 0;
        }
        if (!__any_sync(0xffffffffu, mine > 0))
            continue;
        int place = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, place, o);
            place += lane >= o ? n : 0;
        }
        const int tot = __shfl_sync(0xffffffffu, place, 31);
        place += next - mine;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (v[i] >= 0)
                list[place++] = make_int2(static_cast<int>(v[i] / kEmbedBuckets), static_cast<int>(at + i));
        next += tot;
    }
    __syncthreads();

    // one warp gives each match its place, the next 32 read ahead (equal rows in
    // one step are told apart by match_any)
    if (warp == 0) {
        int2 m = lane < matches ? list[lane] : make_int2(-1 - lane, 0);
        for (int i0 = 0; i0 < matches; i0 += 32) {
            const int2 now = m;
            m = i0 + 32 + lane < matches ? list[i0 + 32 + lane] : make_int2(-1 - lane, 0);
            const uint32_t same = __match_any_sync(0xffffffffu, now.x);
            const int before = __popc(same & below);
            const int at = now.x >= 0 ? cnt[now.x] : 0;
            __syncwarp();
            if (now.x >= 0) {
                p.order[at + before] = now.y;
                if (before == 0)
                    cnt[now.x] = at + __popc(same);
            }
            __syncwarp();
        }
    }
}

// -------------------------------------------------------------- reduction --

// The eight consumer warps of k_embed_reduce, without its other warps.
constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;

__device__ __forceinline__ void sum_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSumThreads) : "memory"); }

// Whether every consumer thread says so.
__device__ __forceinline__ bool sum_all(bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(ok)), "n"(kSumThreads)
                 : "memory");
    return r != 0;
}

// Sums over the consumer threads: the same bits for all (an xor butterfly in the
// warp, then the warps in order).
struct SumRed {
    float *sm; // [2][kSumWarps][2]
    int slot = 0;
    template <int N, class Op>
    __device__ __forceinline__ void across(float (&v)[N], Op op)
    {
        float *s = sm + slot * (2 * kSumWarps);
        slot ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i)
                s[(threadIdx.x >> 5) * 2 + i] = v[i];
        sum_barrier();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = s[i];
#pragma unroll
            for (int w = 1; w < kSumWarps; ++w)
                t = op(t, s[w * 2 + i]);
            v[i] = t;
        }
    }
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N])
    {
        warp_sum(v);
        across(v, [](float a, float b) { return a + b; });
    }
    __device__ __forceinline__ float max(float v)
    {
        float a[1] = {warp_max(v)};
        across(a, [](float x, float y) { return fmaxf(x, y); });
        return a[0];
    }
    __device__ __forceinline__ bool any(bool b) const { return b; } // sums are uniform
};

// An octet of a row in shared memory; columns at and past `valid` read 0.
__device__ __forceinline__ void smem8(const float *p, float (&v)[8], int valid)
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    if (valid < 8)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < valid ? v[i] : 0.f;
}
__device__ __forceinline__ void smem8(const bf16_t *p, float (&v)[8], int valid)
{
    uint4 a = *reinterpret_cast<const uint4 *>(p);
    if (valid < 8)
        a = valid > 0 ? mask_octet(a, valid) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = bf_get(a, i);
}

// Row v's gradient from its sums G, octet u = k T + tid of a team of T threads.
// w: the row in shared memory (unit rows).
template <class WT, int F, int T, class Red>
__device__ __forceinline__ void finish_row(const EGradParams &p, int64_t v, float (&G)[F][8], const WT *w, float gain,
                                           Red &red, int tid)
{
    const int cols = p.cols;
    float *gw = p.grad_w + v * p.ld_g;
    auto put = [&](int k, float (&o)[8]) {
        const int u = k * T + tid;
        if (p.accumulate) {
            float old[8];
            load8_plain(gw + 8 * u, old, cols - 8 * u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] += old[i];
        }
        store8(gw + 8 * u, o, cols - 8 * u);
    };
    if (!p.unit) {
#pragma unroll
        for (int k = 0; k < F; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                G[k][i] *= p.radius;
            put(k, G[k]);
        }
        return;
    }
    float x[F][8];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < F; ++k) {
        const int u = k * T + tid;
        if (8 * u < cols) {
            smem8(w + 8 * u, x[k], cols - 8 * u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[k][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[0] = fmaf(x[k][i], x[k][i], s[0]);
            s[1] = fmaf(x[k][i], G[k][i], s[1]);
        }
    }
    red.sum(s);
    // rows whose fp32 sums overflow or vanish: w scaled by 2^m first (the
    // unit row w / n is the same; grad_w takes the factor back)
    float Ss = s[0];
    auto each = [&](auto &&fn) {
#pragma unroll
        for (int k = 0; k < F; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                fn(x[k][i]);
    };
    const int m = rescale_exponent(s[0], p.eps, red, each, Ss);
    float eps = p.eps;
    if (m != 0) { // uniform
        eps = scalbnf(p.eps, 2 * m);
        s[0] = Ss;
        s[1] = 0.f;
#pragma unroll
        for (int k = 0; k < F; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[k][i] = scalbnf(x[k][i], m);
                s[1] = fmaf(x[k][i], G[k][i], s[1]);
            }
        float d[1] = {s[1]};
        red.sum(d);
        s[1] = d[0];
    }
    const float n2 = s[0] + eps;
    const float inv = 1.0f / sqrtf(n2);
    const float f = scalbnf(gain * p.radius * inv, m), q = s[1] / n2;
    if (p.grad_g && tid == 0) {
        const float gg = p.radius * s[1] * inv;
        p.grad_g[v] = p.accumulate ? p.grad_g[v] + gg : gg;
    }
#pragma unroll
    for (int k = 0; k < F; ++k) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = f * fmaf(-x[k][i], q, G[k][i]);
        put(k, o);
    }
}

// What a stage of the ring holds.
struct StageHead {
    int tokens;    // rows of dy (0: the row of w; -1: the end)
    int row;       // the row of the table
    int start;     // place of the row's first token
    int n;         // the row's tokens
    int chunk;     // which of its chunks this is
    int last;      // 1: the chunk's last tokens
    float gain;
    int pad;
};

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// The chunks of all lists in one numbering: first[b] is list b's first, base[b]
// the place of its records (one warp).
__device__ __forceinline__ void number_items(const EGradParams &p, int *first, int *base, int lane)
{
    int run = 0;
    for (int i0 = 0; i0 < kEmbedBuckets; i0 += 32) {
        const int2 c = p.nitems[i0 + lane];
        int v = c.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += n;
        }
        first[i0 + lane] = run + v - c.y;
        base[i0 + lane] = c.x;
        run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0)
        first[kEmbedBuckets] = run;
}

// The record of chunk `it`: row, place of its first token, its tokens, chunk.
__device__ __forceinline__ int4 item_of(const EGradParams &p, const int *first, const int *base, int it)
{
    int lo = 0, hi = kEmbedBuckets - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= it)
            lo = mid;
        else
            hi = mid - 1;
    }
    return p.items[base[lo] + it - first[lo]];
}

// Zeros to the rows that no token named, a lane a row, from a buffer of zeros in
// shared memory by bulk copies (one warp of each block).
__device__ __forceinline__ void zero_rows(const EGradParams &p, const float *zero, int lane)
{
    const uint32_t bytes = static_cast<uint32_t>(p.cols) * 4 / 16 * 16;
    for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * 32; v0 < p.vocab; v0 += static_cast<int64_t>(gridDim.x) * 32) {
        const int64_t v = v0 + lane;
        if (v >= p.vocab)
            break;
        const int64_t b = v & (kEmbedBuckets - 1), r = v / kEmbedBuckets;
        if ((p.named[b * p.named_ld + r / 32] >> (r & 31)) & 1u)
            continue;
        float *gw = p.grad_w + v * p.ld_g;
        for (uint32_t at = 0; at < bytes; at += kEmbedZeros)
            bulk_s2g(reinterpret_cast<char *>(gw) + at, zero, min(static_cast<uint32_t>(kEmbedZeros), bytes - at));
        for (int c = bytes / 4; c < p.cols; ++c)
            gw[c] = 0.f;
        if (p.grad_g)
            p.grad_g[v] = 0.f;
    }
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// A chunk of a row with several: its sums to the workspace.  Whoever comes last
// of eight chunks adds these in order, whoever comes last of the eights adds
// theirs.  Returns (uniform in the team) whether G now is the whole row's.
// tell(f): f() of the team's first thread, for all.
template <int F, int T, class Barrier, class Tell>
__device__ __forceinline__ bool join_chunks(const EGradParams &p, float (&G)[F][8], int start, int n, int chunk, int tid,
                                            Barrier barrier, Tell tell)
{
    constexpr int kAtOnce = F >= 8 ? 1 : 8 / F; // lines on their way
    const int ch = embed_chunk(n, p.l), nch = (n + ch - 1) / ch;
    if (nch == 1)
        return true;
    auto line = [&](int c) { return embed_line(start + c * ch, c == 0, p.l); };
    auto leave = [&](int c) {
        float *to = p.lines + line(c) * p.line_ld;
#pragma unroll
        for (int k = 0; k < F; ++k) {
            const int u = k * T + tid;
            if (8 * u < p.cols)
                store8(to + 8 * u, G[k], 8);
        }
        __threadfence();
        barrier();
    };
    auto add = [&](int first, int count, int stride) { // lines first, first + stride, ... in order
        __threadfence();
#pragma unroll
        for (int k = 0; k < F; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                G[k][i] = 0.f;
        for (int c0 = 0; c0 < count; c0 += kAtOnce) {
            float4 a[kAtOnce][F], b[kAtOnce][F];
#pragma unroll
            for (int c = 0; c < kAtOnce; ++c) {
                const float *from = p.lines + line(first + min(c0 + c, count - 1) * stride) * p.line_ld;
#pragma unroll
                for (int k = 0; k < F; ++k) {
                    const int u = k * T + tid;
                    a[c][k] = b[c][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (8 * u < p.cols && c0 + c < count) {
                        a[c][k] = __ldcg(reinterpret_cast<const float4 *>(from + 8 * u));
                        b[c][k] = __ldcg(reinterpret_cast<const float4 *>(from + 8 * u) + 1);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
                for (int k = 0; k < F; ++k) {
                    G[k][0] += a[c][k].x, G[k][1] += a[c][k].y, G[k][2] += a[c][k].z, G[k][3] += a[c][k].w;
                    G[k][4] += b[c][k].x, G[k][5] += b[c][k].y, G[k][6] += b[c][k].z, G[k][7] += b[c][k].w;
                }
        }
    };
    const int g = chunk / kEmbedJoin * kEmbedJoin, members = min(kEmbedJoin, nch - g);
    leave(chunk);
    if (!tell([&]() { return atomicAdd(&p.arrived[line(g)], 1) == members - 1; }))
        return false;
    add(g, members, 1);
    const int groups = (nch + kEmbedJoin - 1) / kEmbedJoin;
    if (groups == 1)
        return true;
    leave(g);
    if (!tell([&]() { return atomicAdd(&p.arrived[p.nlines + line(0)], 1) == groups - 1; }))
        return false;
    add(0, groups, kEmbedJoin);
    return true;
}

struct WarpRed {
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) const { warp_sum(v); }
    __device__ __forceinline__ float max(float v) const { return warp_max(v); }
    __device__ __forceinline__ bool any(bool b) const { return b; } // sums are uniform
};

// Rows of at most 1024 columns: a warp per chunk (K octets a lane), eight and a
// warp of zeros per block, no barrier between them.  Each warp copies the rows
// it needs next (the chunk's rows of dy, the row of w, then the next chunk's)
// into a ring of its own.  A block per chunk, as below, takes 1.9 us from chunk
// to chunk however short the rows: 16,384 tokens of 768 columns in 32,000 rows
// took 77 us that way (102 us with every token as frequent), 63 us (50) this way.
template <class WT, class DT, int K>
__global__ void __launch_bounds__(kSumThreads + 32, 2) k_embed_reduce_warp(const __grid_constant__ EGradParams p)
{
    __shared__ int first[kEmbedBuckets + 1], base[kEmbedBuckets];
    __shared__ uint64_t full[kSumWarps][kEmbedSlots];
    extern __shared__ __align__(128) unsigned char dyn[];
    float *zero = reinterpret_cast<float *>(dyn + kSumWarps * p.stages * p.stage);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = p.cols;
    if (warp == 0)
        number_items(p, first, base, lane);
    if (warp < kSumWarps && lane < p.stages)
        mbar_init(&full[warp][lane], 1);
    mbar_init_fence();
    for (int i = tid; i < kEmbedZeros / 16; i += kSumThreads + 32)
        reinterpret_cast<float4 *>(zero)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    fence_proxy_async_smem(); // the zeros are read by bulk copies
    __syncthreads();
    if (warp == kSumWarps) {
        if (!p.accumulate)
            zero_rows(p, zero, lane);
        return;
    }
    const int total = first[kEmbedBuckets];
    const int step = gridDim.x * kSumWarps, mine = blockIdx.x * kSumWarps + warp;
    unsigned char *ring = dyn + warp * p.stages * p.stage;
    uint64_t *bar = full[warp];
    const uint32_t dyb = (static_cast<uint32_t>(cols) * sizeof(DT) + 15) / 16 * 16;
    const uint32_t wb = (static_cast<uint32_t>(cols) * sizeof(WT) + 15) / 16 * 16;

    // 32 chunks' records at a time, a lane each: one set for the copies that run
    // ahead, one for the sums
    struct Batch {
        int4 item;
        int token;
        float gain;
    };
    auto batch = [&](int it0, bool tokens) {
        Batch b{make_int4(0, 0, 0, 0), 0, 1.f};
        const int64_t it = it0 + static_cast<int64_t>(lane) * step;
        if (it < total) {
            b.item = item_of(p, first, base, static_cast<int>(it));
            if (tokens)
                b.token = p.order[b.item.y + b.item.w * embed_chunk(b.item.z, p.l)];
            else if (p.gain)
                b.gain = __ldg(p.gain + (p.gain_scalar ? 0 : b.item.x));
        }
        return b;
    };
    // the copies: chunk pi of this warp, its token pj
    const int count = mine < total ? (total - mine + step - 1) / step : 0;
    int pi = 0, pj = 0, pn = 0, pfrom = 0, prow = 0, ptok = 0;
    int flying = 0, to = 0, at = 0, phase = 0; // copies on their way; the next slot to fill and to read, its phase
    Batch pb = batch(mine, true);
    auto open = [&]() { // chunk pi's fields
        if (pi > 0 && pi % 32 == 0)
            pb = batch(mine + pi * step, true);
        const int k = pi & 31;
        prow = __shfl_sync(0xffffffffu, pb.item.x, k);
        const int start = __shfl_sync(0xffffffffu, pb.item.y, k), n = __shfl_sync(0xffffffffu, pb.item.z, k);
        const int chunk = __shfl_sync(0xffffffffu, pb.item.w, k), ch = embed_chunk(n, p.l);
        pfrom = start + chunk * ch;
        pn = min(ch, n - chunk * ch);
        ptok = __shfl_sync(0xffffffffu, pb.token, k);
    };
    auto ahead = [&]() { // as many copies as the ring has room for
        while (flying < p.stages && pi < count) {
            if (pj == 0)
                open();
            const void *src;
            uint32_t bytes;
            if (pj < pn) {
                if (pn > 1 && pj % 32 == 0)
                    ptok = pj + lane < pn ? p.order[pfrom + pj + lane] : 0;
                const int64_t t = __shfl_sync(0xffffffffu, ptok, pn > 1 ? pj % 32 : 0);
                src = static_cast<const DT *>(p.dy) + t * p.ld_y;
                bytes = dyb;
            } else {
                src = static_cast<const WT *>(p.w) + static_cast<int64_t>(prow) * p.ld;
                bytes = wb;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar[to], bytes);
                bulk_g2s(ring + to * p.stage, src, bytes, &bar[to]);
            }
            ++flying;
            to = to + 1 == p.stages ? 0 : to + 1;
            if (++pj == pn + (p.unit ? 1 : 0)) {
                pj = 0;
                ++pi;
            }
        }
    };
    bool ok = true;
    auto arrives = [&]() { // the next copy
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[at], phase, p.wait_limit_ns));
        return ok;
    };
    auto release = [&]() { // the slot that was read
        __syncwarp();
        --flying;
        if (++at == p.stages) {
            at = 0;
            phase ^= 1;
        }
    };
    ahead();
    Batch cb = batch(mine, false);
    WarpRed red;
    for (int ci = 0; ci < count && ok; ++ci) {
        if (ci > 0 && ci % 32 == 0)
            cb = batch(mine + ci * step, false);
        const int k32 = ci & 31;
        const int row = __shfl_sync(0xffffffffu, cb.item.x, k32), start = __shfl_sync(0xffffffffu, cb.item.y, k32);
        const int n = __shfl_sync(0xffffffffu, cb.item.z, k32), chunk = __shfl_sync(0xffffffffu, cb.item.w, k32);
        const float gain = __shfl_sync(0xffffffffu, cb.gain, k32);
        const int ch = embed_chunk(n, p.l), nj = min(ch, n - chunk * ch);
        float G[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                G[k][i] = 0.f;
        for (int j = 0; j < nj; ++j) {
            if (!arrives())
                break;
            const DT *d = reinterpret_cast<const DT *>(ring + at * p.stage);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int u = k * 32 + lane;
                if (8 * u < cols) {
                    float x[8];
                    smem8(d + 8 * u, x, cols - 8 * u);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[k][i] += x[i];
                }
            }
            release();
            ahead();
        }
        if (!ok)
            break;
        const bool whole = join_chunks<K, 32>(p, G, start, n, chunk, lane, []() { __syncwarp(); }, [&](auto f) {
            int b = 0;
            if (lane == 0)
                b = f();
            return __shfl_sync(0xffffffffu, b, 0) != 0;
        });
        const WT *w = nullptr;
        if (p.unit) {
            if (!arrives())
                break;
            w = reinterpret_cast<const WT *>(ring + at * p.stage);
        }
        if (whole)
            finish_row<WT, K, 32>(p, row, G, w, gain, red, lane);
        if (p.unit) {
            release();
            ahead();
        }
    }
    if (!ok) { // a copy did not come: none may be in flight at the end
        if (lane == 0)
            raise_device_error(DS_ERR_DEVICE_TIMEOUT, kSiteEmbedWait);
        while (flying > 0) {
            mbar_wait_bounded(&bar[at], phase, drain_limit(p.wait_limit_ns));
            release();
        }
    }
}

// Longer rows: eight consumer warps, a producer warp and a warp of zeros per block.
//  * The producer walks the block's chunks, 32 at a time (a lane looks up one
//    each), and copies the rows of dy that they name, then the row of w, into
//    a ring of stages of `stage` bytes: a row of dy, or as many as fit.
//  * The consumers add.  S slots of L threads (K octets a thread) take every
//    S-th token of a stage; at the chunk's end the slots are added in order, one
//    octet or (S = 1) K octets a thread, which also is the layout of the finish.
//  * The third kind writes zeros to the rows that no token named, from a
//    buffer in shared memory by bulk copies, beside the sums.
template <class WT, class DT, int L, int K>
__global__ void __launch_bounds__(kSumThreads + 64) k_embed_reduce(const __grid_constant__ EGradParams p)
{
    constexpr int T = kSumThreads, S = T / L, F = S == 1 ? K : 1;
    static_assert(L * K <= T * F, "the finish holds every octet");
    __shared__ float scratch[4 * kSumWarps];
    __shared__ int first[kEmbedBuckets + 1], base[kEmbedBuckets];
    __shared__ StageHead head[kEmbedStages];
    __shared__ uint64_t full[kEmbedStages], empty[kEmbedStages];
    __shared__ int last_flag;
    extern __shared__ __align__(128) unsigned char dyn[];
    unsigned char *ring = dyn;                                                  // [stages][stage]
    float *zero = reinterpret_cast<float *>(dyn + p.stages * p.stage);          // [kEmbedZeros bytes]
    float *slots = zero + kEmbedZeros / 4;                                      // S > 1: [S][L K 8]
    const int tid = threadIdx.x, wl = tid & 31;
    const int cols = p.cols;
    if (tid < 32)
        number_items(p, first, base, wl);
    if (tid == 32) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kSumWarps);
        }
        mbar_init_fence();
    }
    for (int i = tid; i < kEmbedZeros / 16; i += T + 64)
        reinterpret_cast<float4 *>(zero)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    fence_proxy_async_smem(); // the zeros are read by bulk copies
    __syncthreads();
    const int total = first[kEmbedBuckets];

    if (tid >= T + 32) { // zeros
        if (!p.accumulate)
            zero_rows(p, zero, wl);
        return;
    }

    if (tid >= T) { // the producer
        bool ok = true;
        int st = 0, phase = 0, sent = 0;
        const uint32_t dyb = (static_cast<uint32_t>(cols) * sizeof(DT) + 15) / 16 * 16;
        const uint32_t wb = (static_cast<uint32_t>(cols) * sizeof(WT) + 15) / 16 * 16;
        const int per = p.per_stage;
        // a free stage, its head filled in and its bytes expected (lane 0)
        auto open = [&](const StageHead &h, uint32_t bytes) {
            if (sent >= p.stages) {
                if (wl == 0 && !mbar_wait_bounded(&empty[st], phase ^ 1, p.wait_limit_ns)) {
                    raise_device_error(DS_ERR_DEVICE_TIMEOUT, kSiteEmbedWait);
                    ok = false;
                }
                ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
                if (!ok)
                    return false;
            }
            if (wl == 0) {
                head[st] = h;
                mbar_arrive_expect_tx(&full[st], bytes);
            }
            __syncwarp();
            return true;
        };
        auto step = [&]() {
            ++sent;
            if (++st == p.stages) {
                st = 0;
                phase ^= 1;
            }
        };
        for (int i0 = blockIdx.x; i0 < total && ok; i0 += 32 * gridDim.x) {
            const int it = i0 + wl * gridDim.x;
            int4 mine = make_int4(0, 0, 0, 0);
            int token = 0;
            float gain = 1.f;
            if (it < total) {
                mine = item_of(p, first, base, it);
                token = p.order[mine.y + mine.w * embed_chunk(mine.z, p.l)];
                if (p.gain)
                    gain = __ldg(p.gain + (p.gain_scalar ? 0 : mine.x));
            }
            for (int k = 0; k < 32 && ok; ++k) {
                if (i0 + k * gridDim.x >= total)
                    break;
                StageHead h;
                h.row = __shfl_sync(0xffffffffu, mine.x, k);
                h.start = __shfl_sync(0xffffffffu, mine.y, k);
                h.n = __shfl_sync(0xffffffffu, mine.z, k);
                h.chunk = __shfl_sync(0xffffffffu, mine.w, k);
                h.gain = __shfl_sync(0xffffffffu, gain, k);
                h.pad = 0;
                const int only = __shfl_sync(0xffffffffu, token, k);
                const int ch = embed_chunk(h.n, p.l), from = h.start + h.chunk * ch, n = min(ch, h.n - h.chunk * ch);
                int tok = 0;
                for (int j = 0; j < n; j += per) { // per divides 32
                    if (j % 32 == 0)
                        tok = n == 1 ? only : j + wl < n ? p.order[from + j + wl] : 0;
                    h.tokens = min(per, n - j);
                    h.last = j + per >= n;
                    if (!open(h, h.tokens * dyb))
                        break;
                    const int64_t t = __shfl_sync(0xffffffffu, tok, (j % 32 + wl) & 31);
                    if (wl < h.tokens)
                        bulk_g2s(ring + st * p.stage + wl * dyb, static_cast<const DT *>(p.dy) + t * p.ld_y, dyb, &full[st]);
                    step();
                }
                if (p.unit && ok) {
                    h.tokens = 0;
                    if (open(h, wb)) {
                        if (wl == 0)
                            bulk_g2s(ring + st * p.stage, static_cast<const WT *>(p.w) + static_cast<int64_t>(h.row) * p.ld, wb,
                                     &full[st]);
                        step();
                    }
                }
            }
        }
        StageHead end{};
        end.tokens = -1;
        if (ok && open(end, 0))
            step();
        if (wl == 0) // no copy may be in flight at the end, whoever stopped waiting
            for (int i = max(0, sent - p.stages); i < sent; ++i)
                mbar_wait_bounded(&full[i % p.stages], (i / p.stages) & 1, drain_limit(p.wait_limit_ns));
        return;
    }

    // the consumers
    SumRed red{scratch};
    const int slot = tid / L, lane = tid % L;
    int st = 0, phase = 0;
    float A[K][8];
    auto clear = [&]() {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                A[k][i] = 0.f;
    };
    clear();
    auto next = [&]() {
        const bool got = mbar_wait_bounded(&full[st], phase, p.wait_limit_ns);
        if (!sum_all(got)) { // uniform
            if (tid == 0)
                raise_device_error(DS_ERR_DEVICE_TIMEOUT, kSiteEmbedWait);
            return false;
        }
        return true;
    };
    auto release = [&]() {
        __syncwarp();
        if (wl == 0)
            mbar_arrive(&empty[st]);
        if (++st == p.stages) {
            st = 0;
            phase ^= 1;
        }
    };
    int taken = 0; // tokens of the chunk so far (which slot takes the next)
    while (next()) {
        const StageHead h = head[st];
        if (h.tokens < 0)
            break;
        const DT *rows = reinterpret_cast<const DT *>(ring + st * p.stage);
        const int dy_ld = (cols * static_cast<int>(sizeof(DT)) + 15) / 16 * 16 / static_cast<int>(sizeof(DT));
        // token j of the chunk belongs to slot j mod S
        for (int j = (slot - taken % S + S) % S; j < h.tokens; j += S) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int u = k * L + lane;
                if (8 * u < cols) {
                    float d[8];
                    smem8(rows + j * dy_ld + 8 * u, d, cols - 8 * u);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        A[k][i] += d[i];
                }
            }
        }
        taken += h.tokens;
        release();
        if (!h.last)
            continue;
        // the chunk is summed
        taken = 0;
        float G[F][8];
        if constexpr (S == 1) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    G[k][i] = A[k][i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                G[0][i] = 0.f;
            // slots without a token hold zeros: adding them changes nothing
            const int used = min(S, min(embed_chunk(h.n, p.l), h.n - h.chunk * embed_chunk(h.n, p.l)));
            if (slot < used)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    store8_smem(slots + (slot * L * K + k * L + lane) * 8, A[k]);
            sum_barrier();
            if (tid < L * K)
                for (int s = 0; s < used; ++s) {
                    float d[8];
                    smem8(slots + (s * L * K + tid) * 8, d, 8);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[0][i] += d[i];
                }
            sum_barrier();
        }
        clear();
        const bool finish = join_chunks<F, T>(p, G, h.start, h.n, h.chunk, tid, []() { sum_barrier(); }, [&](auto f) {
            if (tid == 0)
                last_flag = f();
            sum_barrier();
            return last_flag != 0;
        });
        const WT *w = nullptr;
        if (p.unit) { // its row of w comes next
            if (!next())
                break;
            w = reinterpret_cast<const WT *>(ring + st * p.stage);
        }
        if (finish)
            finish_row<WT, F, T>(p, h.row, G, w, h.gain, red, tid);
        if (p.unit)
            release();
    }
}

template <class WT, class YT, int T, int K>
int launch_rows(const EParams<kLmSegs> &p, int64_t units, cudaStream_t st)
{
    constexpr int threads = T < 128 ? 128 : T;
    const int64_t teams = threads / T, grid64 = (units + teams - 1) / teams;
    const unsigned grid = static_cast<unsigned>(grid64);
    if (p.nseg == 1) {
        EParams<1> one = only_segment(p);
        one.eps = p.eps;
        k_embed<WT, YT, T, K, 1><<<grid, threads, 0, st>>>(one);
    } else {
        k_embed<WT, YT, T, K, kLmSegs><<<grid, threads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

template <class WT, class YT>
int launch_fwd(const EParams<kLmSegs> &p, int cls, int64_t units, cudaStream_t st)
{
    switch (cls) {
    case 0: return launch_rows<WT, YT, 32, 1>(p, units, st);
    case 1: return launch_rows<WT, YT, 32, 2>(p, units, st);
    case 2: return launch_rows<WT, YT, 128, 1>(p, units, st);
    case 3: return launch_rows<WT, YT, 128, 2>(p, units, st);
    case 4: return launch_rows<WT, YT, 256, 2>(p, units, st);
    case 5: return launch_rows<WT, YT, 256, 4>(p, units, st);
    case 6: return launch_rows<WT, YT, 256, 8>(p, units, st);
    default: return launch_rows<WT, YT, 256, 0>(p, units, st);
    }
}

template <class WT, class DT, int L, int K>
int launch_sums(EGradParams p, int sms, cudaStream_t st)
{
    static DeviceFlags done;
    constexpr int S = kSumThreads / L, slots = S > 1 ? S * L * K * 8 * 4 : 0;
    auto *kernel = k_embed_reduce<WT, DT, L, K>;
    if (cudaError_t e = enable_dynamic_smem(kernel, kEmbedSmemMax, done); e != cudaSuccess)
        return e;
    // stages hold the longer of a row of dy and one of w; two blocks an SM
    // where four stages of 16 KB (or fewer) leave room, else one
    auto up = [](int b) { return (b + 15) / 16 * 16; };
    const int dyb = up(p.cols * static_cast<int>(sizeof(DT))), wb = p.unit ? up(p.cols * static_cast<int>(sizeof(WT))) : 0;
    const int need = std::max(dyb, wb);
    p.stage = need <= 16384 ? 16384 : need <= 32768 ? 32768 : 65536;
    p.stages = need <= 16384 ? 5 : need <= 32768 ? 6 : 3;
    p.per_stage = 1; // tokens of a stage: a power of two, at most 32
    while (p.per_stage < 32 && 2 * p.per_stage * dyb <= p.stage)
        p.per_stage *= 2;
    const int smem = p.stages * p.stage + kEmbedZeros + slots;
    const int blocks = sms * (need <= 16384 ? 2 : 1);
    kernel<<<blocks, kSumThreads + 64, smem, st>>>(p);
    return cudaGetLastError();
}

template <class WT, class DT, int K>
int launch_sums_warp(EGradParams p, int sms, cudaStream_t st)
{
    static DeviceFlags done;
    auto *kernel = k_embed_reduce_warp<WT, DT, K>;
    if (cudaError_t e = enable_dynamic_smem(kernel, kEmbedSmemMax, done); e != cudaSuccess)
        return e;
    // a slot holds the longer of a row of dy and one of w; 12 KB of slots a warp
    // let two blocks share an SM
    auto up = [](int b, int to) { return (b + to - 1) / to * to; };
    const int dyb = up(p.cols * static_cast<int>(sizeof(DT)), 16);
    const int wb = p.unit ? up(p.cols * static_cast<int>(sizeof(WT)), 16) : 0;
    p.stage = up(std::max(dyb, wb), 128);
    p.stages = std::min(kEmbedSlots, 12288 / p.stage);
    kernel<<<sms * 2, kSumThreads + 32, kSumWarps * p.stages * p.stage + kEmbedZeros, st>>>(p);
    return cudaGetLastError();
}

template <class WT, class DT>
int launch_grad(const EGradParams &p, int cls, int sms, cudaStream_t st)
{
    switch (cls) {
    case 0: return launch_sums_warp<WT, DT, 1>(p, sms, st);
    case 1: return launch_sums_warp<WT, DT, 2>(p, sms, st);
    case 2: return launch_sums_warp<WT, DT, 4>(p, sms, st);
    case 3: return launch_sums<WT, DT, 128, 2>(p, sms, st);
    case 4: return launch_sums<WT, DT, 256, 2>(p, sms, st);
    case 5: return launch_sums<WT, DT, 256, 4>(p, sms, st);
    default: return launch_sums<WT, DT, 256, 8>(p, sms, st);
    }
}

} // namespace

// Rows by length: (threads, octets per thread) of k_embed, (threads of a slot,
// octets per thread) of k_embed_reduce.
int embed_class(int64_t cols)
{
    const int64_t top[7] = {256, 512, 1024, 2048, 4096, 8192, 16384};
    for (int c = 0; c < 7; ++c)
        if (cols <= top[c])
            return c;
    return 7;
}

int launch_embed(bool w_bf16, bool y_bf16, int cls, const EParams<kLmSegs> &p, int64_t units, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (w_bf16)
        return y_bf16 ? launch_fwd<bf16_t, bf16_t>(p, cls, units, st) : launch_fwd<bf16_t, float>(p, cls, units, st);
    return y_bf16 ? launch_fwd<float, bf16_t>(p, cls, units, st) : launch_fwd<float, float>(p, cls, units, st);
}

int launch_embed_group(const EGroupParams &p, void *stream)
{
    static DeviceFlags done;
    const int rows = static_cast<int>((p.vocab + kEmbedBuckets - 1) / kEmbedBuckets);
    if (cudaError_t e = enable_dynamic_smem(k_embed_group, kGroupSmemFixed + kEmbedMaxRows * 4, done); e != cudaSuccess)
        return e;
    k_embed_group<<<kEmbedBuckets, kGroupThreads, kGroupSmemFixed + rows * 4, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError();
}

int launch_embed_reduce(bool w_bf16, bool dy_bf16, int cls, const EGradParams &p, int sms, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (w_bf16)
        return dy_bf16 ? launch_grad<bf16_t, bf16_t>(p, cls, sms, st) : launch_grad<bf16_t, float>(p, cls, sms, st);
    return dy_bf16 ? launch_grad<float, bf16_t>(p, cls, sms, st) : launch_grad<float, float>(p, cls, sms, st);
}

int embed_read_and_clear_error(uint32_t *code, uint32_t *site) { return module_read_and_clear_error(code, site); }

} // namespace ds
