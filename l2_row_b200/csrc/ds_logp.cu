// ds_logp.cu -- log probabilities of given tokens from rows of logits on
// sm_100a, with the entropy and the top alternatives of each row, and the
// gradient to the logits.
//
// With z = scale x:  lse = log sum exp z,  logp = z_id - lse,
// H = lse - sum p z,  and the k largest logits (equal ones by the lower column).
// Backward:  dx = scale (dlogp ([j = id] - p) - dH p (z - lse + H) + dlse p).
//
// Forward, one read of the logits, which a producer warp streams through a ring
// of shared-memory stages with bulk copies, ahead of the row that is being
// finished (loads into registers left the SM waiting: 174 us instead of 90 for
// 4,096 x 50,257 in bf16 without the top k).  Per element: one fused product
// for its exponent, one exp2, a sum (and a product for H); at bf16 the exp2 unit
// (16 a clock and SM) is busy about 70% of the time the copy takes.
// A step is 64 bytes a thread; the steps of a row make at most 8 groups, and
// the partial results (maximum, sum, sum of exponent times exp) of a thread are
// joined in the order of its steps within a group and of the groups.  When
// there are few rows a cluster of 2, 4 or 8 CTAs takes a row, each CTA some
// groups: the same operations in the same order, so a row's results have the
// same bits in a batch of one and of thousands.
//
// The top k need no second pass over the row: each thread's largest logit is
// known after the first.  A warp of its own takes the largest of 32 sets of
// threads; the k-th of these is a bound that at least k logits reach (for
// k = 20 about 31 do), and only the threads whose largest reaches it have their
// columns read again (out of L2) and put to a list that is then ranked.  A list
// that overflows (equal logits, masked rows) falls back to a scan of the row
// that keeps the best 32.
#include <algorithm>
#include <type_traits>

#include <cuda_runtime.h>

#include "ds_device.cuh"
#include "ds_lm.cuh"

namespace ds {

namespace {

constexpr int kGroups = 8; // groups of steps of a row
constexpr int kUnits = 4;  // 16-byte units of a thread in a step
constexpr int kLogpThreads = 256; // consumers of a row of more than 4096
constexpr int kLogpStages = 4;
template <int NT>
constexpr int kLogpCtas = NT == 128 ? 4 : 2; // CTAs of an SM
constexpr int kCand = 128;  // candidates of the ranking list
constexpr int kAgain = 128; // threads, and groups of threads, that are read again
constexpr int kFinishers = 3;
constexpr float kNegInf = -INFINITY;
constexpr float kFloor = -0x1.92p99f; // bf16 0xF149, about -1e30
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A thread's 64 bytes of a step.
template <class T>
struct Step {
    static constexpr int E = 16 / sizeof(T);       // columns of a unit
    static constexpr int kPairs = kUnits * E / 2;
    uint4 a[kUnits];

    __device__ __forceinline__ uint32_t word(int i) const
    {
        const uint4 &v = a[i / 4];
        return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        if constexpr (sizeof(T) == 2)
            return make_float2(bf_lo(word(i)), bf_hi(word(i)));
        else
            return make_float2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    }
    // Columns at and past `valid` of unit u become -inf.
    __device__ __forceinline__ void mask(int u, int valid)
    {
        uint32_t *w = reinterpret_cast<uint32_t *>(&a[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                if (2 * i >= valid)
                    w[i] = 0xFF80FF80u;
                else if (2 * i + 1 >= valid)
                    w[i] = (w[i] & 0xFFFFu) | 0xFF800000u;
            } else {
                if (i >= valid)
                    w[i] = 0xFF800000u;
            }
        }
    }
    // No column below kFloor; NaN stays.
    __device__ __forceinline__ void floor()
    {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            uint32_t *w = reinterpret_cast<uint32_t *>(&a[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2)
                    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(0xF149F149u));
                else
                    asm("max.NaN.f32 %0, %0, %1;" : "+r"(w[i]) : "r"(0xF1490000u));
            }
        }
    }
    __device__ __forceinline__ float max() const // NaN does not count
    {
        if constexpr (sizeof(T) == 2) {
            __nv_bfloat162 m[2];
#pragma unroll
            for (int i = 0; i < 4 * kUnits; ++i) {
                uint32_t w = word(i);
                const __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162 *>(&w);
                m[i & 1] = i < 2 ? v : __hmax2(m[i & 1], v);
            }
            const __nv_bfloat162 t = __hmax2(m[0], m[1]);
            return fmaxf(__low2float(t), __high2float(t));
        } else {
            float m[2] = {kNegInf, kNegInf};
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                m[i & 1] = fmaxf(m[i & 1], fmaxf(pair(i).x, pair(i).y));
            return fmaxf(m[0], m[1]);
        }
    }
};

// The columns of a 16-byte unit.
template <class T>
__device__ __forceinline__ float unit_value(const uint4 &v, int i)
{
    if constexpr (sizeof(T) == 2)
        return bf_get(v, i);
    else
        return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
}

// s = sum of 2^(x c - r) and w = sum of that times (x c - r), with the reference
// r = fl(m c) of the maximum m.  Everything uses the rounded r, so its rounding
// cancels.  Where r is so large that its rounding is no small exponent any more
// (2^24: up to 1), or leaves fp32 (a mask of the type's lowest value), the
// reference is m c itself and the exponents are (x - m) c.
struct Acc {
    float m, r, s, w;
};

constexpr float kFar = 0x1p24f;

__device__ __forceinline__ Acc no_acc() { return {kNegInf, kNegInf, 0.f, 0.f}; }
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) < INFINITY; }
__device__ __forceinline__ bool is_near(float r) { return fabsf(r) < kFar; }

// The exponent that takes sums of maximum m and rounded product r to the
// reference of maximum om >= m (its rounded product: orf), in any case.
__device__ __noinline__ float far_shift(float m, float r, float om, float orf, float c)
{
    if (is_near(r) && is_near(orf))
        return r - orf;
    if (m == kNegInf) // sums of 0
        return -1e30f;
    const float d = is_near(r) ? fmaf(-om, c, r) : is_near(orf) ? fmaf(m, c, -orf) : (m - om) * c;
    return fmaxf(d, -1e30f);
}

template <bool ENT>
__device__ __forceinline__ Acc joined(const Acc &a, const Acc &b, float c)
{
    Acc o;
    o.m = fmaxf(a.m, b.m);
    o.r = fmaxf(a.r, b.r);
    float da = a.r - o.r, db = b.r - o.r;
    if (!(is_near(a.r) && is_near(b.r))) {
        da = far_shift(a.m, a.r, o.m, o.r, c);
        db = far_shift(b.m, b.r, o.m, o.r, c);
    }
    const float fa = ex2(da), fb = ex2(db);
    o.s = fmaf(b.s, fb, a.s * fa);
    o.w = ENT ? fmaf(fmaf(db, b.s, b.w), fb, fmaf(da, a.s, a.w) * fa) : 0.f;
    return o;
}

// A whole step of a thread.  FLOOR: logits below kFloor (masked ones) count as
// kFloor, where their exp is 0 but their exponent finite (see holds_floor); the
// others, and so a step without masked ones, give the same bits either way.
template <bool ENT, bool FLOOR, class T>
__device__ __forceinline__ Acc step_acc(Step<T> &x, float c)
{
    if (FLOOR)
        x.floor();
    Acc o;
    o.m = x.max();
    o.r = __fmul_rn(o.m, c); // (never fused into what it is subtracted from)
    const float2 cc = make_float2(c, c), rr = make_float2(-o.r, -o.r);
    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, w[2] = {s[0], s[0]};
#pragma unroll
    for (int i = 0; i < Step<T>::kPairs; ++i) {
        const float2 y = __ffma2_rn(x.pair(i), cc, rr);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        s[i & 1] = __fadd2_rn(s[i & 1], e);
        if (ENT)
            w[i & 1] = __ffma2_rn(e, y, w[i & 1]);
    }
    s[0] = __fadd2_rn(s[0], s[1]);
    o.s = s[0].x + s[0].y;
    o.w = 0.f;
    if (ENT) {
        w[0] = __fadd2_rn(w[0], w[1]);
        o.w = w[0].x + w[0].y;
    }
    return o;
}

// A step whose exponents are finite, its masked logits at kFloor with exp 0.
__device__ __forceinline__ bool holds_floor(const Acc &a, float c) { return is_near(a.r) && (a.m - kFloor) * c > 200.f; }

// The columns of one unit that lie in the row (valid of E), in any case:
// masked logits (0 times -inf), a maximum of -inf or a far one.
template <bool ENT, class T>
__device__ __forceinline__ Acc unit_acc(const uint4 &v, int valid, float c)
{
    constexpr int E = 16 / sizeof(T);
    Acc o = no_acc();
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < valid)
            o.m = fmaxf(o.m, unit_value<T>(v, i));
    o.r = __fmul_rn(o.m, c); // (never fused into what it is subtracted from)
    const bool far = !is_near(o.r); // (a maximum of -inf: no sums)
    const float m = o.m == kNegInf ? 0.f : o.m, r = o.m == kNegInf ? 0.f : o.r;
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < valid) {
            const float f = unit_value<T>(v, i);
            const float y = far ? (f - m) * c : fmaf(f, c, -r), e = ex2(y);
            o.s += e;
            if (ENT)
                o.w = fmaf(e, fmaxf(y, -1e4f), o.w);
        }
    return o;
}

// Whether a step's sums stand: 0 times the exponent of a masked logit is no
// number, and a far maximum (or -inf) wants other exponents.
template <bool ENT>
__device__ __forceinline__ bool is_plain(const Acc &a) { return is_near(a.r) && !(ENT && a.w != a.w); }

// A step in any case, out of the common path: the row's end, masked logits,
// far maxima.  left: columns of the row from this thread's first on.
template <bool ENT, class T, int NT>
__device__ __noinline__ Acc careful_acc(const uint4 *from, int left, float c)
{
    constexpr int E = 16 / sizeof(T);
    Step<T> v;
    auto read = [&]() {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            v.a[u] = from[u * NT];
            if (left - u * NT * E < E) // the row ends in it, or before
                v.mask(u, left - u * NT * E);
        }
    };
    if (left <= 0)
        return no_acc();
    read();
    Acc a = step_acc<ENT, true>(v, c);
    if (holds_floor(a, c) && a.w == a.w)
        return a;
    // what the common path would have given, so that a thread's result depends
    // on its columns alone, not on how its warp came here
    read();
    a = step_acc<ENT, false>(v, c);
    if (is_plain<ENT>(a))
        return a;
    a = no_acc();
#pragma unroll 1
    for (int u = 0; u < kUnits; ++u) {
        const int valid = left - u * NT * E;
        if (valid > 0)
            a = joined<ENT>(a, unit_acc<ENT, T>(from[u * NT], valid, c), c);
    }
    return a;
}

// --------------------------------------------------------------- the top k --

// Order of logits as integers: NaN last (0), -inf next, +0 and -0 equal.
__device__ __forceinline__ uint32_t rank_bits(float x)
{
    if (x != x)
        return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ unsigned long long key_of(float x, int col)
{
    return (static_cast<unsigned long long>(rank_bits(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(col));
}

// The logit back from its order (NaN from 0).
__device__ __forceinline__ float unranked(uint32_t u)
{
    return u == 0 ? NAN : __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

// Bitonic sort of one value per lane, largest in lane 0.
__device__ __forceinline__ uint32_t warp_sort_desc(uint32_t v, int lane)
{
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
            const bool up = ((lane & k) == 0) == ((lane & j) == 0); // keeps the larger
            v = up ? max(v, o) : min(v, o);
        }
    return v;
}

__device__ __forceinline__ unsigned long long kmax(unsigned long long a, unsigned long long b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned long long kmin(unsigned long long a, unsigned long long b) { return a > b ? b : a; }

// Bitonic sort of one key per lane, largest in lane 0.
__device__ __forceinline__ unsigned long long warp_sort_desc(unsigned long long v, int lane)
{
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, j);
            v = ((lane & k) == 0) == ((lane & j) == 0) ? kmax(v, o) : kmin(v, o);
        }
    return v;
}

// The best 32 of two lists, each sorted over the lanes.
__device__ __forceinline__ unsigned long long warp_merge_desc(unsigned long long a, unsigned long long b, int lane)
{
    a = kmax(a, __shfl_sync(0xffffffffu, b, 31 - lane)); // the best 32, falling then rising
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, a, j);
        a = (lane & j) == 0 ? kmax(a, o) : kmin(a, o);
    }
    return a;
}

template <class T>
__device__ __forceinline__ float logit(const T *x, int64_t col)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float(static_cast<uint32_t>(x[col].bits) << 16);
    else
        return x[col];
}

struct TopShared {
    int cols[kCand];
    int threads[kAgain];
    int pairs[kAgain]; // group * 1024 + thread
};

// A logit as the consumers keep the largest of a group: in its own type.
__device__ __forceinline__ float widened(bf16_t v) { return __uint_as_float(static_cast<uint32_t>(v.bits) << 16); }
__device__ __forceinline__ float widened(float v) { return v; }
template <class T>
__device__ __forceinline__ T narrowed(float v) // exact: v came from a T
{
    if constexpr (sizeof(T) == 2)
        return {static_cast<uint16_t>(__float_as_uint(v) >> 16)};
    else
        return v;
}

// One bit per column of a unit that is at least b (a number; NaN is not).
template <class T>
__device__ __forceinline__ uint32_t at_least(const uint4 &v, float b)
{
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i)
        hits |= unit_value<T>(v, i) >= b ? 1u << i : 0u;
    return hits;
}

// One warp: the best 32 (the best k in any case) of the columns of steps
// [step0, step0 + steps) of a row, one key per lane in order.  part[t].x: the
// largest logit of thread t there, gmax[g][t]: of its columns in group g
// (`groups`, at most OWN, of `per` steps).
template <class T, int NT, int OWN>
__device__ __forceinline__ unsigned long long warp_top(TopShared &top, const T *x, int cols, int step0, int steps, int per,
                                                       int groups, const float4 *part, const T (*gmax)[NT], int k, int lane)
{
    constexpr int W = NT / 32, E = 16 / sizeof(T);
    const int units = (cols + E - 1) / E;
    const uint32_t below = (1u << lane) - 1u;
    float u[W], best = kNegInf;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        u[w] = part[w * 32 + lane].x;
        best = fmaxf(best, u[w]);
    }
    // the k-th of the lanes' best
    const uint32_t ob = __shfl_sync(0xffffffffu, warp_sort_desc(rank_bits(best), lane), k - 1);
    const float bound = unranked(ob);
    int n = kCand + 1;
    if (ob > rank_bits(kNegInf)) { // at -inf stand the lanes without a column, or of NaN and -inf only
        // the threads that reach the bound, then their groups that do
        int nt = 0, np = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t who = __ballot_sync(0xffffffffu, u[w] >= bound);
            const int at = nt + __popc(who & below);
            if (u[w] >= bound && at < kAgain)
                top.threads[at] = w * 32 + lane;
            nt += __popc(who);
        }
        __syncwarp();
        const int items = nt <= kAgain ? nt * OWN : 0;
        for (int i0 = 0; i0 < items; i0 += 32) {
            const int t = top.threads[(i0 + lane) / OWN], g = (i0 + lane) % OWN;
            const bool in = i0 + lane < items && g < groups && widened(gmax[g < groups ? g : 0][t]) >= bound;
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            const int at = np + __popc(who & below);
            if (in && at < kAgain)
                top.pairs[at] = g * 1024 + t;
            np += __popc(who);
        }
        __syncwarp();
        if (nt <= kAgain && np <= kAgain) {
            // their columns, `per` steps of kUnits units of 16 bytes; eight loads
            // at once, over the pairs or over the steps.  A lane notes its columns
            // in the list at the place that a scan of the lanes' counts gives.
            n = 0;
            const int sh = per >= 4 ? 1 : per >= 2 ? 2 : 3, wide = 1 << sh;
            for (int s = 0; s < per; s += 8 >> sh)
                for (int i0 = 0; i0 < np * kUnits; i0 += 32 * wide) {
                    auto unit_of = [&](int a) { // slot a's unit of the row (`units`: none)
                        const int i = i0 + (a & (wide - 1)) * 32 + lane, in = s + (a >> sh);
                        if (i >= np * kUnits || in >= per)
                            return units;
                        const int code = top.pairs[i / kUnits], step = (code >> 10) * per + in;
                        return step < steps ? min(units, ((step0 + step) * kUnits + i % kUnits) * NT + (code & 1023)) : units;
                    };
                    uint4 v[8];
#pragma unroll
                    for (int a = 0; a < 8; ++a) {
                        const int g = unit_of(a);
                        // a unit that is not there: NaN, which reaches no bound
                        v[a] = g < units ? ld16(x + static_cast<int64_t>(g) * E) : make_uint4(~0u, ~0u, ~0u, ~0u);
                    }
                    uint64_t hits = 0; // bit 8 a + i: column i of slot a
#pragma unroll
                    for (int a = 0; a < 8; ++a)
                        hits |= static_cast<uint64_t>(at_least<T>(v[a], bound)) << (8 * a);
                    const int mine = __popcll(hits);
                    int incl = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int other = __shfl_up_sync(0xffffffffu, incl, o);
                        incl += lane >= o ? other : 0;
                    }
                    int to = n + incl - mine;
                    n += __shfl_sync(0xffffffffu, incl, 31);
                    while (hits) {
                        const int bit = __ffsll(static_cast<long long>(hits)) - 1;
                        hits &= hits - 1;
                        if (to < kCand)
                            top.cols[to] = unit_of(bit >> 3) * E + (bit & 7);
                        ++to;
                    }
                    __syncwarp();
                }
        }
    }
    if (n <= kCand) {
        unsigned long long best = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            unsigned long long key = 0;
            if (i0 + lane < n) {
                const int col = top.cols[i0 + lane];
                key = col < cols ? key_of(logit(x, col), col) : 0; // (the row's last unit may hold more)
            }
            key = warp_sort_desc(key, lane);
            best = i0 == 0 ? key : warp_merge_desc(best, key, lane);
        }
        return best;
    }
    // too many reach the bound (equal or masked logits): all columns, keeping the best 32
    unsigned long long have = 0; // lane l: the l-th best so far
    const int64_t from = static_cast<int64_t>(step0) * kUnits * NT;
    const int64_t to = min(static_cast<int64_t>(units), from + static_cast<int64_t>(steps) * kUnits * NT);
    for (int64_t g0 = from; g0 < to; g0 += 32) {
        const int64_t g = g0 + lane;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (g < to)
            v = ld16(x + g * E);
        unsigned long long least = __shfl_sync(0xffffffffu, have, 31);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int64_t col = g * E + i;
            const unsigned long long key = g < to && col < cols ? key_of(unit_value<T>(v, i), static_cast<int>(col)) : 0;
            uint32_t in = __ballot_sync(0xffffffffu, key > least);
            while (in) {
                const unsigned long long one = __shfl_sync(0xffffffffu, key, __ffs(in) - 1);
                in &= in - 1;
                const int at = __popc(__ballot_sync(0xffffffffu, have > one));
                const unsigned long long up = __shfl_up_sync(0xffffffffu, have, 1);
                if (lane == at)
                    have = one;
                else if (lane > at)
                    have = up;
                least = __shfl_sync(0xffffffffu, have, 31);
            }
        }
    }
    return have;
}

// ---------------------------------------------------------------- forward --

// The steps of a row that CTA `rank` of CL takes: whole groups of `per` steps.
struct Share {
    int steps, per, from, to;
};

template <class T, int NT, int CL>
__device__ __forceinline__ Share share_of(int cols, int rank)
{
    constexpr int kCols = NT * kUnits * 16 / sizeof(T); // columns of a step
    Share h;
    h.steps = (cols + kCols - 1) / kCols;
    h.per = (h.steps + kGroups - 1) / kGroups;
    h.from = min(h.steps, rank * (kGroups / CL) * h.per);
    h.to = min(h.steps, (rank + 1) * (kGroups / CL) * h.per);
    return h;
}

// Warps: NT / 32 consumers, one producer, three finishers.  The consumers leave
// the partial results of a row in one of three buffers and go on with the next
// row; the finishers, a row each in turn, join them and find the top k.
template <class T, int NT, int CL, bool TOP, bool ENT>
__global__ void __launch_bounds__(NT + 32 + 32 * kFinishers, kLogpCtas<NT>) k_logp(const __grid_constant__ LParams<kLmSegs> p)
{
    constexpr int E = 16 / sizeof(T);
    constexpr int kStage = NT * kUnits * 16;        // bytes of a step
    constexpr int kCols = kStage / sizeof(T);
    constexpr int kStages = kLogpStages;
    constexpr int kOwn = kGroups / CL;              // groups of this CTA
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kStages], empty[kStages], done[kFinishers], freed[kFinishers];
    __shared__ float4 part[CL > 1 ? 2 : kFinishers][NT];                  // (m, r, s, w) of a row's threads
    __shared__ T gmax[TOP && CL == 1 ? kFinishers : 1][TOP ? kOwn : 1][TOP ? NT : 1]; // largest logit of each group
    __shared__ std::conditional_t<TOP, TopShared, int> top[CL > 1 ? 1 : kFinishers];
    __shared__ unsigned long long peer_best[TOP && CL > 1 ? CL * 32 : 1];
    // behind the ring, in a cluster: the groups of every CTA's threads
    float4 (*from_peers)[NT] = reinterpret_cast<float4 (*)[NT]>(ring + kStages * kStage);
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    if (CL > 1)
        cluster_arrive_relaxed();
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], NT / 32);
        }
#pragma unroll
        for (int i = 0; i < kFinishers; ++i) {
            mbar_init(&done[i], NT / 32);
            mbar_init(&freed[i], 1);
        }
        mbar_init_fence();
    }
    __syncthreads();
    const int64_t total = p.unit_start[p.nseg], stride = gridDim.x / CL;
    // A wait that ran out: the rest runs through without waits, its results do not
    // count.  A lane that gave up arrives nowhere any more (the lane that arrives for a
    // warp has waited itself), so the producer reuses a stage only when every consumer
    // warp has seen it full, no barrier has two copies on their way or an arrival
    // too many, and whoever depends on that lane runs into its own limit.
    bool waiting = true;
    auto wait = [&](uint64_t *bar, int phase) {
        if (waiting && !mbar_wait_bounded(bar, phase & 1, p.wait_limit_ns)) {
            raise_device_error(DS_ERR_DEVICE_TIMEOUT, kSiteLogpWait);
            waiting = false;
        }
    };

    if (tid >= NT && tid < NT + 32) { // the producer
        if (lane == 0) {
            int n = 0; // steps sent
            for (int64_t unit = blockIdx.x / CL; unit < total && waiting; unit += stride) {
                const int si = find_segment(p, unit);
                const LSegK &sg = p.seg[si];
                const char *x = static_cast<const char *>(sg.x) + (unit - p.unit_start[si]) * sg.ld * static_cast<int64_t>(sizeof(T));
                const Share h = share_of<T, NT, CL>(sg.cols, rank);
                for (int s = h.from; s < h.to; ++s, ++n) {
                    const int st = n % kStages;
                    if (n >= kStages)
                        wait(&empty[st], n / kStages - 1);
                    if (!waiting)
                        break;
                    // the row's last bytes up to their 16-byte boundary
                    const int left = sg.cols - s * kCols;
                    const uint32_t bytes = left >= kCols ? kStage : (left + E - 1) / E * 16;
                    mbar_arrive_expect_tx(&full[st], bytes);
                    bulk_g2s(ring + st * kStage, x + static_cast<int64_t>(s) * kStage, bytes, &full[st]);
                }
            }
            // no copy may be in flight at the end, whoever stopped waiting
            for (int i = max(0, n - kStages); i < n; ++i)
                mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1, drain_limit(p.wait_limit_ns));
        }
        if constexpr (CL > 1) { // the cluster's barriers count every thread
            __syncwarp();
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }

    if (tid < NT) { // the consumers
        int st = 0, phase = 0, rows = 0; // stage and its phase; rows taken
        bool masked = false;             // this warp has met a masked logit
        const int warp_first = (tid & ~31) * E; // its first column of a step
        for (int64_t unit = blockIdx.x / CL; unit < total; unit += stride, ++rows) {
            const LSegK &sg = p.seg[find_segment(p, unit)];
            const int cols = sg.cols;
            const float c = sg.scale * kLog2e;
            const Share h = share_of<T, NT, CL>(cols, rank);
            Acc own = no_acc(), group = no_acc(); // the groups joined; the steps of one
            int in_group = 0, g = 0;
            const int b = rows % kFinishers;
            if (rows >= kFinishers)
                wait(&freed[b], rows / kFinishers - 1);
            for (int s = h.from; s < h.to; ++s) {
                wait(&full[st], phase);
                const uint4 *from = reinterpret_cast<const uint4 *>(ring + st * kStage) + tid;
                const int left = cols - s * kCols;
                Acc a;
                if (left >= kCols && !masked) { // uniform in the warp: the row does not end here
                    Step<T> v;
#pragma unroll
                    for (int u = 0; u < kUnits; ++u)
                        v.a[u] = from[u * NT];
                    a = step_acc<ENT, false>(v, c);
                    if (ENT && __any_sync(0xffffffffu, a.w != a.w))
                        masked = true; // from here on this warp floors its logits at once
                    if (!is_plain<ENT>(a))
                        a = careful_acc<ENT, T, NT>(from, left - tid * E, c);
                } else if (left > warp_first) {
                    a = careful_acc<ENT, T, NT>(from, left - tid * E, c);
                } else { // none of its columns are left
                    a = no_acc();
                }
                __syncwarp();
                if (lane == 0 && waiting)
                    mbar_arrive(&empty[st]);
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
                group = in_group == 0 ? a : joined<ENT>(group, a, c);
                if (++in_group == h.per || s + 1 == h.to) {
                    in_group = 0;
                    own = g == 0 ? group : joined<ENT>(own, group, c);
                    if constexpr (TOP)
                        gmax[b][g][tid] = narrowed<T>(group.m);
                    if constexpr (CL > 1)
                        from_peers[rank * kOwn + g][tid] = make_float4(group.m, group.r, group.s, group.w);
                    ++g;
                }
            }
            part[b][tid] = make_float4(own.m, own.r, own.s, own.w);
            __syncwarp();
            if (lane == 0 && waiting)
                mbar_arrive(&done[b]);
            if constexpr (CL > 1) {
                namespace cg = cooperative_groups;
                cluster_wait(); // every CTA of the cluster has started
                if (rank != 0)
                    for (int a = 0; a < g; ++a)
                        *cg::this_cluster().map_shared_rank(&from_peers[rank * kOwn + a][tid], 0) = from_peers[rank * kOwn + a][tid];
                cluster_arrive();
                cluster_wait();
                if (rank != 0)
                    return;
                // the row's groups in order, as one CTA joins them
                for (int a = 0; a * h.per < h.steps; ++a) {
                    const float4 f = from_peers[a][tid];
                    const Acc one{f.x, f.y, f.z, f.w};
                    own = a == 0 ? one : joined<ENT>(own, one, c);
                }
                part[1][tid] = make_float4(own.m, own.r, own.s, own.w);
                __syncwarp();
                if (lane == 0 && waiting)
                    mbar_arrive(&done[1]);
                return; // one row a cluster
            }
        }
        return;
    }

    // the finishers
    const int turn = (tid - NT - 32) / 32;
    if (CL > 1 && turn > 0) { // one row a cluster: nothing to do but its barriers
        cluster_wait();
        cluster_arrive();
        cluster_wait();
        return;
    }
    int rows = turn;
    for (int64_t unit = blockIdx.x / CL + turn * stride; unit < total; unit += kFinishers * stride, rows += kFinishers) {
        const int si = find_segment(p, unit);
        const LSegK &sg = p.seg[si];
        const int64_t row = unit - p.unit_start[si];
        const T *x = static_cast<const T *>(sg.x) + row * sg.ld;
        const int cols = sg.cols;
        const float c = sg.scale * kLog2e;
        const Share h = share_of<T, NT, CL>(cols, rank);
        int64_t id = -1;
        float xt = 0.f;
        if (rank == 0 && lane == 0 && sg.ids) {
            id = load_id(sg.ids, sg.ids_i64, row);
            if (id >= cols) {
                raise_device_error(DS_ERR_INVALID_ARG, kSiteLogpId);
                id = -1;
            }
            if (id >= 0)
                xt = logit(x, id);
        }
        int b = turn;
        wait(&done[b], rows / kFinishers);
        unsigned long long key = 0; // this lane's place among the top
        if constexpr (TOP)
            key = warp_top<T, NT, kOwn>(top[CL > 1 ? 0 : turn], x, cols, h.from, h.to - h.from, h.per,
                                  (h.to - h.from + h.per - 1) / h.per, part[b], gmax[b], sg.top, lane);
        if constexpr (CL > 1) {
            namespace cg = cooperative_groups;
            __syncwarp(); // (lanes may have left the wait apart)
            cluster_wait();
            if constexpr (TOP)
                *cg::this_cluster().map_shared_rank(&peer_best[rank * 32 + lane], 0) = key;
            cluster_arrive();
            cluster_wait();
            if (rank != 0)
                return;
            if constexpr (TOP)
                {
                unsigned long long keys[CL]; // pair by pair: the merges of a level run side by side
#pragma unroll
                for (int r = 0; r < CL; ++r)
                    keys[r] = peer_best[r * 32 + lane];
#pragma unroll
                for (int half = CL / 2; half > 0; half /= 2)
#pragma unroll
                    for (int r = 0; r < half; ++r)
                        keys[r] = warp_merge_desc(keys[r], keys[r + half], lane);
                key = keys[0];
            }
            b = 1;
            wait(&done[1], 0);
        }
        // the threads: the maximum, then the sums at it, NT / 32 threads a lane
        float m = kNegInf, r = kNegInf;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            m = fmaxf(m, part[b][w * 32 + lane].x);
            r = fmaxf(r, part[b][w * 32 + lane].y);
        }
        const float M = warp_max(m), R = warp_max(r);
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const float4 f = part[b][w * 32 + lane];
            const float d = is_near(f.y) && is_near(R) ? f.y - R : far_shift(f.x, f.y, M, R, c), k = ex2(d);
            t[0] = fmaf(f.z, k, t[0]);
            if (ENT)
                t[1] = fmaf(fmaf(d, f.z, f.w), k, t[1]);
        }
        __syncwarp();
        if (lane == 0 && waiting)
            mbar_arrive(&freed[b]);
        warp_sum(t);
        const bool none = M == kNegInf && t[0] == 0.f; // no logit above -inf
        const float ln_s = logf(t[0]);
        const bool far = !is_near(R) && is_finite(M);
        auto log_prob = [&](float v) {
            const float y = fmaf(v, c, -R);
            const bool lost = far || (!is_finite(y) && is_finite(v)); // an exponent past fp32
            return none ? kNegInf : lost ? fmaf(v - M, sg.scale, -ln_s) : fmaf(y, kLn2, -ln_s);
        };
        if (lane == 0) {
            if (sg.lse)
                // (the sums stand at R, not at M c: the difference is exact.  R ln 2 would carry
                // the roundings of c, R and ln 2, each as large as that of the result)
                sg.lse[row] = none ? kNegInf : fmaf(M, sg.scale, far ? ln_s : fmaf(fmaf(-M, c, R), kLn2, ln_s));
            if (sg.logp)
                sg.logp[row] = id < 0 ? 0.f : log_prob(xt);
            if (ENT && sg.entropy)
                sg.entropy[row] = none ? 0.f : fmaf(-kLn2, t[1] / t[0], ln_s);
        }
        if constexpr (TOP) {
            if (lane < sg.top) {
                const int64_t at = row * sg.top + lane;
                sg.top_id[at] = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
                if (sg.top_logp)
                    sg.top_logp[at] = log_prob(unranked(static_cast<uint32_t>(key >> 32)));
            }
        }
        if constexpr (CL > 1)
            return;
    }
}

// --------------------------------------------------------------- backward --

constexpr int kGradThreads = 128;

constexpr int kGradOctets = 2; // octets of a thread, side by side

// exp of it is 0 in fp32, and dh times it finite (for any |dh| below 2^120).
constexpr float kNoProb = -128.f;

// One octet's gradient: p (A - dh (z - lse)), p = exp(z - lse).  A masked logit
// (-inf) has p = 0, times a finite value.
template <bool ENT, class T>
__device__ __forceinline__ void octet_grad(const Raw8<T> &x, float (&d)[8], float scale, float lse, float A, float dh)
{
    const float2 sc = make_float2(scale, scale), off = make_float2(-lse, -lse), l2e = make_float2(kLog2e, kLog2e);
    const float2 aa = make_float2(A, A), dd = make_float2(-dh, -dh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lp = __ffma2_rn(make_float2(x.get(2 * i), x.get(2 * i + 1)), sc, off);
        const float2 y = __fmul2_rn(lp, l2e);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        float2 f = aa;
        if (ENT)
            f = __ffma2_rn(dd, make_float2(fmaxf(lp.x, kNoProb), fmaxf(lp.y, kNoProb)), aa);
        const float2 o = __fmul2_rn(e, f);
        d[2 * i] = o.x, d[2 * i + 1] = o.y;
    }
}

// Both octets of a thread: 32 bytes of bf16 move in one access where they can.
template <class T>
__device__ __forceinline__ void load16(const T *p, Raw8<T> (&v)[2])
{
    if constexpr (sizeof(T) == 2) {
        if (on32(p)) {
            float4 a, b;
            ld32(p, a, b);
            v[0].a = as_u4(a), v[1].a = as_u4(b);
            return;
        }
    }
    v[0].load(p, 8);
    v[1].load(p + 8, 8);
}

__device__ __forceinline__ uint4 packed8(const float (&d)[8])
{
    return make_uint4(pack_bf2(d[0], d[1]), pack_bf2(d[2], d[3]), pack_bf2(d[4], d[5]), pack_bf2(d[6], d[7]));
}

template <class T>
__device__ __forceinline__ void store16(T *p, const float (&d)[2][8])
{
    if constexpr (sizeof(T) == 2) {
        if (on32(p)) {
            st32(p, packed8(d[0]), packed8(d[1]));
            return;
        }
    }
    store8(p, d[0], 8);
    store8(p + 8, d[1], 8);
}

// A block takes a part of a row, a thread 16 columns of it.  The bound is memory:
// the copy rate in fp32, 89% of it in bf16, where the instructions count as well
// (each logit is 4 bytes of traffic).  Small blocks of few columns a thread and
// every warp that fits measured best: 183 us for 8,192 x 32,000 in bf16, 204
// with 42 registers a thread instead of 32, 225 with 32 columns a thread.
template <class T, class GT, int N>
__global__ void __launch_bounds__(kGradThreads, 16) k_logp_grad(const __grid_constant__ LParams<N> p)
{
    constexpr int kCols = 8 * kGradThreads * kGradOctets;
    const int si = N == 1 ? 0 : find_segment(p, blockIdx.x);
    const LSegK &sg = p.seg[si];
    const uint32_t unit = blockIdx.x - static_cast<uint32_t>(p.unit_start[si]);
    const int cols = sg.cols;
    const uint32_t parts = (static_cast<uint32_t>(cols) + kCols - 1) / kCols;
    const int64_t row = unit / parts;
    const int part = static_cast<int>(unit - static_cast<uint32_t>(row) * parts);
    int64_t id = sg.ids && sg.dlogp ? load_id(sg.ids, sg.ids_i64, row) : -1;
    const float lse = __ldg(sg.lse + row), scale = sg.scale;
    float g = sg.dlogp ? __ldg(sg.dlogp + row) * scale : 0.f;
    const float dh = sg.dentropy ? __ldg(sg.dentropy + row) * scale : 0.f;
    const float h = sg.dentropy ? __ldg(sg.entropy + row) : 0.f;
    const float dl = sg.dlse ? __ldg(sg.dlse + row) * scale : 0.f;
    if (id >= cols) {
        if (part == 0 && threadIdx.x == 0)
            raise_device_error(DS_ERR_INVALID_ARG, kSiteLogpId);
        id = -1;
    }
    g = id >= 0 ? g : 0.f;
    const int first = part * kCols + 16 * static_cast<int>(threadIdx.x), left = cols - first;
    if (left <= 0)
        return;
    GT *dx = static_cast<GT *>(sg.dx) + row * sg.ld_d + first;
    float d[2][8] = {};
    if ((g != 0.f || dh != 0.f || dl != 0.f) && lse != kNegInf) { // uniform; else nothing comes back
        const T *x = static_cast<const T *>(sg.x) + row * sg.ld + first;
        const float A = dl - g - dh * h;
        Raw8<T> v[2];
        if (left >= 16) {
            load16(x, v);
        } else {
            v[0].load(x, left);
            v[1].load(x + 8, left - 8);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (dh != 0.f) // uniform
                octet_grad<true>(v[k], d[k], scale, lse, A, dh);
            else
                octet_grad<false>(v[k], d[k], scale, lse, A, 0.f);
        const int64_t at = id - first; // the token's column, from this thread's first
        if (id >= 0 && at >= 0 && at < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (at == i)
                    d[i / 8][i % 8] += g;
        }
    }
    if (left >= 16) {
        store16(dx, d);
    } else {
        store8(dx, d[0], left);
        store8(dx + 8, d[1], left - 8);
    }
}

// ---------------------------------------------------------------- launches --

template <class T, int NT, int CL, bool TOP, bool ENT>
cudaError_t launch_one(const LParams<kLmSegs> &p, int64_t units, int sms, cudaStream_t st)
{
    static DeviceFlags done;
    constexpr int bytes = kLogpStages * NT * kUnits * 16 + (CL > 1 ? kGroups * NT * 16 : 0);
    auto *kernel = k_logp<T, NT, CL, TOP, ENT>;
    if (cudaError_t e = enable_dynamic_smem(kernel, bytes, done); e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    // rows in turn over the CTAs that fit at once; a cluster takes one row
    const int64_t fit = int64_t(sms) * kLogpCtas<NT>;
    cfg.gridDim = dim3(static_cast<unsigned>(CL > 1 ? units * CL : std::min(units, fit)));
    cfg.blockDim = dim3(NT + 32 + 32 * kFinishers);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (CL > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = CL;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T, int NT, int CL>
cudaError_t launch_flags(bool top, bool ent, const LParams<kLmSegs> &p, int64_t units, int sms, cudaStream_t st)
{
    if (top)
        return ent ? launch_one<T, NT, CL, true, true>(p, units, sms, st) : launch_one<T, NT, CL, true, false>(p, units, sms, st);
    return ent ? launch_one<T, NT, CL, false, true>(p, units, sms, st) : launch_one<T, NT, CL, false, false>(p, units, sms, st);
}

template <class T>
cudaError_t launch_fwd(int cls, int cl, bool top, bool ent, const LParams<kLmSegs> &p, int64_t units, int sms, cudaStream_t st)
{
    if (cls == 0)
        return launch_flags<T, 128, 1>(top, ent, p, units, sms, st);
    switch (cl) {
    case 1: return launch_flags<T, kLogpThreads, 1>(top, ent, p, units, sms, st);
    case 2: return launch_flags<T, kLogpThreads, 2>(top, ent, p, units, sms, st);
    case 4: return launch_flags<T, kLogpThreads, 4>(top, ent, p, units, sms, st);
    default: return launch_flags<T, kLogpThreads, 8>(top, ent, p, units, sms, st);
    }
}

template <class T, class GT>
void launch_grad(const LParams<kLmSegs> &p, int64_t units, cudaStream_t st)
{
    const unsigned g = static_cast<unsigned>(units);
    if (p.nseg == 1)
        k_logp_grad<T, GT, 1><<<g, kGradThreads, 0, st>>>(only_segment(p));
    else
        k_logp_grad<T, GT, kLmSegs><<<g, kGradThreads, 0, st>>>(p);
}

} // namespace

int logp_class(int64_t cols) { return cols <= 4096 ? 0 : 1; }

int64_t logp_steps(bool bf16, int64_t cols)
{
    const int64_t per = kLogpThreads * kUnits * 16 / (bf16 ? 2 : 4);
    return (cols + per - 1) / per;
}

int launch_logp(bool bf16, int cls, int cl, bool top, bool ent, const LParams<kLmSegs> &p, int64_t units, int sms, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return bf16 ? launch_fwd<bf16_t>(cls, cl, top, ent, p, units, sms, st) : launch_fwd<float>(cls, cl, top, ent, p, units, sms, st);
}

int64_t logp_grad_parts(int64_t cols)
{
    constexpr int64_t per = 8 * kGradThreads * kGradOctets; // columns of a block
    return (cols + per - 1) / per;
}

int launch_logp_grad(bool bf16, bool grad_bf16, const LParams<kLmSegs> &p, int64_t units, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (bf16)
        grad_bf16 ? launch_grad<bf16_t, bf16_t>(p, units, st) : launch_grad<bf16_t, float>(p, units, st);
    else
        grad_bf16 ? launch_grad<float, bf16_t>(p, units, st) : launch_grad<float, float>(p, units, st);
    return cudaGetLastError();
}

int logp_read_and_clear_error(uint32_t *code, uint32_t *site) { return module_read_and_clear_error(code, site); }

} // namespace ds
