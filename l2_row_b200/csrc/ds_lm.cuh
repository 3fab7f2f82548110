// ds_lm.cuh -- building blocks shared by the embedding, q/k norm and token log
// probability kernels: octets (8 columns) of bf16 or fp32 rows with a ragged
// end, 32- or 64-bit ids, and reductions over a team of one warp or one block.
#pragma once

#include "ds_device.cuh"
#include "ds_lm.h"

namespace ds {

struct bf16_t {
    uint16_t bits;
};

__device__ __forceinline__ int64_t load_id(const void *ids, int i64, int64_t t)
{
    return i64 ? __ldg(static_cast<const long long *>(ids) + t) : static_cast<int64_t>(__ldg(static_cast<const int32_t *>(ids) + t));
}

// One 32-byte load (sm_100's 256-bit vector load); p 32-byte aligned.
__device__ __forceinline__ void ld32(const void *p, float4 &a, float4 &b)
{
    uint4 x, y;
    asm volatile("ld.global.nc.L1::no_allocate.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                 : "l"(p));
    a = as_f4(x), b = as_f4(y);
}

// fp32 octets on 32 bytes move in one access: as two of 16 bytes, a warp's
// accesses would touch every 32-byte sector twice.
__device__ __forceinline__ bool on32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// An octet as loaded: 16 bytes of bf16, 32 bytes of fp32.  `valid` columns
// (any number; <= 0: nothing is read) keep their value, the others are 0.  A
// row may be read up to the 16-byte boundary after its last column.
template <class T>
struct Raw8;

template <>
struct Raw8<bf16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16_t *p, int valid)
    {
        a = make_uint4(0, 0, 0, 0);
        if (valid > 0) {
            a = ld16(p);
            if (valid < 8)
                a = mask_octet(a, valid);
        }
    }
    __device__ __forceinline__ float get(int i) const { return bf_get(a, i); }
};

template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, int valid)
    {
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (valid >= 8 && on32(p)) {
            ld32(p, a, b);
            return;
        }
        if (valid > 0) {
            a = as_f4(ld16(p));
            if (valid < 4)
                a = mask_quad(a, valid);
        }
        if (valid > 4) {
            b = as_f4(ld16(p + 4));
            if (valid < 8)
                b = mask_quad(b, valid - 4);
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        const float4 &q = i < 4 ? a : b;
        const int j = i & 3;
        return j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
    }
};

template <class T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8], int valid)
{
    Raw8<T> r;
    r.load(p, valid);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = r.get(i);
}

// The same from memory that this kernel writes (no read-only path).
__device__ __forceinline__ void load8_plain(const float *p, float (&v)[8], int valid)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = 0.f;
    if (valid >= 8) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid)
                v[i] = p[i];
    }
}

// The first `valid` of 8 columns; bf16 rounds to nearest even.
__device__ __forceinline__ void store8(bf16_t *p, const float (&v)[8], int valid)
{
    const uint4 w = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
    if (valid >= 8) {
        st16(p, w);
    } else {
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid)
                p[i].bits = static_cast<uint16_t>(h[i / 2] >> (16 * (i & 1)));
    }
}

__device__ __forceinline__ void store8(float *p, const float (&v)[8], int valid)
{
    if (valid >= 8 && on32(p)) {
        st32(p, as_u4(make_float4(v[0], v[1], v[2], v[3])), as_u4(make_float4(v[4], v[5], v[6], v[7])));
    } else if (valid >= 8) {
        st16(p, as_u4(make_float4(v[0], v[1], v[2], v[3])));
        st16(p + 4, as_u4(make_float4(v[4], v[5], v[6], v[7])));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid)
                p[i] = v[i];
    }
}

// The bound of the waits for copies still on their way when a block ends, so
// that none lands in shared memory that is no longer its own: at least 2 s,
// however short the other waits are.
__device__ __forceinline__ uint64_t drain_limit(uint64_t limit_ns) { return limit_ns > 2000000000ull ? limit_ns : 2000000000ull; }

__device__ __forceinline__ void store8_smem(float *p, const float (&v)[8])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Sums over a team of T threads: one warp (T = 32), or a whole block of T
// threads.  Every thread gets the same bits: an xor butterfly in the warp,
// then the warps in order.  At most two values at once.
template <int T>
struct TeamRed {
    static constexpr int W = T / 32;
    float *sm; // [2][W][2]; two slots in turn, so one barrier a sum is enough
    int slot = 0;
    __device__ explicit TeamRed(float *scratch) : sm(scratch) {}

    __device__ __forceinline__ void barrier() const
    {
        if constexpr (W == 1)
            __syncwarp();
        else
            __syncthreads();
    }
    template <int N, class Op>
    __device__ __forceinline__ void across(float (&v)[N], Op op)
    {
        if constexpr (W > 1) {
            float *s = sm + slot * (2 * W);
            slot ^= 1;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    s[(threadIdx.x >> 5) * 2 + i] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float t = s[i];
#pragma unroll
                for (int w = 1; w < W; ++w)
                    t = op(t, s[w * 2 + i]);
                v[i] = t;
            }
        }
    }
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N])
    {
        static_assert(N <= 2, "scratch holds two values");
        warp_sum(v);
        across(v, [](float a, float b) { return a + b; });
    }
    __device__ __forceinline__ float max(float v)
    {
        float a[1] = {warp_max(v)};
        across(a, [](float x, float y) { return fmaxf(x, y); });
        return a[0];
    }
    __device__ __forceinline__ bool any(bool b) const { return b; } // sums are uniform in the team
};

} // namespace ds
