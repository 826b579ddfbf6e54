// lf_kv4.cuh -- device pieces of the 4-bit KV cache: conversions between the
// format's bytes and FP16 pairs, and row loads and stores by element type.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "lf_kv4.h"
#include "lf_internal.cuh"
#include "lf_ptx.cuh"

namespace lfq {

// Four bytes of two E2M1 codes each -> FP16 pairs (low nibble first), exact.
__device__ __forceinline__ void e2m1x8_h2(unsigned w, unsigned &h0, unsigned &h1, unsigned &h2, unsigned &h3)
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
        : "r"(w));
}
// Two FP32 values -> one byte of E2M1 codes (`lo` in the low nibble), to nearest even, saturating at 6.
__device__ __forceinline__ unsigned e2m1x2(float lo, float hi)
{
    unsigned short d;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "mov.b16 %0, {b, 0};\n\t}"
        : "=h"(d)
        : "f"(hi), "f"(lo));
    return d;
}
// Two E4M3 bytes (low one first) -> an FP16 pair, exact.
__device__ __forceinline__ unsigned e4m3x2_h2(unsigned b)
{
    unsigned d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((unsigned short)b));
    return d;
}
// One E4M3 byte in both halves of a pair.
__device__ __forceinline__ unsigned e4m3_h2_same(unsigned b) { return e4m3x2_h2(b | (b << 8)); }
// Two scale bytes of V for the attention, where the one that stands for NaN counts as 448 (the minimum's other
// operand): a NaN would meet the zero probability of rows that do not see its position, and make those NaN as well.  (A
// position that was never written holds whatever the memory held, and padded rows behind a block's end see it.  A NaN
// of K stays in the scores of its position, which such rows leave out.)
__device__ __forceinline__ unsigned scales_h2(unsigned b)
{
    unsigned d;
    asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(e4m3x2_h2(b)), "r"(0x5f005f00u));
    return d;
}
__device__ __forceinline__ unsigned hmul2(unsigned a, unsigned b)
{
    unsigned d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// 2^x on the special-function unit (about 2 ulp; exact 0 for -inf).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- programmatic dependent launches: the next kernel may start its prologue; wait for the previous one's end
__device__ __forceinline__ void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_prerequisites() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A load of what a kernel before this one wrote.  A plain one: the read-only path's is for data that nothing writes
// while the kernel runs, and a dependent launch runs beside its predecessors until it has waited for them; the
// compiler may move such a load ahead of the wait.
template <class T>
__device__ __forceinline__ T ld(const T *p) { return *p; }

// ---- clusters: a barrier, and loads from another CTA's shared memory
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_smem(const void *p, int rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(lfk::smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

// ---- packed FP32 pairs
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
    return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// ---- rows by element type: 16 consecutive values (16-byte aligned), and the bits of the largest magnitude as FP32
// (NaN's above infinity's above all; 16-bit types find it two values at a time)
template <class T>
__device__ __forceinline__ unsigned load16(const T *p, float (&x)[16]);
__device__ __forceinline__ unsigned top_of(const float (&x)[16])
{
    unsigned top = 0u;
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    return top;
}
__device__ __forceinline__ unsigned top_of(const uint4 &a, const uint4 &b)
{
    const unsigned m = 0x7fff7fffu;
    const unsigned t = __vmaxu2(__vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m)),
                                __vmaxu2(__vmaxu2(b.x & m, b.y & m), __vmaxu2(b.z & m, b.w & m)));
    return max(t & 0xffffu, t >> 16);
}
__device__ __forceinline__ unsigned halves(const uint4 &a, const uint4 &b, float (&x)[16])
{
    const unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[u]));
        x[2 * u] = f.x, x[2 * u + 1] = f.y;
    }
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top_of(a, b))));
}
template <>
__device__ __forceinline__ unsigned load16<float>(const float *p, float (&x)[16])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = ld(reinterpret_cast<const float4 *>(p) + j);
        x[4 * j] = v.x, x[4 * j + 1] = v.y, x[4 * j + 2] = v.z, x[4 * j + 3] = v.w;
    }
    return top_of(x);
}
template <>
__device__ __forceinline__ unsigned load16<__half>(const __half *p, float (&x)[16])
{
    const uint4 *v = reinterpret_cast<const uint4 *>(p);
    return halves(ld(v), ld(v + 1), x);
}
template <>
__device__ __forceinline__ unsigned load16<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[16])
{
    const uint4 a = ld(reinterpret_cast<const uint4 *>(p)), b = ld(reinterpret_cast<const uint4 *>(p) + 1);
    const unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        x[2 * u] = __uint_as_float(w[u] << 16);
        x[2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
    }
    return top_of(a, b) << 16;
}
__device__ __forceinline__ float2 h2_f2(unsigned h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }
__device__ __forceinline__ unsigned pack_bf2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&b);
}
// Block b of row (t, h) of `in`, by element type (Tagged, Swizzled: the decoder's own buffers).
struct Tagged {};
struct Swizzled {};
template <class T>
__device__ __forceinline__ unsigned load_block(const Rows &in, long long t, int h, int b, float (&x)[16])
{
    return load16<T>(static_cast<const T *>(in.p) + t * in.ts + h * in.hs + b * 16, x);
}
template <>
__device__ __forceinline__ unsigned load_block<Tagged>(const Rows &in, long long t, int h, int b, float (&x)[16])
{
    load16<float>(static_cast<const float *>(in.p) + t * in.ts + h * in.hs + b * 16, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(__float_as_uint(x[j]) & ~1u);   // an infinity with a tag is a NaN
    return top_of(x);
}
template <>
__device__ __forceinline__ unsigned load_block<Swizzled>(const Rows &in, long long t, int h, int b, float (&x)[16])
{
    const __half *row = static_cast<const __half *>(in.p) + t * in.ts + h * in.hs;
    const int sw = (int)((in.aux + t) & 7);
    return halves(ld(reinterpret_cast<const uint4 *>(row + ((2 * b) ^ sw) * 8)),
                  ld(reinterpret_cast<const uint4 *>(row + ((2 * b + 1) ^ sw) * 8)), x);
}
// 16 bytes of cached values, FP16 pairs in h, as T (exact: at most 6 significant bits)
__device__ __forceinline__ void store_values(__half *p, const unsigned (&h)[4])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ void store_values(__nv_bfloat16 *p, const unsigned (&h)[4])
{
    unsigned w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = h2_f2(h[j]);
        w[j] = pack_bf2(f.x, f.y);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_values(float *p, const unsigned (&h)[4])
{
    const float2 a = h2_f2(h[0]), b = h2_f2(h[1]);
    *reinterpret_cast<float4 *>(p) = make_float4(a.x, a.y, b.x, b.y);
}
// Four values at element offset `at` of o (rounded once, to nearest even).
__device__ __forceinline__ void store4(const Rows &o, size_t at, float a, float b, float c, float d)
{
    if (o.dtype == F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(o.p) + at) = make_float4(a, b, c, d);
    } else if (o.dtype == F16 || o.dtype == BF16) {
        unsigned x, y;
        if (o.dtype == F16) {
            const __half2 u = __floats2half2_rn(a, b), v = __floats2half2_rn(c, d);
            x = *reinterpret_cast<const unsigned *>(&u);
            y = *reinterpret_cast<const unsigned *>(&v);
        } else {
            x = pack_bf2(a, b);
            y = pack_bf2(c, d);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.p) + at) = make_uint2(x, y);
    } else if (o.dtype == TAG32) {
        const unsigned tag = (unsigned)o.aux;
        *reinterpret_cast<uint4 *>(static_cast<unsigned *>(o.p) + at) =
            make_uint4((__float_as_uint(a) & ~1u) | tag, (__float_as_uint(b) & ~1u) | tag, (__float_as_uint(c) & ~1u) | tag,
                       (__float_as_uint(d) & ~1u) | tag);
    } else {   // SPLIT16
        __half h[4], m[4];
        lfk::split_h(a, h[0], m[0]);
        lfk::split_h(b, h[1], m[1]);
        lfk::split_h(c, h[2], m[2]);
        lfk::split_h(d, h[3], m[3]);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.p) + at) =
            make_uint2(lfk::pack_h2(h[0], h[1]), lfk::pack_h2(h[2], h[3]));
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.p2) + at) =
            make_uint2(lfk::pack_h2(m[0], m[1]), lfk::pack_h2(m[2], m[3]));
    }
}
// One row of q, HD / 32 consecutive values per lane (zeros for a row that is not there).
template <int HD>
__device__ __forceinline__ void load_q(const Rows &q, bool live, int tok, int head, int lane, float (&x)[HD / 32])
{
    const size_t at = (size_t)tok * q.ts + (size_t)head * q.hs + lane * (HD / 32);
#pragma unroll
    for (int j = 0; j < HD / 32; j += 2) {
        float2 v = make_float2(0.f, 0.f);
        if (live) {
            if (q.dtype == F32) {
                v = *reinterpret_cast<const float2 *>(static_cast<const float *>(q.p) + at + j);
            } else {
                const unsigned w = *reinterpret_cast<const unsigned *>(static_cast<const uint16_t *>(q.p) + at + j);
                v = q.dtype == F16 ? h2_f2(w) : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            }
        }
        x[j] = v.x;
        x[j + 1] = v.y;
    }
}
template <int N>
__device__ __forceinline__ float warp_amax(const float (&x)[N])
{
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(x[j]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
// A power of two that brings values of largest magnitude m into [1, 2) (into [1, 4)
// at the top of FP32's range; 1 for zero, subnormal or non-finite m): exact to
// multiply with and, as the inverse is a power of two, to divide by.
__device__ __forceinline__ float range_factor(float m)
{
    const unsigned e = __float_as_uint(m) >> 23;
    if (e == 0u || e == 255u) return 1.f;
    return __uint_as_float((254u - min(e, 253u)) << 23);
}

// ---- one lane's share of a K row: HD / 4 dims, as KS k-steps of 4 (two pairs each)
template <int HD>
struct KRaw;
template <>
struct KRaw<128> {
    uint4 c;
    unsigned s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales)
    {
        c = ld(reinterpret_cast<const uint4 *>(codes));
        s = ld(reinterpret_cast<const unsigned short *>(scales));
    }
    __device__ __forceinline__ void values(unsigned (&v)[8][2]) const
    {
        const unsigned w[4] = {c.x, c.y, c.z, c.w};
        const unsigned sc2 = e4m3x2_h2(s);
        const __half2 sh = *reinterpret_cast<const __half2 *>(&sc2);
        const __half2 s0 = __low2half2(sh), s1 = __high2half2(sh);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e2m1x8_h2(w[j], v[2 * j][0], v[2 * j][1], v[2 * j + 1][0], v[2 * j + 1][1]);
            const __half2 sc = j < 2 ? s0 : s1;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&v[2 * j + u / 2][u % 2]), sc);
                v[2 * j + u / 2][u % 2] = *reinterpret_cast<const unsigned *>(&x);
            }
        }
    }
};
template <>
struct KRaw<64> {
    uint2 c;
    unsigned s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales)
    {
        c = ld(reinterpret_cast<const uint2 *>(codes));
        s = ld(scales);
    }
    __device__ __forceinline__ void values(unsigned (&v)[4][2]) const
    {
        const unsigned s0 = e4m3_h2_same(s);
        e2m1x8_h2(c.x, v[0][0], v[0][1], v[1][0], v[1][1]);
        e2m1x8_h2(c.y, v[2][0], v[2][1], v[3][0], v[3][1]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u][0] = hmul2(v[u][0], s0);
            v[u][1] = hmul2(v[u][1], s0);
        }
    }
};
// ---- one lane's share of a V row: HD / 8 dims of one block
template <int HD>
struct VRaw;
template <>
struct VRaw<128> {
    uint2 c;
    unsigned s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales)
    {
        c = ld(reinterpret_cast<const uint2 *>(codes));
        s = ld(scales);
    }
    __device__ __forceinline__ unsigned word(int j) const { return j ? c.y : c.x; }
};
template <>
struct VRaw<64> {
    unsigned c;
    unsigned s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales)
    {
        c = ld(reinterpret_cast<const unsigned *>(codes));
        s = ld(scales);
    }
    __device__ __forceinline__ unsigned word(int) const { return c; }
};
// Rows a and b of V woven: v[k][e] = the FP16 pair (a[dim 2k + e], b[dim 2k + e]).
template <int HD>
__device__ __forceinline__ void weave(const VRaw<HD> &a, const VRaw<HD> &b, unsigned (&v)[HD / 16][2])
{
    const unsigned sc = scales_h2(a.s | (b.s << 8));
#pragma unroll
    for (int j = 0; j < HD / 64; ++j) {
        const unsigned x = a.word(j), y = b.word(j), m = 0x0f0f0f0fu;
        const unsigned even = (x & m) | ((y << 4) & ~m), odd = ((x >> 4) & m) | (y & ~m);
        e2m1x8_h2(even, v[4 * j][0], v[4 * j + 1][0], v[4 * j + 2][0], v[4 * j + 3][0]);
        e2m1x8_h2(odd, v[4 * j][1], v[4 * j + 1][1], v[4 * j + 2][1], v[4 * j + 3][1]);
    }
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        v[k][0] = hmul2(v[k][0], sc);
        v[k][1] = hmul2(v[k][1], sc);
    }
}

}  // namespace lfq
