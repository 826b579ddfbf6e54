// lf_paged_attn.cu -- attention of one new token per sequence over a paged KV
// cache.
//
// For every sequence and query head: out = sum_j softmax_j(scale q . K[j]) V[j]
// over the sequence's positions j, which lie in pages anywhere in the pools.
// Each byte of K and V is needed once and meets 2 G products (G query heads
// share a KV head): bound by memory, so all that counts is that loads never
// pause.
//
// The unit of work is a slab: 16 positions of one KV head, a stretch of one
// page (pages are whole slabs).  A warp works alone.  It copies its slabs into
// a ring of its own in shared memory with asynchronous 16-byte copies, two of
// three stages on the way at any time, forms
//   S^T = K Q^T   (16 positions x 8 query heads, ldmatrix, warp-level products)
//   O^T += V^T P^T (16 dims x 8 heads per step, ldmatrix transposed)
// and carries its softmax state (reference, sum, O) in registers.  No barrier
// joins the warps of a CTA on the way: 8 warps x 2 slabs of 8 KB are 128 KB on
// the way per SM, twice what the memory's latency asks for.  Warp-level
// products suit this shape (8 heads wide, 16 positions deep), and at 2 G
// operations a byte the tensor cores wait for memory.
//
// Accuracy: scores, softmax and sums are FP32.  A query of the cache's type
// enters the products as it is, one in FP32 as the sum of two FP16 terms (scaled
// by a power of two: 22 bits) or three BF16 terms (24 bits).  P is split in the
// same way whatever q is, so that the output's own rounding is the only one that
// counts.  The further products of each step are nearly free while memory is
// waited for (BF16, two terms of P instead of three: 33 rows in a window of 1,000 8.2
// us instead of 8.5, 64 x 8 heads to 16,384 0.2 % less, weights of 16 bits).
//
// Measured (one GB300): 64 sequences of up to 16,384 positions, 32/8 heads x
// 128, BF16: 291-296 us, 7.4 TB/s (a copy's rate is 6.8); one of 131,071 81 us,
// 6.6 TB/s; one of 512, 20/5 heads x 128 4.9 us.  With FP32 queries on BF16 and
// 16 heads per KV head the instructions count: 5.2 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "../../include/lf.h"
#include "lf_kv4.cuh"
#include "lf_paged.h"
#include "lf_rows.cuh"

namespace lfpg {

using lfq::ex2;

template <class T>
struct Half16;
template <>
struct Half16<__half> {
    static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ unsigned pair(float x, float y)
    {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const unsigned *>(&h);
    }
    static __device__ __forceinline__ float2 values(unsigned p) { return __half22float2(*reinterpret_cast<const __half2 *>(&p)); }
    // d = a b + (d, or 0)
    static __device__ __forceinline__ void mma(float (&d)[4], const unsigned (&a)[4], const unsigned (&b)[2], bool first = false)
    {
        const float c[4] = {first ? 0.f : d[0], first ? 0.f : d[1], first ? 0.f : d[2], first ? 0.f : d[3]};
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    }
};
template <>
struct Half16<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ unsigned pair(float x, float y)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const unsigned *>(&h);
    }
    static __device__ __forceinline__ float2 values(unsigned p) { return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)); }
    static __device__ __forceinline__ void mma(float (&d)[4], const unsigned (&a)[4], const unsigned (&b)[2], bool first = false)
    {
        const float c[4] = {first ? 0.f : d[0], first ? 0.f : d[1], first ? 0.f : d[2], first ? 0.f : d[3]};
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    }
};
// x and y as sums of N terms of type T, the largest first: pairs (term of x, term of y)
template <class T, int N>
__device__ __forceinline__ void split_pair(float x, float y, unsigned (&out)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        out[i] = Half16<T>::pair(x, y);
        if (i + 1 < N) {
            const float2 v = Half16<T>::values(out[i]);
            x -= v.x;
            y -= v.y;
        }
    }
}

__device__ __forceinline__ void sts(uint32_t at, unsigned x) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory"); }
__device__ __forceinline__ void lds2(unsigned (&x)[2], uint32_t at)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(at));
}

// 16 bytes global -> shared, zeros where `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const char *src, unsigned bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const char *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Positions that a sequence's query sees and the table has, [lo, hi), and the slabs that hold them, [s0, s1).
struct Seen {
    int lo, hi, s0, s1;
    __device__ __forceinline__ Seen(const Attn &a, int len)
    {
        lo = a.win > 0 && len > a.win ? len - a.win : 0;
        hi = (int)min((long long)len, (long long)a.width * a.c.page);
        if (hi <= lo) lo = hi = 0;
        s0 = lo >> 4;
        s1 = (hi + 15) >> 4;
    }
    __device__ __forceinline__ int slabs() const { return s1 - s0; }
};

template <int HD>
struct Ring {
    static constexpr int SLAB = 16 * HD * 2;                 // bytes of K, and of V
    static constexpr int STAGES = 24576 / (2 * SLAB);        // 3 of 8 KB, 6 of 4
    static constexpr int COPIES = STAGES * 2 * SLAB;         // bytes of a warp's slabs
};

// A warp's softmax state and its products, for 8 NT query heads of one KV head.
// QT: terms of q (1: it has the cache's type).
template <int HD, int NT, class T, int QT>
struct Work {
    static constexpr int KS = HD / 16, RT = 8 * NT;
    static constexpr int PT = std::is_same_v<T, __half> ? 2 : 3;   // terms of P
    static constexpr float P_EXP = 7.f, P_SUM = 32768.f;
    // q's fragments: in registers, or where they would take 64 of them or 96 in shared memory, one copy for the CTA
    static constexpr bool QS = QT * NT >= 4;
    static constexpr int Q_BYTES = QS ? NT * KS * 32 * QT * 8 : 0;
    unsigned q[QS ? 1 : QT][QS ? 1 : NT][QS ? 1 : KS][2];
    uint32_t qs;
    // Score = f st in log2 units, f >= 0 (q carries the scale's sign).  The reference is a value of st, subtracted before
    // f multiplies, so that equal scores differ by 0 and the largest one from itself, however far apart FP32's steps are.
    float f[NT][2], ref[NT][2], l[NT][2], o[NT][KS][4];

    __device__ __forceinline__ void begin(const Attn &a, int row, int ht, int warp, int warps, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        const int kvh = ht / a.tiles, h0 = (ht - kvh * a.tiles) * RT;
        const float base = fminf(fabsf(a.scale) * 1.4426950408889634f, FLT_MAX);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int hh = h0 + 8 * i + g;
            const bool live = hh < a.G;
            const size_t at = (size_t)row * a.q.ts + (size_t)(kvh * a.G + hh) * a.q.hs + 2 * t;
            if (QT == 1) {
                const T *src = static_cast<const T *>(a.q.p) + at;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        q[0][i][k][u] = live ? lfq::ld(reinterpret_cast<const unsigned *>(src + 16 * k + 8 * u)) : 0u;
                f[i][0] = f[i][1] = base;
            } else {
                const float *src = static_cast<const float *>(a.q.p) + at;
                float2 x[KS][2];
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        x[k][u] = live ? lfq::ld(reinterpret_cast<const float2 *>(src + 16 * k + 8 * u)) : make_float2(0.f, 0.f);
                        top = fmaxf(top, fmaxf(fabsf(x[k][u].x), fabsf(x[k][u].y)));
                    }
                // a power of two brings the row to [1, 2): the terms' remainders stay in FP16's range, and BF16's
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float r = lfq::range_factor(top), rq = a.scale < 0.f ? -r : r;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        unsigned w[QT];
                        split_pair<T, QT>(x[k][u].x * rq, x[k][u].y * rq, w);
#pragma unroll
                        for (int n = 0; n < QT; ++n) {
                            if constexpr (!QS) q[n][i][k][u] = w[n];
                            else if (k % warps == warp) sts(q_at(n, i, k, lane) + 4 * u, w[n]);
                        }
                    }
                f[i][0] = fminf(base / __shfl_sync(0xffffffffu, r, 8 * t), FLT_MAX);       // rows 2t and 2t + 1 of the tile
                f[i][1] = fminf(base / __shfl_sync(0xffffffffu, r, 8 * t + 4), FLT_MAX);
            }
            ref[i][0] = ref[i][1] = -INFINITY;
            l[i][0] = l[i][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) o[i][k][0] = o[i][k][1] = o[i][k][2] = o[i][k][3] = 0.f;
        }
    }

    // The scale's sign on a 16-bit q, once the first copies are on their way: begin() does not wait for its loads.
    __device__ __forceinline__ void sign(const Attn &a)
    {
        if constexpr (QT == 1) {
            if (a.scale < 0.f) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int k = 0; k < KS; ++k) q[0][i][k][0] ^= 0x80008000u, q[0][i][k][1] ^= 0x80008000u;
            }
        }
    }

    // Where term n of fragment (i, k) of this lane lies.
    __device__ __forceinline__ uint32_t q_at(int n, int i, int k, int lane) const { return qs + (((n * NT + i) * KS + k) * 32 + lane) * 8; }

    // One slab from position p on, of which [lo, hi) counts; ks, vs: its rows in shared memory, 16-byte groups XOR-ed
    // with the position mod 8 (so that the 8 rows of a fragment lie in different banks).  `meanwhile` runs while the
    // scores' products are on their way.
    template <class M>
    __device__ __forceinline__ void slab(uint32_t ks, uint32_t vs, int p, int lo, int hi, int lane, M meanwhile)
    {
        const int g = lane >> 2;
        // ---- scores: position rows g, g + 8 by heads 2t, 2t + 1.  Each product waits for the one before it into the
        // same sum: CH sums, by the terms of q or by the dims in turn, are on their way at a time.
        constexpr int CH = QT > 1 ? QT : NT == 1 ? 4 : 2;
        float st[NT][4], sc[CH][NT][4];
        const uint32_t ka = ks + (lane & 15) * (HD * 2) + (((lane >> 4) ^ (lane & 7)) << 4);
        constexpr int KB = 4;                                // fragments loaded ahead of their products
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += KB) {
            unsigned x[KB][4];
#pragma unroll
            for (int k = 0; k < KB; ++k) lfk::ldsm_x4(x[k], ka ^ ((k0 + k) << 5));
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int n = 0; n < QT; ++n)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const int to = QT == 1 ? k % CH : n;
                        const bool first = QT == 1 ? k0 + k < CH : k0 + k == 0;
                        if constexpr (QS) {
                            unsigned b[2];
                            lds2(b, q_at(n, i, k0 + k, lane));
                            Half16<T>::mma(sc[to][i], x[k], b, first);
                        } else {
                            Half16<T>::mma(sc[to][i], x[k], q[n][i][k0 + k], first);
                        }
                    }
        }
        meanwhile();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                st[i][e] = sc[CH - 1][i][e];                // the smallest terms first
#pragma unroll
                for (int n = CH - 2; n >= 0; --n) st[i][e] += sc[n][i][e];
            }
        // ---- P relative to the reference, and the lanes' sums.  No maximum is formed where a lane's P sum to no more
        // than FP16 can hold; otherwise, and at the first position, the reference becomes the largest, whose P is 2^P_EXP.
        const bool whole = p >= lo && p + 16 <= hi;
        const bool in0 = whole || (p + g >= lo && p + g < hi), in1 = whole || (p + g + 8 >= lo && p + g + 8 < hi);
        float pr[NT][4], sum[NT][2];
        auto probs = [&] {
            bool bad = false;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float r = ref[i][e] == -INFINITY ? 0.f : ref[i][e];
                    const float x = ex2(fmaf(st[i][e] - r, f[i][e], P_EXP)), y = ex2(fmaf(st[i][2 + e] - r, f[i][e], P_EXP));
                    pr[i][e] = in0 ? x : 0.f;
                    pr[i][2 + e] = in1 ? y : 0.f;
                    sum[i][e] = pr[i][e] + pr[i][2 + e];
                    bad = bad || !(sum[i][e] <= P_SUM) || ref[i][e] == -INFINITY;
                }
            return bad;
        };
        if (__any_sync(0xffffffffu, probs())) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (a score of -inf is a position seen all the same: the reference -inf is for none)
                    float mx = fmaxf(in0 ? fmaxf(st[i][e], -FLT_MAX) : -INFINITY, in1 ? fmaxf(st[i][2 + e], -FLT_MAX) : -INFINITY);
#pragma unroll
                    for (int sh = 4; sh <= 16; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                    float &r = ref[i][e];
                    if (mx > r && (r == -INFINITY || (mx - r) * f[i][e] > P_EXP + 1.f)) {
                        const float alpha = r == -INFINITY ? 0.f : ex2((r - mx) * f[i][e]);
                        l[i][e] *= alpha;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[i][k][e] *= alpha;
                            o[i][k][2 + e] *= alpha;
                        }
                        r = mx;
                    }
                }
            probs();
        }
        // ---- O^T += V^T P^T
        unsigned pb[PT][NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            l[i][0] += sum[i][0];
            l[i][1] += sum[i][1];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                unsigned w[PT];
                split_pair<T, PT>(pr[i][2 * u], pr[i][2 * u + 1], w);
#pragma unroll
                for (int n = 0; n < PT; ++n) pb[n][i][u] = lfk::movm_t(w[n]);
            }
        }
        const uint32_t va = vs + ((lane & 7) + (lane >> 4) * 8) * (HD * 2) + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += KB) {
            unsigned x[KB][4];
#pragma unroll
            for (int k = 0; k < KB; ++k) lfk::ldsm_x4_t(x[k], va ^ ((k0 + k) << 5));
            // The products' own sums are cut off, not rounded, at each step: a slab's is formed from zero, and added with
            // rounding (FP32, 11,000 positions in one warp: 2.8e-6 off without; 16-bit types lost 6e-5 per 1,000 slabs).
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float y[KB][4];
#pragma unroll
                for (int n = PT - 1; n >= 0; --n)
#pragma unroll
                    for (int k = 0; k < KB; ++k) Half16<T>::mma(y[k], x[k], pb[n][i], n == PT - 1);
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][k0 + k][e] += y[k][e];
            }
        }
    }

    // The sums of all positions (each lane holds those of its rows), and the references in log2 units.
    __device__ __forceinline__ void sums()
    {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int sh = 4; sh <= 16; sh <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], sh);
                if (ref[i][e] != -INFINITY) ref[i][e] = fmaxf(ref[i][e] * f[i][e], -FLT_MAX);
            }
    }
    // The state as it lies in the lanes: O as [NT][KS][lane] x 4, then (reference, sum) of each head.
    __device__ __forceinline__ void store_state(float *dst, int lane) const
    {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < KS; ++k)
                *reinterpret_cast<float4 *>(dst + ((i * KS + k) * 32 + lane) * 4) =
                    make_float4(o[i][k][0], o[i][k][1], o[i][k][2], o[i][k][3]);
        if (lane < 4) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *reinterpret_cast<float4 *>(dst + RT * HD + (8 * i + 2 * lane) * 2) =
                    make_float4(ref[i][0], l[i][0], ref[i][1], l[i][1]);
        }
    }
};

// Two heads' outputs of dims 16 k + g and + 8, normalised: v = O of (head 0, head 1) at both dims; ml: reference and sum of
// head 0, then of head 1.  A head that saw no position (reference -inf) gives zeros, one whose scores were all -inf NaN.
template <int HD, int NT, class O>
__device__ __forceinline__ void store_out(const Attn &a, int row, int ht, int i, int k, int lane, float4 v, float4 ml)
{
    const int g = lane >> 2, t = lane & 3;
    const int kvh = ht / a.tiles, hh = (ht - kvh * a.tiles) * 8 * NT + 8 * i + 2 * t;
    auto inverse = [](float m, float l) { return l > 0.f ? 1.0f / l : m == -INFINITY ? 0.f : NAN; };
    const float r0 = inverse(ml.x, ml.y), r1 = inverse(ml.z, ml.w);
    O *dst = static_cast<O *>(a.o.p) + (size_t)row * a.o.ts + (size_t)(kvh * a.G + hh) * a.o.hs + 16 * k + g;
    auto put = [](O *p, float x) {
        if constexpr (sizeof(O) == 4) *p = x;
        else *p = Half16<O>::from(x);
    };
    if (hh < a.G) {
        put(dst, v.x * r0);
        put(dst + 8, v.z * r0);
    }
    if (hh + 1 < a.G) {
        put(dst + a.o.hs, v.y * r1);
        put(dst + a.o.hs + 8, v.w * r1);
    }
}

// States of the same heads added up, relative to the largest reference so far; a thread holds two heads at two dims.
struct Joined {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    // ml: reference and sum of head 0, then of head 1
    __device__ __forceinline__ void add(float4 ml, float4 x)
    {
        const float n0 = fmaxf(m0, ml.x), n1 = fmaxf(m1, ml.z);
        const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
        const float a0 = ex2(m0 - z0), b0 = ex2(ml.x - z0), a1 = ex2(m1 - z1), b1 = ex2(ml.z - z1);
        m0 = n0;
        m1 = n1;
        l0 = fmaf(ml.y, b0, l0 * a0);
        l1 = fmaf(ml.w, b1, l1 * a1);
        v.x = fmaf(x.x, b0, v.x * a0);
        v.z = fmaf(x.z, b0, v.z * a0);
        v.y = fmaf(x.y, b1, v.y * a1);
        v.w = fmaf(x.w, b1, v.w * a1);
    }
    __device__ __forceinline__ float4 ml() const { return make_float4(m0, l0, m1, l1); }
};

// The ring of one warp, and where its slabs come from.
template <int HD>
struct Feed {
    using R = Ring<HD>;
    static constexpr int CPR = HD / 8, RPI = 32 / CPR, N = 16 / RPI;   // 16-byte groups a row, rows per instruction, instructions
    uint32_t base;
    int lane;
    long long place;   // this lane's entry of the next 32 slabs: byte offset in the pools, -1 for none
    long long next;    // the next slab's (looked up ahead: a shuffle takes as long as two copies)
    unsigned none;     // bit st: stage st holds zeros, its slab lies on no page of the pool

    // Looks the places of slabs s, s + step, .. (below end) up, one per lane.
    __device__ __forceinline__ void look_up(const Attn &a, int row, int kvh, int s, int step, int end)
    {
        const int pp = a.c.page >> 4, mine = s + lane * step;
        place = -1;
        if (mine < end) {
            const int col = mine / pp;
            const int id = lfq::ld(a.tables + (size_t)row * a.tstride + col);
            if ((unsigned)id < (unsigned)a.c.n_pages)
                place = id * a.c.page_b + kvh * a.c.head_b + (long long)((mine - col * pp) * 16) * a.c.pos_b;
        }
        next = __shfl_sync(0xffffffffu, place, 0);
    }
    // Begins the copies of the slab at position p, of which [lo, hi) counts, into stage `st`; it is the j-th that was
    // looked up.
    __device__ __forceinline__ void fetch(const Attn &a, int st, int j, int p, int lo, int hi)
    {
        const int r0 = lane / CPR, c = lane % CPR;
        // row r = i RPI + r0, and (r mod 8) = (i RPI mod 8) xor r0
        const uint32_t dst = base + st * 2 * R::SLAB + r0 * (HD * 2), swz = (uint32_t)(c ^ r0) << 4;
        auto to = [&](int i) { return dst + i * RPI * (HD * 2) + (swz ^ (i * RPI % 8 << 4)); };
        const bool gone = next < 0;
        const char *k = a.c.k + next + r0 * a.c.pos_b + c * 16, *v = k + (a.c.v - a.c.k);
        const long long step = RPI * a.c.pos_b;
        none = gone ? none | 1u << st : none & ~(1u << st);
        if (!gone && p >= lo && p + 16 <= hi) {
#pragma unroll
            for (int i = 0; i < N; ++i) copy16(to(i), k + i * step);
#pragma unroll
            for (int i = 0; i < N; ++i) copy16(to(i) + R::SLAB, v + i * step);
        } else {
            // rows that do not count become zeros (what they hold may be anything, and 0 x inf is not 0)
            for (int i = 0; i < N; ++i) {
                const int r = i * RPI + r0;
                const bool in = !gone && p + r >= lo && p + r < hi;
                copy16(to(i), in ? k + i * step : a.c.k, in ? 16u : 0u);
                copy16(to(i) + R::SLAB, in ? v + i * step : a.c.v, in ? 16u : 0u);
            }
        }
        next = __shfl_sync(0xffffffffu, place, j + 1);
    }
};

// ---------------------------------------------------------------- clusters

// A sequence's slabs for one tile of query heads (an item) are taken by `parts` clusters of `cl` CTAs of CW warps: a
// stretch for each part, whose slabs the cluster's warps take in turn (neighbours in memory are read at the same time,
// which DRAM rewards).  The warps' states are joined in shared memory, the CTA's first, then the cluster's; where
// there is one part that is the output, in one launch, else a second one joins the parts.  How many parts a sequence
// really needs, its length says: every warp gets MIN_SLABS slabs before there is another part.
constexpr int MIN_SLABS = 4;
__device__ __forceinline__ int parts_of(const Attn &a, int slabs)
{
    return min(a.parts, max(1, slabs / (a.cl * a.cw * MIN_SLABS)));
}

// The row that comes `rank`-th where long ones come first: in classes of like numbers of slabs (two per octave), in row
// order within one.  Where the clusters come in several rounds the last one then is of short rows (200 rows of up to
// 20,000 positions, most of them short, FP32 queries: 160 us, 191 in row order).  Called by all threads; `scratch`: 65 words
// of shared memory, free again after the next barrier.
__device__ __forceinline__ int row_by_length(const Attn &a, int rank, int *scratch)
{
    auto class_of = [&](int r) {
        const int n = Seen(a, lfq::ld(a.lens + r)).slabs();
        if (n == 0) return 0;
        const int top = 31 - __clz(n);                       // 0 .. 26
        return 2 * top + 1 + (top ? n >> (top - 1) & 1 : 0);  // 1 .. 54
    };
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 64) scratch[threadIdx.x] = 0;
    __syncthreads();
    for (int r = threadIdx.x; r < a.n; r += blockDim.x) atomicAdd(scratch + class_of(r), 1);
    __syncthreads();
    if (threadIdx.x < 32) {
        // lane l: classes 63 - 2 l and 62 - 2 l, the longest first
        const int x = scratch[63 - 2 * lane], y = scratch[62 - 2 * lane];
        int incl = x + y;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += z;
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, incl > rank)) - 1;    // (all rows are counted: there is one)
        const int before = __shfl_sync(0xffffffffu, incl - x - y, at), first = __shfl_sync(0xffffffffu, x, at);
        int left = rank - before, cls = 63 - 2 * at;
        if (left >= first) left -= first, --cls;
        for (int base = 0; base < a.n; base += 32) {
            const bool mine = base + lane < a.n && class_of(base + lane) == cls;
            unsigned set = __ballot_sync(0xffffffffu, mine);
            const int count = __popc(set);
            if (left < count) {
                while (left--) set &= set - 1;
                if (lane == 0) scratch[64] = base + __ffs(set) - 1;
                break;
            }
            left -= count;
        }
    }
    __syncthreads();
    return scratch[64];
}

template <int HD, int NT, class T, int QT, int CW>
__global__ void __launch_bounds__(CW * 32, 8 / CW) attn_cluster(const __grid_constant__ Attn a)
{
    using W = Work<HD, NT, T, QT>;
    using R = Ring<HD>;
    using O = std::conditional_t<QT == 1, T, float>;
    constexpr int STATE = W::RT * (HD + PADF), KS = W::KS, F = NT * KS * 32;
    static_assert((CW + 1) * STATE * 4 <= CW * R::COPIES, "the states take the ring's memory");
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    lfq::dependents_may_launch();
    lfq::wait_for_prerequisites();
    const int rank = blockIdx.x % a.cl, cluster = blockIdx.x / a.cl;
    const int item = cluster / a.parts, part = cluster - item * a.parts, ht = item % a.ht;
    const int row = a.sorted ? row_by_length(a, item / a.ht, reinterpret_cast<int *>(smem)) : item / a.ht;
    if (a.sorted) __syncthreads();
    const int me = rank * CW + warp, kvh = ht / a.tiles;
    Feed<HD> feed;
    feed.lane = lane;
    feed.base = lfk::smem_u32(smem) + warp * R::COPIES;
    feed.none = 0;
    Seen seen(a, lfq::ld(a.lens + row));
    const int parts = parts_of(a, seen.slabs());
    if (part >= parts) return;   // (all CTAs of the cluster)
    if (parts > 1) {
        const int n = seen.slabs(), s0 = seen.s0;
        seen.s0 = s0 + (int)((long long)n * part / parts);
        seen.s1 = s0 + (int)((long long)n * (part + 1) / parts);
    }
    // A short row needs fewer CTAs: the others leave, and the cluster's barriers count those that are left.
    const int cl = max(1, min(a.cl, seen.slabs() / (CW * 2))), nw = cl * CW;
    if (rank >= cl) return;
    feed.look_up(a, row, kvh, seen.s0 + me, nw, seen.s1);
    W work;
    work.qs = lfk::smem_u32(smem) + CW * R::COPIES;
    work.begin(a, row, ht, warp, CW, lane);
    if (W::QS) __syncthreads();
    int s = seen.s0 + me, j = 0;
    auto issue = [&](int st) {
        if (s < seen.s1) {
            if (j == 32) {
                j = 0;
                feed.look_up(a, row, kvh, s, nw, seen.s1);
            }
            feed.fetch(a, st, j, s * 16, seen.lo, seen.hi);
            ++j;
            s += nw;
        }
        copies_commit();
    };
#pragma unroll 1
    for (int i = 0; i < R::STAGES - 1; ++i) issue(i);
    work.sign(a);
    int st = 0;
#pragma unroll 1
    for (int x = seen.s0 + me; x < seen.s1; x += nw) {
        copies_wait<R::STAGES - 2>();
        __syncwarp();
        const uint32_t ks = feed.base + st * 2 * R::SLAB;
        work.slab(ks, ks + R::SLAB, x * 16, seen.lo, feed.none >> st & 1 ? 0 : seen.hi, lane, [&] { issue(st == 0 ? R::STAGES - 1 : st - 1); });
        st = st + 1 == R::STAGES ? 0 : st + 1;
    }
    work.sums();
    copies_wait<0>();
    __syncthreads();             // the states take the ring's memory
    float *states = reinterpret_cast<float *>(smem), *own = states + CW * STATE;
    float *const out = parts > 1 ? a.part + ((size_t)item * a.parts + part) * STATE : nullptr;   // a partial state
    auto finish = [&](const Joined &x, int f, int i, int k, int ln, int ml) {
        if (out) {
            *reinterpret_cast<float4 *>(out + f * 4) = x.v;
            if (k == 0 && ln < 4) *reinterpret_cast<float4 *>(out + ml) = x.ml();
        } else {
            store_out<HD, NT, O>(a, row, ht, i, k, ln, x.v, x.ml());
        }
    };
    work.store_state(states + warp * STATE, lane);
    __syncthreads();
    for (int f = threadIdx.x; f < F; f += CW * 32) {
        const int i = f / (KS * 32), k = f / 32 % KS, ln = f % 32, ml = W::RT * HD + (8 * i + 2 * (ln & 3)) * 2;
        Joined x;
#pragma unroll
        for (int w = 0; w < CW; ++w)
            x.add(*reinterpret_cast<const float4 *>(states + w * STATE + ml), *reinterpret_cast<const float4 *>(states + w * STATE + f * 4));
        if (cl == 1) {
            finish(x, f, i, k, ln, ml);
        } else {
            *reinterpret_cast<float4 *>(own + f * 4) = x.v;
            if (k == 0 && ln < 4) *reinterpret_cast<float4 *>(own + ml) = x.ml();
        }
    }
    if (cl == 1) return;
    lfq::cluster_sync();
    for (int f = rank * CW * 32 + threadIdx.x; f < F; f += nw * 32) {
        const int i = f / (KS * 32), k = f / 32 % KS, ln = f % 32, ml = W::RT * HD + (8 * i + 2 * (ln & 3)) * 2;
        Joined x;
        for (int c = 0; c < cl; ++c) {
            const uint32_t base = lfq::cluster_smem(own, c);
            x.add(lfq::ld_cluster4(base + ml * 4), lfq::ld_cluster4(base + f * 16));
        }
        finish(x, f, i, k, ln, ml);
    }
    lfq::cluster_sync();         // no CTA leaves while its state may be read
}

// Joins the parts of the items that have more than one.  A block takes 256 / groups of the 16-byte places of a state's O
// (dims and heads), `groups` threads each: thread `grp` adds every groups-th part.
constexpr int JOIN_THREADS = 256;
template <int HD, int NT, class O>
__global__ void __launch_bounds__(JOIN_THREADS, 4) attn_join(const __grid_constant__ Attn a, int groups)
{
    constexpr int KS = HD / 16, F = NT * KS * 32, RT = 8 * NT, STATE = RT * (HD + PADF);
    __shared__ float4 sh[2][JOIN_THREADS];
    lfq::dependents_may_launch();
    lfq::wait_for_prerequisites();
    const int per = JOIN_THREADS / groups, blocks = F / per;    // places a block; blocks an item
    const int item = blockIdx.x / blocks, row = item / a.ht, ht = item - row * a.ht;
    const int f = (blockIdx.x - item * blocks) * per + threadIdx.x % per, grp = threadIdx.x / per;
    const int parts = parts_of(a, Seen(a, lfq::ld(a.lens + row)).slabs());
    if (parts == 1) return;                                    // it has its output
    const int i = f / (KS * 32), k = f / 32 % KS, lane = f % 32;
    Joined j;
    constexpr int AHEAD = 4;                                   // loads on the way at a time
    for (int p0 = grp; p0 < parts; p0 += AHEAD * groups) {
        float4 ml[AHEAD], v[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            const int p = p0 + x * groups;
            if (p >= parts) continue;
            const float *src = a.part + ((size_t)item * a.parts + p) * STATE;
            ml[x] = lfq::ld(reinterpret_cast<const float4 *>(src + RT * HD + (8 * i + 2 * (lane & 3)) * 2));
            v[x] = lfq::ld(reinterpret_cast<const float4 *>(src + f * 4));
        }
#pragma unroll
        for (int x = 0; x < AHEAD; ++x)
            if (p0 + x * groups < parts) j.add(ml[x], v[x]);
    }
    // the groups, pairwise
    for (int half = groups >> 1; half; half >>= 1) {
        __syncthreads();
        sh[0][threadIdx.x] = j.ml();
        sh[1][threadIdx.x] = j.v;
        __syncthreads();
        if (grp < half) j.add(sh[0][threadIdx.x + half * per], sh[1][threadIdx.x + half * per]);
    }
    if (grp == 0) store_out<HD, NT, O>(a, row, ht, i, k, lane, j.v, j.ml());
}

// ---------------------------------------------------------------- launches

template <int HD, int NT, class T, int QT>
static cudaError_t run(const Attn &a, cudaStream_t s)
{
    using O = std::conditional_t<QT == 1, T, float>;
    static bool ready[2][64] = {};
    auto go = [&](auto warps, bool (&ready)[64]) {
        constexpr int CW = decltype(warps)::value, smem = CW * Ring<HD>::COPIES + Work<HD, NT, T, QT>::Q_BYTES;
        const cudaError_t e = lfr::allow_smem(attn_cluster<HD, NT, T, QT, CW>, smem, ready);
        if (e != cudaSuccess) return e;
        return lfr::launch(attn_cluster<HD, NT, T, QT, CW>, dim3((unsigned)(a.n * a.ht * a.parts * a.cl)), CW * 32, smem, a.cl, s, a);
    };
    const cudaError_t e = a.cw == 4 ? go(std::integral_constant<int, 4>(), ready[0]) : go(std::integral_constant<int, 8>(), ready[1]);
    if (e != cudaSuccess || a.parts == 1) return e;
    constexpr int F = NT * (HD / 16) * 32;
    int groups = JOIN_THREADS / F > 1 ? JOIN_THREADS / F : 1;
    while (groups < 16 && groups * 4 < a.parts) groups *= 2;
    return lfr::launch(attn_join<HD, NT, O>, dim3((unsigned)(a.n * a.ht * (F * groups / JOIN_THREADS))), JOIN_THREADS, 0, 1, s, a, groups);
}

template <class T, int QT>
static cudaError_t run(const Attn &a, cudaStream_t s)
{
    if (a.c.hd == 128) return a.rt == 8 ? run<128, 1, T, QT>(a, s) : run<128, 2, T, QT>(a, s);
    return a.rt == 8 ? run<64, 1, T, QT>(a, s) : run<64, 2, T, QT>(a, s);
}

void set_workspace(Attn &a, void *ws) { a.part = static_cast<float *>(ws); }

cudaError_t launch_attn(const Attn &a, cudaStream_t s)
{
    if (a.c.bf16) return a.q.dtype == LF_F32 ? run<__nv_bfloat16, 3>(a, s) : run<__nv_bfloat16, 1>(a, s);
    return a.q.dtype == LF_F32 ? run<__half, 2>(a, s) : run<__half, 1>(a, s);
}

}  // namespace lfpg
