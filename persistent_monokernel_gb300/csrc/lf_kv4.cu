// lf_kv4.cu -- a KV cache held in 4 bits: rows quantised as they are written,
// read back, and attended to without a wider copy.
//
// Format.  A row of head_dim values is cut into blocks of 16.  A block with
// largest magnitude A is stored as the scale s = E4M3(A / 6) and the codes
// c_i = E2M1(x_i / s), both rounded to nearest, ties to even; its values are
// s c_i.  s has 4 significant bits and c_i two, so every value has at most 6
// and lies in 2^-10 .. 2,688: exact in FP16 and BF16.  The products of the
// attention therefore see the cache's values themselves, and dequantising
// costs no accuracy.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/lf.h"
#include "lf_kv4.h"
#include "lf_kv4.cuh"
#include "lf_internal.cuh"
#include "lf_ptx.cuh"
#include "lf_rows.cuh"

namespace lfq {

using lfr::launch;

// ---------------------------------------------------------------- append and read

// One thread per block of 16 values, one grid row per KV head and K or V (no division finds a thread's row).
// Non-finite inputs: an infinity counts as the largest finite value (the block then saturates), a NaN as 0, so
// that the cache holds finite values only and a masked position can never reach a result.
//
// x / s decides which code is nearest, and only its side of a half-way value t counts.  With r = 1 / s rounded,
// q = x r corrected once by its exact remainder x - q s is the quotient rounded to nearest, to about 2^-46 before
// that rounding; and an FP32 x other than t s is at least mant(t) / mant(t s) >= 1 / 1.875 steps of t away from it
// in the quotient, more than the half step that would round it to t.  So the codes are those of the exact quotient
// (the same holds for A / 6 and the scales' half-way values).
//
// Bound by memory, the arithmetic close behind: 32,767 positions of 5 heads x 128 take 18.8 us from FP16 (5.7 TB/s)
// and 29 from FP32 (6.5 TB/s), a copy's rate being 6.7; one position takes 1.3 us.  Products two to an
// instruction: 21.8 us without.  One block a thread: the loads in flight come from many threads of few registers (two
// blocks of raw bytes a thread: 18.1 us, but 2.0 instead of 1.6 at 777 positions).
template <class T>
__global__ void __launch_bounds__(256) append_rows(Cache c, Rows k, Rows v, int n, int pos, int shift)
{
    dependents_may_launch();
    wait_for_prerequisites();
    const bool isv = blockIdx.y & 1;
    const int h = blockIdx.y >> 1;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, t = i >> shift;   // 2^shift blocks per row
    const int b = (int)(i & ((1 << shift) - 1));
    if (t >= n) return;
    const Rows &in = isv ? v : k;
    float x[16];
    unsigned top = load_block<T>(in, t, h, b, x);
    if (top >= 0x7f800000u) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = x[j] != x[j] ? 0.f : fminf(fmaxf(x[j], -3.402823466e38f), 3.402823466e38f);
        top = top_of(x);
    }
    const unsigned s8 = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(top), 6.0f), __NV_SATFINITE, __NV_E4M3);
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3)));
    unsigned w[2] = {0u, 0u};
    if (s > 0.f) {   // a block below E4M3's range (A < 6 * 2^-10) is stored as zeros
        const float r = __frcp_rn(s);
        const uint64_t rr = pack2(r, r), ss = pack2(-s, -s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t v = pack2(x[2 * j], x[2 * j + 1]), q = mul2(v, rr);
            const float2 y = unpack2(fma2(fma2(q, ss, v), rr, q));   // -q s + x = q (-s) + x
            w[j / 4] |= e2m1x2(y.x, y.y) << (8 * (j % 4));
        }
    }
    const size_t row = (size_t)h * c.cap + (size_t)pos + (size_t)t;
    *reinterpret_cast<uint2 *>((isv ? c.vc : c.kc) + row * code_bytes(c.hd) + b * 8) = make_uint2(w[0], w[1]);
    ((isv ? c.vs : c.ks) + row * scale_bytes(c.hd))[b] = (uint8_t)s8;
}

// A thread takes 16 bytes of the output (8 values, 4 in FP32) of READ_U places 256 apart: a warp's stores are
// contiguous, and each thread has several loads on their way.  Bound by the stores: 32,767 positions of 5 heads x 128
// take 15.6 us in FP16 (6.9 TB/s; 20.9 with a division per place), one position 1.1 us.
constexpr int READ_U = 4;
template <class T>
__global__ void __launch_bounds__(256) read_rows(Cache c, Rows k, Rows v, int n, int pos, int shift)
{
    constexpr int N = 16 / sizeof(T);
    dependents_may_launch();
    wait_for_prerequisites();
    const bool isv = blockIdx.y & 1;
    const int h = blockIdx.y >> 1;
    const long long i0 = (long long)blockIdx.x * (256 * READ_U) + threadIdx.x;              // 2^shift places per row
    const int b = (int)(threadIdx.x & ((1 << shift) - 1));                                  // 256 is a multiple of it
    const size_t row0 = (size_t)h * c.cap + (size_t)pos;
    const uint8_t *codes = (isv ? c.vc : c.kc) + row0 * code_bytes(c.hd) + b * (N / 2);
    const uint8_t *scales = (isv ? c.vs : c.ks) + row0 * scale_bytes(c.hd) + b * N / 16;
    unsigned w[READ_U], s[READ_U];
#pragma unroll
    for (int u = 0; u < READ_U; ++u) {
        const long long t = (i0 + u * 256) >> shift;
        if (t >= n) continue;
        w[u] = N == 8 ? ld(reinterpret_cast<const unsigned *>(codes + t * code_bytes(c.hd)))
                      : ld(reinterpret_cast<const unsigned short *>(codes + t * code_bytes(c.hd)));
        s[u] = ld(scales + t * scale_bytes(c.hd));
    }
    const Rows &out = isv ? v : k;
    T *dst = static_cast<T *>(out.p) + h * out.hs + b * N;
#pragma unroll
    for (int u = 0; u < READ_U; ++u) {
        const long long t = (i0 + u * 256) >> shift;
        if (t >= n) continue;
        const unsigned s2 = e4m3_h2_same(s[u]);
        unsigned hv[4];
        e2m1x8_h2(w[u], hv[0], hv[1], hv[2], hv[3]);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) hv[j] = hmul2(hv[j], s2);
        store_values(dst + t * out.ts, hv);
    }
}

// ---------------------------------------------------------------- attention, few rows

// A tile of 8 NT query rows of one KV head against the positions of one split.
//
// The contraction runs on warp-level tensor-core products (m16n8k16, FP16
// operands, FP32 sums) whose operands come straight from the cache's bytes in
// global memory, with no pass through shared memory: the order of the
// contracted index is free, so each lane takes the bytes that lie together.
//   S^T = K Q^T   A = 16 positions x 16 dims of K.  Lane (g, t) holds dims
//                 [HD/4 t, HD/4 (t+1)) of two positions: one wide load each;
//                 k-step s uses 4 of them.
//   O^T = V^T P^T A = 16 dims x 16 positions of V.  Lane (g, t) holds dims
//                 [HD/8 g, HD/8 (g+1)) of the positions 4t .. 4t + 3; the codes of
//                 two positions are woven nibble by nibble, so that one
//                 conversion yields the pair of positions the product wants.
// The position of row i of a 16-position slab is 4 (i / 2) + i % 2 for i < 8
// and 2 more for i + 8, the same in both products, so that the scores become
// the second product's operand by one 8x8 transpose in registers.
//
// The softmax is online, FP32, exponentials to base 2.  P is taken relative to a
// reference of the row, and no maximum is formed on the common path: a lane whose
// P sum to at most 2^15 has none that FP16 could not hold.  Otherwise, and at a
// row's first position, the maximum over the chunk is taken, the reference put
// 2^P_EXP below it and O and l rescaled.  P is rounded to FP16: relative error
// 2^-11, below that of a half-precision output, down to 2^-(14 + P_EXP) of the
// row's largest, where FP16 runs out of exponents.  With FP32 queries (SPLIT) q
// and P are split into an FP16 head and remainder and the products are formed
// twice, which leaves errors near 2^-22.
//
// What bounds it: the wait for loads, and in short contexts latency.  A warp loads a
// chunk and then works on it, with nothing of its own on the way meanwhile; 16 warps
// an SM do not cover that (waiting for a load is the largest stall, 2.6 warps per
// issue, while neither the issue slots, at 52 %, nor memory is at its limit).
// A cached value costs a conversion and a multiply by its scale per pair, half an
// instruction to bring its byte to the converter, and its share of the product;
// everything else is kept off the loop (addresses advance by constants, no maximum,
// no rescaling).  One token over 131,072 positions of 8 KV heads x 128: 39.4 us, 3.8 TB/s
// of 6.7 (65 us with a maximum per chunk, 48 before clusters joined); over 512
// positions of 5 heads: 4.5 us.  FP16 values through shared memory
// would write and read four times the cache's bytes there; its raw bytes, loaded ahead
// of their use, would cost no registers and were not tried.  The next chunk's loads
// one phase ahead in registers gained 4 % at 131,072, but lost 3 % with FP32 queries and 8 % at 512
// (two slabs), as they run out; a third CTA per SM costs 75 % (spills).
__device__ __forceinline__ void add_scaled(float4 &acc, const float4 &v, float x)
{
    acc.x = fmaf(v.x, x, acc.x);
    acc.y = fmaf(v.y, x, acc.y);
    acc.z = fmaf(v.z, x, acc.z);
    acc.w = fmaf(v.w, x, acc.w);
}
// Partial softmax states (reference M, sum L, four of the row's outputs) added up, relative to the largest
// reference so far: O = sum 2^(M_s - M) O_s, L likewise.
struct Joined {
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float2 ml, float4 v)
    {
        const float n = fmaxf(M, ml.x), m = n == -INFINITY ? 0.f : n;
        const float x = ex2(M - m), y = ex2(ml.x - m);      // 0 from -inf
        M = n;
        L = fmaf(ml.y, y, L * x);
        acc = make_float4(acc.x * x, acc.y * x, acc.z * x, acc.w * x);
        add_scaled(acc, v, y);
    }
    // row = token * G + head of the group
    __device__ __forceinline__ void store(const Attn &a, int row, int kvh, int d) const
    {
        const float inv = L > 0.f ? 1.0f / L : (L == 0.f ? 0.f : L);   // a row that saw nothing is 0; NaN stays
        const int tt = row_token(a, row), hh = row_head(a, kvh, row, tt);
        store4(a.o, (size_t)tt * a.o.ts + (size_t)hh * a.o.hs + d, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
};

template <int HD, int NT, bool SPLIT>
struct RowCfg {
    static constexpr int NW = 8;                       // warps
    static constexpr int RT = 8 * NT;                  // query rows
    static constexpr int KS = HD / 16;                 // k-steps of S, m-tiles of O
    static constexpr int QW = SPLIT ? 4 : 2;           // words per q fragment
    static constexpr int SMEM = NT * KS * 32 * QW * 4 + (2 * NW + 1) * RT * 4 + NW * RT * HD * 4 +
                                RT * (HD + PAD) * 4;
};
constexpr float P_EXP = 7.f, P_SUM = 32768.f;

// SL: slabs of 16 positions per chunk.
template <int HD, int NT, bool SPLIT, int SL>
__global__ void __launch_bounds__(256, NT == 1 ? 2 : 1) attn_rows(const __grid_constant__ Attn a)
{
    using C = RowCfg<HD, NT, SPLIT>;
    constexpr int NW = C::NW, RT = C::RT, KS = C::KS, CH = 16 * SL;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    unsigned *qf = reinterpret_cast<unsigned *>(smem_raw);              // [NT][KS][32][QW]
    float *rs = reinterpret_cast<float *>(qf + NT * KS * 32 * C::QW);   // [RT] score factor of a row
    float *wm = rs + RT, *wl = wm + NW * RT;                            // [NW][RT]
    float *wo = wl + NW * RT;                                           // [NW][RT][HD]
    float *cs = wo + NW * RT * HD;                                      // [RT][HD + PAD] the CTA's state, for its cluster
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kvh = blockIdx.y, split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
    const int r0 = tile * RT, rows = min(RT, a.n * a.G - r0);
    dependents_may_launch();
    wait_for_prerequisites();                            // the rows appended just before, q

    // ---- q: row r as an FP16 B operand, scaled by a power of two for BF16 and FP32 (their
    // range is wider than FP16's), which the row's score factor takes back; then this lane's rows 2t, 2t + 1 of
    // each n-tile: visible keys and score factors
    int khi[NT][2], klo[NT][2];
    float f[NT][2];
    auto prepare_q = [&] {
        for (int r = warp; r < RT; r += NW) {
            float x[HD / 32];
            const int tt = row_token(a, r0 + r), hh = row_head(a, kvh, r0 + r, tt);
            const bool live = r < rows;
            load_q<HD>(a.q, live, tt, hh, lane, x);
            float f = 1.f;
            if (a.q.dtype != F16) f = range_factor(warp_amax<HD / 32>(x));
            if (lane == 0) rs[r] = a.scale * 1.4426950408889634f / f;
            // dims HD/32 lane ..: element d of the row belongs to lane t = d / (HD/4), k-step (d % (HD/4)) / 4
#pragma unroll
            for (int j = 0; j < HD / 32; j += 2) {
                const int d = lane * (HD / 32) + j, qt = d / (HD / 4), k = d % (HD / 4) / 4, w = d % 4 / 2;
                unsigned *dst = qf + (((r / 8) * KS + k) * 32 + (r % 8) * 4 + qt) * C::QW;
                __half h0, m0, h1, m1;
                lfk::split_h(x[j] * f, h0, m0);
                lfk::split_h(x[j + 1] * f, h1, m1);
                dst[w] = lfk::pack_h2(h0, h1);
                if (SPLIT) dst[2 + w] = lfk::pack_h2(m0, m1);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * t + e, tt = row_token(a, r0 + min(r, rows - 1));
                khi[i][e] = key_hi(a.pos, tt, a.len);
                klo[i][e] = key_lo(a.pos, tt, a.win);
                f[i][e] = rs[r];
            }
    };
    // positions of this CTA: the split's, cut to what the tile's rows see
    const int t_first = row_token(a, r0), t_last = row_token(a, r0 + rows - 1);
    const int lo_t = key_lo(a.pos, t_first, a.win), hi_r = key_hi(a.pos, t_last, a.len);
    const int hi_t = hi_r > lo_t ? hi_r : 0;              // no position at all: an empty range
    const int p0 = max(a.lo + split * a.per, lo_t), p1 = min(a.lo + (split + 1) * a.per, hi_t);
    // inside [all_lo, all_hi) every row sees every position
    const int all_lo = key_lo(a.pos, t_last, a.win), all_hi = min(key_hi(a.pos, t_first, a.len), p1);

    float ref[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        ref[i][0] = ref[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) o[i][k][0] = o[i][k][1] = o[i][k][2] = o[i][k][3] = 0.f;
    }
    const int sg = 4 * (g >> 1) + (g & 1);                 // slab position of rows g (and + 2: of g + 8)
    const size_t first = (size_t)kvh * a.c.cap + (size_t)(p0 + warp * CH);
    const uint8_t *kc = a.c.kc + first * code_bytes(HD) + t * (HD / 8);
    const uint8_t *ks = a.c.ks + first * scale_bytes(HD) + t * (HD / 64);
    const uint8_t *vc = a.c.vc + first * code_bytes(HD) + g * (HD / 16);
    const uint8_t *vs = a.c.vs + first * scale_bytes(HD) + g * (HD / 16) / 8;

    prepare_q();
    // One chunk: SL slabs of 16 positions from p on.  Positions past the end read the last row that counts, and are
    // masked.
    struct Raw {
        KRaw<HD> k[SL][2];
        VRaw<HD> v[SL][4];
    };
    auto load = [&](Raw &w, int p) {
        auto rows = [&](auto row) {
#pragma unroll
            for (int s = 0; s < SL; ++s) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = row(16 * s + sg + 2 * e);
                    w.k[s][e].load(kc + r * code_bytes(HD), ks + r * scale_bytes(HD));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = row(16 * s + 4 * t + e);
                    w.v[s][e].load(vc + r * code_bytes(HD), vs + r * scale_bytes(HD));
                }
            }
        };
        if (p + CH <= p1) rows([](int r) { return r; });
        else rows([&](int r) { return min(r, p1 - 1 - p); });
        kc += (size_t)NW * CH * code_bytes(HD);
        ks += (size_t)NW * CH * scale_bytes(HD);
        vc += (size_t)NW * CH * code_bytes(HD);
        vs += (size_t)NW * CH * scale_bytes(HD);
    };
    auto chunk = [&](const Raw &w, int p) {
        // ---- scores
        float st[SL][NT][4];
#pragma unroll
        for (int s = 0; s < SL; ++s) {
#pragma unroll
            for (int i = 0; i < NT; ++i) st[s][i][0] = st[s][i][1] = st[s][i][2] = st[s][i][3] = 0.f;
            unsigned ka[KS][2], kb[KS][2];
            w.k[s][0].values(ka);
            w.k[s][1].values(kb);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const unsigned *q = qf + ((i * KS + k) * 32 + lane) * C::QW;
                    if (SPLIT) {
                        const uint4 b = *reinterpret_cast<const uint4 *>(q);
                        lfk::mma16816(st[s][i], ka[k][0], kb[k][0], ka[k][1], kb[k][1], b.x, b.y);
                        lfk::mma16816(st[s][i], ka[k][0], kb[k][0], ka[k][1], kb[k][1], b.z, b.w);
                    } else {
                        const uint2 b = *reinterpret_cast<const uint2 *>(q);
                        lfk::mma16816(st[s][i], ka[k][0], kb[k][0], ka[k][1], kb[k][1], b.x, b.y);
                    }
                }
        }
        // ---- P relative to the reference, and the lanes' sums
        const bool whole = p >= all_lo && p + CH <= all_hi;
        float pr[SL][NT][4], sum[NT][2];
        auto probs = [&] {
            bool bad = false;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float neg = ref[i][e] == -INFINITY ? 0.f : -ref[i][e];
                    sum[i][e] = 0.f;
#pragma unroll
                    for (int s = 0; s < SL; ++s)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float x = ex2(fmaf(st[s][i][2 * u + e], f[i][e], neg));
                            const int key = p + 16 * s + sg + 2 * u;
                            if (!whole && !(key >= klo[i][e] && key < min(khi[i][e], p1))) x = 0.f;
                            pr[s][i][2 * u + e] = x;
                            sum[i][e] += x;
                        }
                    bad = bad || !(sum[i][e] <= P_SUM) || ref[i][e] == -INFINITY;
                }
            return bad;
        };
        if (__any_sync(0xffffffffu, probs())) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int s = 0; s < SL; ++s)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int key = p + 16 * s + sg + 2 * u;
                            if (whole || (key >= klo[i][e] && key < min(khi[i][e], p1)))
                                mx = fmaxf(mx, st[s][i][2 * u + e] * f[i][e]);
                        }
#pragma unroll
                    for (int sh = 4; sh <= 16; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                    float &r = ref[i][e];
                    if (mx > r && (r == -INFINITY || mx - r > P_EXP + 1.f)) {
                        float n = mx - P_EXP;
                        if (!(mx - n <= 15.f)) n = mx;     // scores so large that their steps are
                        const float alpha = ex2(r - n);    // 0 from -inf
                        l[i][e] *= alpha;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[i][k][e] *= alpha;
                            o[i][k][2 + e] *= alpha;
                        }
                        r = n;
                    }
                }
            probs();
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            l[i][0] += sum[i][0];
            l[i][1] += sum[i][1];
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int s = 0; s < SL; ++s) {
            unsigned pb[NT][2], pm[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float x = pr[s][i][2 * u], y = pr[s][i][2 * u + 1];
                    const __half2 h = __floats2half2_rn(x, y);
                    pb[i][u] = lfk::movm_t(*reinterpret_cast<const unsigned *>(&h));
                    if (SPLIT) {
                        const float2 b = __half22float2(h);
                        const __half2 r = __floats2half2_rn(x - b.x, y - b.y);
                        pm[i][u] = lfk::movm_t(*reinterpret_cast<const unsigned *>(&r));
                    }
                }
            unsigned va[KS][2], vb[KS][2];                 // positions 4t, 4t+1 and 4t+2, 4t+3
            weave<HD>(w.v[s][0], w.v[s][1], va);
            weave<HD>(w.v[s][2], w.v[s][3], vb);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    lfk::mma16816(o[i][k], va[k][0], va[k][1], vb[k][0], vb[k][1], pb[i][0], pb[i][1]);
                    if (SPLIT) lfk::mma16816(o[i][k], va[k][0], va[k][1], vb[k][0], vb[k][1], pm[i][0], pm[i][1]);
                }
        }
    };
    for (int p = p0 + warp * CH; p < p1; p += NW * CH) {
        Raw w;
        load(w, p);
        chunk(w, p);
    }

    // ---- the warps' states, joined: O = sum 2^(m_w - M) O_w over l likewise
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * i + 2 * t + e;
            float s = l[i][e];
#pragma unroll
            for (int sh = 4; sh <= 16; sh <<= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
            if (g == 0) {
                wm[warp * RT + r] = ref[i][e];
                wl[warp * RT + r] = s;
            }
            float *dst = wo + ((size_t)warp * RT + r) * HD + g * (HD / 8);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                dst[2 * k] = o[i][k][e];
                dst[2 * k + 1] = o[i][k][2 + e];
            }
        }
    __syncthreads();
    // joined state of (row r, dims d ..): the CTA's, then over the splits
    auto state = [&](int r, int d, float &M, float &L, float4 &acc) {
        M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * RT + r]);
        const float m = M == -INFINITY ? 0.f : M;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float x = ex2(wm[w * RT + r] - m);
            L = fmaf(wl[w * RT + r], x, L);
            add_scaled(acc, *reinterpret_cast<const float4 *>(wo + ((size_t)w * RT + r) * HD + d), x);
        }
    };
    auto finish = [&](int r, int d, const Joined &j) {
        if (!a.part) {
            j.store(a, r0 + r, kvh, d);
            return;
        }
        float *part = a.part + ((size_t)((size_t)(kvh * a.tiles + tile) * (a.splits / a.cl) + split / a.cl) * RT + r) * (HD + PAD);
        *reinterpret_cast<float4 *>(part + d) = j.acc;
        if (d == 0) *reinterpret_cast<float2 *>(part + HD) = make_float2(j.M, j.L);
    };
    if (a.cl == 1) {
        for (int i = threadIdx.x; i < rows * (HD / 4); i += NW * 32) {
            const int r = i / (HD / 4), d = i % (HD / 4) * 4;
            Joined j;
            state(r, d, j.M, j.L, j.acc);
            finish(r, d, j);
        }
        return;
    }
    // a cluster: each CTA leaves its state in its shared memory and joins its share of the rows
    for (int i = threadIdx.x; i < rows * (HD / 4); i += NW * 32) {
        const int r = i / (HD / 4), d = i % (HD / 4) * 4;
        float M, L;
        float4 acc;
        state(r, d, M, L, acc);
        *reinterpret_cast<float4 *>(cs + r * (HD + PAD) + d) = acc;
        if (d == 0) *reinterpret_cast<float2 *>(cs + r * (HD + PAD) + HD) = make_float2(M, L);
    }
    cluster_sync();
    for (int i = split % a.cl * NW * 32 + threadIdx.x; i < rows * (HD / 4); i += a.cl * NW * 32) {
        const int r = i / (HD / 4), d = i % (HD / 4) * 4;
        Joined j;
        for (int s = 0; s < a.cl; ++s) {
            const uint32_t base = cluster_smem(cs + r * (HD + PAD), s);
            j.add(ld_cluster2(base + HD * 4), ld_cluster4(base + d * 4));
        }
        finish(r, d, j);
    }
    cluster_sync();   // no CTA leaves while its state may be read
}

// Joins the partial states of a row: `groups` x hd / 4 threads per query row and KV head, each group taking every
// groups-th state, then the groups through shared memory.  Bound by the launch and
// one round of loads: 3 of the 40 us of one token over 131,072 positions.
constexpr int JOIN_THREADS = 256;
__global__ void __launch_bounds__(JOIN_THREADS) attn_join(const __grid_constant__ Attn a, int groups)
{
    __shared__ float sh[JOIN_THREADS][6];
    const int hd = a.c.hd, lanes = hd / 4, per = JOIN_THREADS / (lanes * groups);   // rows per block
    const int row = blockIdx.x * per + threadIdx.x / (lanes * groups), kvh = blockIdx.y;
    const int grp = threadIdx.x / lanes % groups, d = threadIdx.x % lanes * 4;
    dependents_may_launch();
    wait_for_prerequisites();
    Joined j;
    int parts = 0;
    if (row < a.n * a.G) {
        // state s of the row's tile: number at(s) of all
        const size_t tile = (size_t)kvh * a.tiles + row / a.rt, step = (size_t)a.rt * (hd + PAD);
        const int2 pc = a.pieces ? ld(a.pieces + tile) : make_int2(0, a.splits / a.cl);
        parts = pc.y;
        const float *part = a.part + (size_t)(row % a.rt) * (hd + PAD);
#pragma unroll 4
        for (int s = grp; s < parts; s += groups) {
            // a CTA's second place holds the tile that it begins and leaves, its first the one it goes on with
            const size_t at = a.pieces ? 2 * (size_t)(pc.x + s) + (s == 0 ? 1 : 0) : tile * parts + s;
            j.add(ld(reinterpret_cast<const float2 *>(part + at * step + hd)),
                  ld(reinterpret_cast<const float4 *>(part + at * step + d)));
        }
    }
    if (groups > 1) {
        float *x = sh[threadIdx.x];
        x[0] = j.acc.x, x[1] = j.acc.y, x[2] = j.acc.z, x[3] = j.acc.w, x[4] = j.M, x[5] = j.L;
        __syncthreads();
        if (grp) return;
        for (int g = 1; g < groups; ++g) {
            const float *y = sh[threadIdx.x + g * lanes];
            j.add(make_float2(y[4], y[5]), make_float4(y[0], y[1], y[2], y[3]));
        }
    }
    if (parts) j.store(a, row, kvh, d);   // (a tile of one piece has its output)
}

// ---------------------------------------------------------------- launches

// Workspace of the tiles kernel: two states per CTA, and where each tile's are.
static size_t tiles_workspace(const Cache &c, size_t ctas, size_t tiles)
{
    return (2 * ctas * 128 * (c.hd + PAD)) * sizeof(float) + tiles * sizeof(int2);
}

// What a tile, or a piece of one, costs beside its chunks, in chunks (about 1,600 cycles each, 3,000 in FP32, beside
// 20,000 a piece, from the CTAs' own clocks): q, the way to the first P and from the last one, the output.
static int piece_cost(const Attn &a) { return a.q.dtype == F32 ? 7 : 12; }

int share_tiles(const Attn &a, int ctas, Shares &sh)
{
    const int all = a.tiles * a.c.Hkv, extra = piece_cost(a);
    int first;
    long long left = 0;   // the cost of what is not dealt out yet
    for (int t = 0; t < a.tiles; ++t) left += tile_chunks(a, t, first) + extra;
    left *= a.c.Hkv;
    Share at = {0, 0, 0};
    for (int c = 0; c < ctas; ++c) {
        sh.at[c] = at;
        // an even part of it, and the piece that the cut at its end makes
        const long long budget = (left + ctas - c - 1) / (ctas - c) + extra;
        long long spent = 0;
        while (at.tile < all) {
            const int have = tile_chunks(a, at.tile % a.tiles, first) - at.skip;
            const int room = (int)std::min<long long>(budget - spent - extra, have);
            if (have <= room + 1 || (spent == 0 && have <= 3) || c == ctas - 1) {   // the rest of the tile
                spent += have + extra;
                left -= have + extra;
                at = {at.tile + 1, 0, 0};
            } else if (room < 2 && spent > 0) {              // too little left to begin another tile
                break;
            } else {
                const int take = std::max(room, 2);          // have is more
                left -= take;
                at = {at.tile, at.skip + take, at.piece + 1};
                break;
            }
        }
        if (at.tile >= all) {
            sh.at[c + 1] = at;
            return c + 1;
        }
    }
    return ctas;   // not reached: the last CTA takes what is left
}

// The tiles kernel's time in microseconds, and its plan but for the shares.
static double plan_tiles(Attn &a, int sms, int rows)
{
    a.rt = 128;
    a.cl = 1;
    a.tiles = (rows + 127) / 128;
    sms = std::min(sms, MAX_CTAS);
    long long total = 0;
    int most = 1, first;
    for (int t = 0; t < a.tiles; ++t) {
        const int c = tile_chunks(a, t, first);
        total += c;
        most = std::max(most, c);
    }
    total *= a.c.Hkv;
    // One CTA per SM at a time.  Either every tile has a CTA of its own, the longest first (the last one to start ends
    // about half a tile after the others), or all SMs share the work evenly, cutting tiles (by whole pieces, hence a
    // tenth more), and a launch joins the pieces (about eight chunks' time, with the pieces written and read).
    const long long t = (long long)a.tiles * a.c.Hkv, ctas = std::min<long long>(sms, std::max<long long>(1, total / 2));
    const double extra = piece_cost(a), shared = 1.1 * (double)(total + (t + ctas) * extra) / (double)ctas + 8.0;
    const double each = t <= sms ? most + extra : (double)(total + t * extra) / (double)sms + (most + extra) / 2.0;
    const bool own = each <= shared && t < (1ll << 30);
    a.splits = own ? (int)t : 0;
    a.per = own ? 0 : (int)ctas;
    const double chunk = (a.q.dtype == F32 ? 1.6 : 0.8) * (a.c.hd == 128 ? 1.0 : 0.8);
    return chunk * (own ? each : shared);
}

// CTAs of the rows kernel that run at a time in clusters of cl: two per SM, one of 16 rows.  A cluster stays within a
// group of SMs, so that larger ones leave some empty: 304, 304, 291, 296, 290, 276, 266, 288 and 152, 152, 138, 144,
// 140, 138, 105, 120 of a GB300's 152 by the runtime's occupancy query.  Behind another kernel that still holds
// SMs the last of them may find no place (45 of 46 clusters of 6: 8 us more): one cluster of 4 or 8, a
// seventh of the other sizes is not counted on.
static int slots_of(int rt, int cl, int sms)
{
    static const int two[9] = {0, 304, 304, 249, 292, 245, 234, 224, 280}, one[9] = {0, 152, 152, 117, 140, 120, 114, 91, 112};
    const int n = (rt == 8 ? two : one)[cl] * sms / 152;
    return std::max(n, cl);
}

// The rows kernel's time in microseconds, its plan and workspace.  The range of a row tile, in eights of chunks (one
// chunk for each of a CTA's warps), is dealt out to one cluster, which does it all in one launch, or to as many clusters as
// run at a time, joined by a second launch (2.7 us on the GPU, and its launch by the host).  Either way the time is that
// of the rounds of CTAs, each a beginning and so many chunks a warp; the figures are measured ones for few CTAs (more
// chunks cost more under load, for every choice alike).  A chunk of one slab begins sooner, two slabs
// cost less each.  One token, 20/5 heads x 128, FP16: over 512 positions 4.8 us with clusters of four and one slab, 5.5
// with two and two, 5.7 with neither; over 4,096 7.1 in one launch, 8.4 in two; over 16,000 14.3 and 11.2.  32/8 heads
// over 131,072: two slabs 39.8, one 43.1.  192 rows at 1,024: clusters of five, which need three rounds, 23.8, of
// two 11.1.  One head at 131,072: clusters of eight 13, without 25.
static double plan_rows(Attn &a, int sms, int rows, size_t &bytes)
{
    a.rt = rows <= 8 ? 8 : 16;
    a.tiles = (rows + a.rt - 1) / a.rt;
    a.lo = key_lo(a.pos, 0, a.win);
    const int range = std::max(1, key_hi(a.pos, a.n - 1, a.len) - a.lo);
    const long long t = (long long)a.tiles * a.c.Hkv;
    const bool f32 = a.q.dtype == F32, wide = a.c.hd == 128, two = a.rt == 16;
    const double slab = (two ? (wide ? 0.83 : 0.62) : (wide ? 0.67 : 0.53)) * (f32 ? 1.22 : 1.0);
    const double first = (two ? (wide ? 5.7 : 4.45) : (wide ? 3.65 : 3.15)) + (f32 ? (two ? 0.6 : 0.2) : 0.0);
    double best = 1e30;
    for (int sl = 1; sl <= 2; ++sl) {
        const int eights = (range - 1) / (128 * sl) + 1;
        const double begin = first + (sl - 1) * 1.1 * slab, chunk = sl == 1 ? slab : 1.72 * slab;
        for (int c = std::min(8, eights); c >= 1; --c) {
            for (int many = 0; many < (eights > 8 ? 2 : 1); ++many) {
                int groups = many ? (int)(slots_of(a.rt, c, sms) / (t * c)) : 1, cl = c;
                if (many && groups < 2) continue;
                const int each = (eights - 1) / (groups * cl) + 1;
                if (!many) cl = (eights - 1) / each + 1;
                groups = (eights - 1) / (each * cl) + 1;
                const int slots = slots_of(a.rt, cl, sms);
                const long long rounds = (t * groups * cl + slots - 1) / slots;
                const double join = cl > 1 ? (two ? 1.0 + 0.12 * cl : 0.95 + 0.05 * cl) : 0.0;
                const double time = (double)rounds * (begin + join + chunk * (each - 1)) + (groups > 1 ? 3.5 + 0.035 * groups : 0.0);
                if (time < best) {
                    best = time;
                    a.sl = sl;
                    a.cl = cl;
                    a.splits = groups * cl;
                    a.per = each * 128 * sl;
                }
            }
        }
    }
    const int groups = a.splits / a.cl;
    bytes = groups > 1 ? (size_t)t * a.rt * groups * (a.c.hd + PAD) * sizeof(float) : 0;
    return best;
}

size_t max_workspace(const Cache &c, int Hq, int n, int sms)
{
    const size_t rows = (size_t)n * (Hq / c.Hkv);
    return std::max((size_t)2 * sms * 16 * (c.hd + PAD) * sizeof(float),
                    rows <= 8 ? (size_t)0 : tiles_workspace(c, (size_t)sms, (rows + 127) / 128 * c.Hkv));
}

void set_workspace(Attn &a, void *ws)
{
    a.part = static_cast<float *>(ws);
    a.pieces = ws && a.rt == 128 ? reinterpret_cast<int2 *>(a.part + (size_t)2 * a.splits * 128 * (a.c.hd + PAD)) : nullptr;
}

size_t plan_attn(Attn &a, int sms)
{
    a.gsh = -1;
    for (int s = 0; s < 30; ++s)
        if (a.G == 1 << s) a.gsh = s;
    const int rows = a.n * a.G;
    size_t bytes;
    const double by_rows = plan_rows(a, sms, rows, bytes);
    if (rows <= 8) return bytes;
    // More rows than one n-tile: the faster kernel by the models above.  (20/5 heads x 128, FP16, rows kernel against
    // tiles kernel: 64 rows at 1,024 8.4 and 16.5 us, at 4,096 11.7 and 15.9, at 16,384 39 and 19.9; 256 rows at 0
    // 5.6 and 9.4, at 1,024 12.3 and 16.9, at 4,096 44 and 20.5; 1,024 rows at 0 17.3 and 11.5.)
    Attn b = a;
    if (by_rows <= plan_tiles(b, sms, rows)) return bytes;
    a = b;
    if (a.per == 0) return 0;
    Shares sh;
    a.splits = share_tiles(a, a.per, sh);
    return tiles_workspace(a.c, (size_t)a.splits, (size_t)a.tiles * a.c.Hkv);
}

template <template <class> class F, class... A>
static cudaError_t by_dtype(int dtype, A... args)
{
    switch (dtype) {
    case F16: return F<__half>::run(args...);
    case BF16: return F<__nv_bfloat16>::run(args...);
    default: return F<float>::run(args...);
    }
}

// Grid of 2^shift places for each of n rows, `per` a block, by KV head and K or V.
static dim3 row_grid(const Cache &c, int n, int shift, int per)
{
    return dim3((unsigned)((((long long)n << shift) + per - 1) / per), (unsigned)(2 * c.Hkv));
}
template <class T>
struct RunAppend {
    static cudaError_t run(Cache c, Rows k, Rows v, int n, int pos, cudaStream_t s)
    {
        const int shift = c.hd == 128 ? 3 : 2;            // blocks of 16
        return launch(append_rows<T>, row_grid(c, n, shift, 256), 256, 0, 1, s, c, k, v, n, pos, shift);
    }
};
template <class T>
struct RunRead {
    static cudaError_t run(Cache c, Rows k, Rows v, int n, int pos, cudaStream_t s)
    {
        const int shift = (c.hd == 128 ? 4 : 3) + (sizeof(T) == 4 ? 1 : 0);
        return launch(read_rows<T>, row_grid(c, n, shift, 256 * READ_U), 256, 0, 1, s, c, k, v, n, pos, shift);
    }
};
cudaError_t launch_append(const Cache &c, const Rows &k, const Rows &v, int n, int pos, cudaStream_t s)
{
    if (k.dtype == TAG32) return RunAppend<Tagged>::run(c, k, v, n, pos, s);
    if (k.dtype == SWZ16) return RunAppend<Swizzled>::run(c, k, v, n, pos, s);
    return by_dtype<RunAppend>(k.dtype, c, k, v, n, pos, s);
}
cudaError_t launch_read(const Cache &c, const Rows &k, const Rows &v, int n, int pos, cudaStream_t s)
{
    return by_dtype<RunRead>(k.dtype, c, k, v, n, pos, s);
}

template <int HD, int NT, bool SPLIT, int SL>
static cudaError_t run_rows(const Attn &a, cudaStream_t s)
{
    constexpr int smem = RowCfg<HD, NT, SPLIT>::SMEM;
    static bool ready[64] = {};   // the attribute is per device; setting it again is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev]) {
        e = cudaFuncSetAttribute(attn_rows<HD, NT, SPLIT, SL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev] = true;
    }
    return launch(attn_rows<HD, NT, SPLIT, SL>, dim3((unsigned)(a.tiles * a.splits), (unsigned)a.c.Hkv), 256, smem,
                  a.cl, s, a);
}

template <int HD, int NT>
static cudaError_t run_rows(const Attn &a, cudaStream_t s)
{
    if (a.q.dtype == F32) return a.sl == 1 ? run_rows<HD, NT, true, 1>(a, s) : run_rows<HD, NT, true, 2>(a, s);
    return a.sl == 1 ? run_rows<HD, NT, false, 1>(a, s) : run_rows<HD, NT, false, 2>(a, s);
}

cudaError_t launch_attn(const Attn &a, cudaStream_t s)
{
    cudaError_t e;
    if (a.rt > 16)
        e = launch_attn_tiles(a, s);
    else if (a.c.hd == 128)
        e = a.rt == 8 ? run_rows<128, 1>(a, s) : run_rows<128, 2>(a, s);
    else
        e = a.rt == 8 ? run_rows<64, 1>(a, s) : run_rows<64, 2>(a, s);
    if (e == cudaSuccess && a.part) {
        // few rows: the splits of a row are spread over a whole block; many: one group each, the traffic counts
        const int lanes = a.c.hd / 4, rows = a.n * a.G;
        const int groups = (long long)rows * a.c.Hkv >= 4096 ? 1 : JOIN_THREADS / lanes;
        const int per = JOIN_THREADS / (lanes * groups);
        e = launch(attn_join, dim3((unsigned)((rows + per - 1) / per), (unsigned)a.c.Hkv), JOIN_THREADS, 0, 1, s, a, groups);
    }
    return e;
}

}  // namespace lfq

// ---------------------------------------------------------------- C entry points

namespace {

using namespace lfq;
using lfr::aligned16;
using lfr::check_rows;
using lfr::sm_count;
using lfr::status_of;

constexpr int kMaxKvHeads = 1024;
constexpr int kMaxPositions = 1 << 30;   // positions rounded up to whole splits stay in 32 bits
constexpr long long kMaxRows = 1ll << 32;   // rows of all heads (8 GB per dim in FP16): their tiles do too

lf_status check_cache(const lf_kv4 *c)
{
    if (!c || c->n_kv_heads < 1 || c->max_seq < 1) return LF_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return LF_ERR_NOT_SUPPORTED;
    if (c->n_kv_heads > kMaxKvHeads || c->max_seq > kMaxPositions) return LF_ERR_NOT_SUPPORTED;
    if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
        return LF_ERR_INVALID_ARG;
    return LF_OK;
}

Cache cache_of(const lf_kv4 *c)
{
    return {static_cast<uint8_t *>(c->k_codes), static_cast<uint8_t *>(c->k_scales), static_cast<uint8_t *>(c->v_codes),
            static_cast<uint8_t *>(c->v_scales), c->n_kv_heads, c->head_dim, c->max_seq};
}
Rows rows_of(const lf_rows *r) { return {r->data, r->dtype, r->token_stride, r->head_stride, 0, nullptr}; }

lf_status check_copy(const lf_kv4 *c, const lf_rows *k, const lf_rows *v, int n, int pos, bool written)
{
    lf_status st = check_cache(c);
    if (st != LF_OK) return st;
    if (n < 0 || pos < 0) return LF_ERR_INVALID_ARG;
    if ((long long)pos + n > c->max_seq) return LF_ERR_CAPACITY;
    if (n == 0) return LF_OK;
    st = check_rows(k, n, c->n_kv_heads, c->head_dim, written);
    if (st == LF_OK) st = check_rows(v, n, c->n_kv_heads, c->head_dim, written);
    if (st == LF_OK && (k->dtype != v->dtype || (written && k->data == v->data))) st = LF_ERR_INVALID_ARG;
    return st;
}

lf_status make_attn(const lf_kv4 *c, const lf_kv4_query *q, Attn *a, size_t *bytes)
{
    lf_status st = check_cache(c);
    if (st != LF_OK) return st;
    if (!q || q->n < 0 || q->n_heads < 1 || q->pos < 0 || q->length < 0 || q->window < 0 || !std::isfinite(q->scale))
        return LF_ERR_INVALID_ARG;
    if (q->length > c->max_seq) return LF_ERR_CAPACITY;
    if (q->n_heads % c->n_kv_heads) return LF_ERR_NOT_SUPPORTED;
    const int G = q->n_heads / c->n_kv_heads;
    if ((long long)q->n * G > (1ll << 28) || (long long)q->n * q->n_heads > kMaxRows || (long long)q->pos + q->n > kMaxPositions)
        return LF_ERR_NOT_SUPPORTED;
    a->c = cache_of(c);
    a->Hq = q->n_heads;
    a->G = G;
    a->n = q->n;
    a->pos = q->pos;
    a->len = q->length;
    a->win = q->window;
    if (q->q.dtype != LF_F16 && q->q.dtype != LF_BF16 && q->q.dtype != LF_F32) return LF_ERR_NOT_SUPPORTED;
    a->q = rows_of(&q->q);
    a->scale = q->scale != 0.f ? q->scale : 1.0f / std::sqrt((float)c->head_dim);
    a->wait_ns = WAIT_NS;
    set_workspace(*a, nullptr);
    *bytes = 0;
    if (q->n == 0) return LF_OK;
    int sms = 0;
    st = sm_count(&sms);
    if (st == LF_OK) *bytes = plan_attn(*a, sms);
    return st;
}

}  // namespace

extern "C" {

lf_status lf_kv4_append(const lf_kv4 *c, const lf_rows *k, const lf_rows *v, int32_t n, int32_t pos, void *stream)
{
    const lf_status st = check_copy(c, k, v, n, pos, false);
    if (st != LF_OK || n == 0) return st;
    return status_of(launch_append(cache_of(c), rows_of(k), rows_of(v), n, pos, static_cast<cudaStream_t>(stream)));
}

lf_status lf_kv4_read(const lf_kv4 *c, const lf_rows *k, const lf_rows *v, int32_t n, int32_t pos, void *stream)
{
    const lf_status st = check_copy(c, k, v, n, pos, true);
    if (st != LF_OK || n == 0) return st;
    return status_of(launch_read(cache_of(c), rows_of(k), rows_of(v), n, pos, static_cast<cudaStream_t>(stream)));
}

lf_status lf_kv4_workspace(const lf_kv4 *c, const lf_kv4_query *q, int64_t *bytes)
{
    if (!bytes) return LF_ERR_INVALID_ARG;
    Attn a = {};
    size_t need = 0;
    const lf_status st = make_attn(c, q, &a, &need);
    if (st == LF_OK) *bytes = (int64_t)need;
    return st;
}

lf_status lf_kv4_attend(const lf_kv4 *c, const lf_kv4_query *q, void *workspace, int64_t workspace_bytes, void *stream)
{
    Attn a = {};
    size_t need = 0;
    lf_status st = make_attn(c, q, &a, &need);
    if (st != LF_OK || a.n == 0) return st;
    st = check_rows(&q->q, a.n, a.Hq, c->head_dim, false);
    if (st == LF_OK) st = check_rows(&q->out, a.n, a.Hq, c->head_dim, true);
    if (st != LF_OK) return st;
    if (q->q.dtype != q->out.dtype || q->q.data == q->out.data) return LF_ERR_INVALID_ARG;
    if (need && (!aligned16(workspace) || workspace_bytes < (int64_t)need)) return LF_ERR_INVALID_ARG;
    a.o = rows_of(&q->out);
    set_workspace(a, need ? workspace : nullptr);
    return status_of(launch_attn(a, static_cast<cudaStream_t>(stream)));
}

lf_status lf_kv4_status(void *stream)
{
    // a synchronisation would end the capture with an error
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cs);
    if (e == cudaSuccess && cs != cudaStreamCaptureStatusNone) return LF_ERR_NOT_SUPPORTED;
    bool expired = false;
    if (e == cudaSuccess) e = tiles_status(expired, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return status_of(e);
    return expired ? LF_ERR_TIMEOUT : LF_OK;
}

}  // extern "C"
