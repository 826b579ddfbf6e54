// lf_kv4_tc.cu -- attention of many query rows over the 4-bit KV cache, on the
// sm_103a tensor cores.
//
// One CTA takes TILES x 128 query rows that share a KV head (row r = token
// r / G, head r % G of the group) and walks its positions in chunks of 128:
//
//   dequantise  four warps, one thread per position: the row's codes and scales
//               (prefetched one chunk ahead into registers) -> FP16, written to
//               shared memory in the 128-byte-swizzle layout, K as a K-major
//               operand, V (the same row layout) as an MN-major one.  Once per
//               chunk for all rows of the CTA.
//   S = Q K^T   tcgen05.mma, FP32 scores in TMEM
//   P           one thread per query row: mask, running maximum and sum, 2^x,
//               FP16 back into the TMEM columns of S
//   O += P V    tcgen05.mma with P as the TMEM operand, FP32 in TMEM
//
// P stays in TMEM because shared memory is the other limit: a 128 x 128 x 16
// product that reads both operands there takes its whole 128 bytes per cycle.
//
// Work items: (chunk, tile) with TILES = 2 (FP16 and BF16 queries), where the
// softmax of one tile runs while the other tile's products do; (chunk) with
// TILES = 1 for FP32 queries, whose q and P are split into an FP16 head and
// remainder (SPLIT: twice the products, and no room for a second tile's
// operands).  Item w uses score buffer w % 2 either way, and the MMA order is
//   S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...
// where S(w + 2) overwrites the P that PV(w) reads, so it waits for it.
//
// The reference that P is relative to moves only when a row's maximum rises
// more than SLACK above it (O and l are then rescaled); the quotient O / l does
// not depend on it.
//
// Every wait is bounded by %globaltimer; on expiry the CTA records a timeout
// in the status word, settles its MMAs, frees TMEM and returns.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lf_internal.cuh"
#include "lf_kv4.cuh"
#include "lf_kv4.h"
#include "lf_ptx.cuh"
#include "lf_tc.cuh"

namespace lfq {

using namespace lftc;

__device__ unsigned g_status[8];   // error record of the kernels below (status[4]: unused abort word)

constexpr int BM = 128, BN = 128;
constexpr float SLACK = 4.f, TC_EXP = 11.f;      // P lies within 2^(TC_EXP + SLACK) = 2^15
constexpr long long kWaitNs = 2000000000LL;      // bound of every wait

template <int HD, bool SPLIT>
struct TcCfg {
    static constexpr int TILES = SPLIT ? 1 : 2;
    static constexpr int NSM = 128 * TILES;                 // softmax threads: one per query row
    static constexpr int W_DQ = NSM / 32, W_MMA = W_DQ + 4; // warps: softmax, dequantisation (4), MMA
    static constexpr int NTHR = NSM + 128 + 32;
    static constexpr uint32_t ATOM = 128 * 128;             // 128 rows x 64 FP16
    static constexpr uint32_t ROWB = (HD / 64) * ATOM;      // a 128-row operand
    static constexpr uint32_t OFF_Q = 0;                    // [TILES][head, remainder if SPLIT]
    static constexpr uint32_t OFF_K = 2 * ROWB, OFF_V = OFF_K + 2 * ROWB, OFF_BAR = OFF_V + 2 * ROWB;
    // score buffers, then the tiles' outputs
    static constexpr uint32_t T_O = 2 * BN, T_COLS = 512;
};

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], pv_done[2], q_ready, drained;
    uint32_t tmem;
    int abort;
};
template <int HD, bool SPLIT>
constexpr uint32_t tc_smem() { return TcCfg<HD, SPLIT>::OFF_BAR + (uint32_t)sizeof(Bars) + 1024u; }

__device__ bool wait_phase(uint64_t *bar, unsigned parity, Bars *b, unsigned where)
{
    if (lfk::mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = lfk::globaltimer_ns();
    for (unsigned it = 0;; ++it) {
        if (lfk::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 63u) {
            if (*reinterpret_cast<volatile int *>(&b->abort)) return false;
            if ((long long)(lfk::globaltimer_ns() - t0) > kWaitNs) {
                *reinterpret_cast<volatile int *>(&b->abort) = 1;
                if (atomicCAS(g_status, 0u, (unsigned)lfk::STATUS_TIMEOUT) == 0u) {
                    g_status[1] = where;
                    g_status[2] = blockIdx.x;
                    g_status[3] = blockIdx.y;
                }
                return false;
            }
        }
    }
}
__device__ void settle_phase(uint64_t *bar, unsigned parity)
{
    const unsigned long long t0 = lfk::globaltimer_ns();
    while (!lfk::mbar_try_wait(bar, parity))
        if ((long long)(lfk::globaltimer_ns() - t0) > kWaitNs) return;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ uint32_t sw128(int row, int c16) { return (uint32_t)(row * 128 + ((c16 ^ (row & 7)) << 4)); }

// MN-major 128-byte-swizzle descriptor: 64-element atoms along MN `lbo` bytes
// apart, 8-row groups along K 1,024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lbo)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
// kind::f16, FP16 operands, FP32 accumulators; B MN-major when b_mn.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn)
{
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] . B[smem]
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(bdesc), "r"(id), "r"(accum)
        : "memory");
}

// One position's row: HD / 2 code bytes and HD / 16 scales, held in registers.
template <int HD>
struct RawRow {
    uint4 c[HD / 32];
    uint2 s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales)
    {
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) c[j] = __ldg(reinterpret_cast<const uint4 *>(codes) + j);
        if (HD == 128) s = __ldg(reinterpret_cast<const uint2 *>(scales));
        else s = make_uint2(__ldg(reinterpret_cast<const unsigned *>(scales)), 0u);
    }
    // row `row` of an operand tile at `base`
    __device__ __forceinline__ void store(uint8_t *base, int row) const
    {
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {
            const unsigned w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {          // 8 values: 16 bytes of FP16
                const int blk = 2 * j + u / 2;     // their block of 16
                const unsigned sc = e4m3_h2_same(((blk < 4 ? s.x : s.y) >> (8 * (blk & 3))) & 255u);
                unsigned h[4];
                e2m1x8_h2(w[u], h[0], h[1], h[2], h[3]);
                const int c16 = 4 * j + u;
                *reinterpret_cast<uint4 *>(base + (c16 / 8) * (128 * 128) + sw128(row, c16 % 8)) =
                    make_uint4(hmul2(h[0], sc), hmul2(h[1], sc), hmul2(h[2], sc), hmul2(h[3], sc));
            }
        }
    }
};

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

// The largest of a row's BN scores at TMEM columns ts .. (WHOLE: of all; else of columns lo .. hi - 1).
template <bool WHOLE>
__device__ __forceinline__ float row_max(uint32_t ts, int lo, int hi)
{
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < BN / 64; ++c) {
        uint32_t u[2][32];
        tmem_ld32(ts + (uint32_t)(64 * c), u[0]);
        tmem_ld32(ts + (uint32_t)(64 * c + 32), u[1]);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 64; ++e) {
            const float x = __uint_as_float(u[e / 32][e % 32]);
            const int k = 64 * c + e;
            if (WHOLE) m[e & 3] = fmaxf(m[e & 3], x);
            else m[e & 3] = k >= lo && k < hi ? fmaxf(m[e & 3], x) : m[e & 3];
        }
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 2^(f s + neg) of a row's BN scores s at TMEM columns ts .., as FP16 pairs over the first 64 of those
// columns (SPLIT: the remainders over the other 64); zeros outside lo .. hi - 1 unless WHOLE.  Returns their
// sum, of the FP32 values.
template <bool WHOLE, bool SPLIT>
__device__ __forceinline__ float row_probs(uint32_t ts, float f, float neg, int lo, int hi)
{
    const uint64_t ff = pack2(f, f), nn = pack2(neg, neg);
    uint64_t sum[2] = {0ull, 0ull};
    auto take = [&](const uint32_t (&u)[32], int k0, uint32_t *hw, uint32_t *lw) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float2 y = unpack2(fma2(pack2u(u[e], u[e + 1]), ff, nn));
            float x0 = ex2(y.x), x1 = ex2(y.y);
            if (!WHOLE) {
                if (!(k0 + e >= lo && k0 + e < hi)) x0 = 0.f;
                if (!(k0 + e + 1 >= lo && k0 + e + 1 < hi)) x1 = 0.f;
            }
            sum[e / 2 & 1] = add2(sum[e / 2 & 1], pack2(x0, x1));
            const __half2 h = __floats2half2_rn(x0, x1);
            hw[e / 2] = *reinterpret_cast<const unsigned *>(&h);
            if (SPLIT) {
                const float2 b = __half22float2(h);
                const __half2 r = __floats2half2_rn(x0 - b.x, x1 - b.y);
                lw[e / 2] = *reinterpret_cast<const unsigned *>(&r);
            }
        }
    };
    uint32_t u[2][32], v[2][32], hw[32], lw[32];
    tmem_ld32(ts, u[0]);
    tmem_ld32(ts + 32u, u[1]);
    if (SPLIT) {   // the remainders land on the second half's scores
        tmem_ld32(ts + 64u, v[0]);
        tmem_ld32(ts + 96u, v[1]);
    }
    tmem_ld_wait();
    take(u[0], 0, hw, lw);
    take(u[1], 32, hw + 16, lw + 16);
    if (!SPLIT) {
        tmem_ld32(ts + 64u, v[0]);
        tmem_ld32(ts + 96u, v[1]);
    }
    tmem_st32(ts, hw);
    if (SPLIT) tmem_st32(ts + 64u, lw);
    if (!SPLIT) tmem_ld_wait();
    take(v[0], 64, hw, lw);
    take(v[1], 96, hw + 16, lw + 16);
    tmem_st32(ts + 32u, hw);
    if (SPLIT) tmem_st32(ts + 96u, lw);
    const float2 t = unpack2(add2(sum[0], sum[1]));
    return t.x + t.y;
}

template <int HD, bool SPLIT>
__global__ void __launch_bounds__(TcCfg<HD, SPLIT>::NTHR, 1) attn_tiles(const __grid_constant__ Attn a)
{
    using C = TcCfg<HD, SPLIT>;
    constexpr int TILES = C::TILES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~uintptr_t(1023));
    Bars *b = reinterpret_cast<Bars *>(smem + C::OFF_BAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % a.splits, tile = a.tiles - 1 - blockIdx.x / a.splits;   // the longest rows first
    const int kvh = blockIdx.y;
    const int r0 = tile * a.rt, rows = min(a.rt, a.n * a.G - r0);
    const int t_first = r0 / a.G, t_last = (r0 + rows - 1) / a.G;
    // positions of this CTA: the split's, cut to what the tile's rows see
    const int lo_t = key_lo(a.pos, t_first, a.win), hi_r = key_hi(a.pos, t_last, a.len);
    const int hi_t = hi_r > lo_t ? hi_r : 0;              // no position at all: an empty range
    const int p0 = max(a.lo + split * a.per, lo_t / BN * BN), p1 = min(a.lo + (split + 1) * a.per, hi_t);
    const int nc = p1 > p0 ? (p1 - p0 + BN - 1) / BN : 0;
    const int ntile = rows > BM ? TILES : 1;              // tiles that hold rows
    const int W = nc * ntile;                             // work items

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            lfk::mbar_init(&b->k_full[i], 128);
            lfk::mbar_init(&b->k_empty[i], 1);
            lfk::mbar_init(&b->v_full[i], 128);
            lfk::mbar_init(&b->v_empty[i], 1);
            lfk::mbar_init(&b->s_full[i], 1);
            lfk::mbar_init(&b->p_full[i], 128);
            lfk::mbar_init(&b->pv_done[i], 1);
        }
        lfk::mbar_init(&b->q_ready, C::NSM);
        lfk::mbar_init(&b->drained, 1);
        b->abort = 0;
        lfk::mbar_fence_init();
    }
    if (warp == C::W_MMA) {
        tmem_alloc(&b->tmem, C::T_COLS);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = b->tmem;

    if (warp == C::W_MMA) {
        if (lane == 0 && W > 0) {
            const uint32_t sb = lfk::smem_u32(smem);
            auto chunk_of = [&](int w) { return ntile == 2 ? w >> 1 : w; };
            auto tile_of = [&](int w) { return ntile == 2 ? w & 1 : 0; };
            auto issue_s = [&](int w) -> bool {
                const int i = chunk_of(w), tl = tile_of(w);
                if (!wait_phase(&b->k_full[i & 1], (unsigned)(i >> 1) & 1u, b, 701)) return false;
                fence_after_sync();
                const uint32_t qb = sb + C::OFF_Q + (SPLIT ? 0u : (uint32_t)tl * C::ROWB);
                const uint32_t kb = sb + C::OFF_K + (uint32_t)(i & 1) * C::ROWB;
                const uint32_t d = tmem + (uint32_t)(w & 1) * BN;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = (uint32_t)(kk / 4) * C::ATOM + (uint32_t)(kk % 4) * 32u;
                    const uint64_t bd = sdesc_kmajor_sw128(kb + off);
                    mma_f16(d, sdesc_kmajor_sw128(qb + off), bd, idesc(BM, BN, false), kk != 0);
                    if (SPLIT) mma_f16(d, sdesc_kmajor_sw128(qb + C::ROWB + off), bd, idesc(BM, BN, false), 1u);
                }
                commit(&b->s_full[w & 1]);
                if (tl == ntile - 1) commit(&b->k_empty[i & 1]);
                return true;
            };
            bool ok = wait_phase(&b->q_ready, 0u, b, 700) && issue_s(0) && (W < 2 || issue_s(1));
            for (int w = 0; ok && w < W; ++w) {
                const int i = chunk_of(w), tl = tile_of(w);
                const unsigned ph = (unsigned)(w >> 1) & 1u;
                if (!wait_phase(&b->v_full[i & 1], (unsigned)(i >> 1) & 1u, b, 702)) break;
                if (!wait_phase(&b->p_full[w & 1], ph, b, 703)) break;
                fence_after_sync();
                const uint32_t vb = sb + C::OFF_V + (uint32_t)(i & 1) * C::ROWB;
                const uint32_t pa = tmem + (uint32_t)(w & 1) * BN, d = tmem + C::T_O + (uint32_t)tl * HD;
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    const uint64_t vd = sdesc_mn_sw128(vb + (uint32_t)kk * 2048u, C::ATOM);
                    mma_f16_ta(d, pa + (uint32_t)kk * 8u, vd, idesc(BM, HD, true), (i | kk) != 0);
                    if (SPLIT) mma_f16_ta(d, pa + BN / 2 + (uint32_t)kk * 8u, vd, idesc(BM, HD, true), 1u);
                }
                if (tl == ntile - 1) commit(&b->v_empty[i & 1]);
                commit(&b->pv_done[w & 1]);
                if (w + 2 < W) {
                    // S(w + 2) lands on the P that PV(w) reads
                    if (!wait_phase(&b->pv_done[w & 1], ph, b, 704)) break;
                    ok = issue_s(w + 2);
                }
            }
        }
    } else if (warp >= C::W_DQ) {
        // ---- dequantisation: thread j takes position j of every chunk
        const int j = threadIdx.x - C::W_DQ * 32;
        const size_t row0 = (size_t)kvh * a.c.cap;
        RawRow<HD> k, v;
        auto fetch = [&](int i) {
            const size_t r = row0 + (size_t)max(min(p0 + i * BN + j, p1 - 1), lo_t);   // outside: a seen row, masked
            k.load(a.c.kc + r * code_bytes(HD), a.c.ks + r * scale_bytes(HD));
            v.load(a.c.vc + r * code_bytes(HD), a.c.vs + r * scale_bytes(HD));
        };
        if (nc > 0) fetch(0);
        for (int i = 0; i < nc; ++i) {
            const int s = i & 1;
            const unsigned ph = ((unsigned)(i >> 1) & 1u) ^ 1u;
            if (!wait_phase(&b->k_empty[s], ph, b, 705)) break;
            k.store(smem + C::OFF_K + (uint32_t)s * C::ROWB, j);
            fence_async_smem();
            lfk::mbar_arrive(&b->k_full[s]);
            if (!wait_phase(&b->v_empty[s], ph, b, 706)) break;
            v.store(smem + C::OFF_V + (uint32_t)s * C::ROWB, j);
            fence_async_smem();
            lfk::mbar_arrive(&b->v_full[s]);
            if (i + 1 < nc) fetch(i + 1);
        }
    } else {
        // ---- softmax and output: one thread per query row
        const int mt = warp >> 2, r = (warp & 3) * 32 + lane;
        const int row = mt * BM + r;                        // of the CTA's rows
        const bool live = row < rows;
        const int tok = (r0 + min(row, rows - 1)) / a.G, head = kvh * a.G + (r0 + min(row, rows - 1)) % a.G;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // score factor: |scale| x log2(e) / the row's power of two; a negative scale turns q
        float f = fabsf(a.scale) * 1.4426950408889634f;
        {
            const size_t at = (size_t)tok * a.q.ts + (size_t)head * a.q.hs;
            auto load = [&](int c, float (&x)[16]) {
                if (a.q.dtype == F16) load16<__half>(static_cast<const __half *>(a.q.p) + at + c * 16, x);
                else if (a.q.dtype == BF16) load16<__nv_bfloat16>(static_cast<const __nv_bfloat16 *>(a.q.p) + at + c * 16, x);
                else load16<float>(static_cast<const float *>(a.q.p) + at + c * 16, x);
            };
            float fac = 1.f;
            if (a.q.dtype != F16) {
                float m = 0.f;
#pragma unroll 1
                for (int c = 0; c < HD / 16; ++c) {
                    float x[16];
                    load(c, x);
#pragma unroll
                    for (int u = 0; u < 16; ++u) m = fmaxf(m, fabsf(x[u]));
                }
                fac = range_factor(m);
                f /= fac;
            }
            if (a.scale < 0.f) fac = -fac;
            uint8_t *qh = smem + C::OFF_Q + (SPLIT ? 0u : (uint32_t)mt * C::ROWB);
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
                float x[16];
                load(c, x);
                unsigned hw[8], lw[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    __half h0, m0, h1, m1;
                    lfk::split_h(live ? x[2 * u] * fac : 0.f, h0, m0);
                    lfk::split_h(live ? x[2 * u + 1] * fac : 0.f, h1, m1);
                    hw[u] = lfk::pack_h2(h0, h1);
                    lw[u] = lfk::pack_h2(m0, m1);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c16 = 2 * c + u;
                    const uint32_t o = (uint32_t)(c16 / 8) * C::ATOM + sw128(r, c16 % 8);
                    *reinterpret_cast<uint4 *>(qh + o) = make_uint4(hw[4 * u], hw[4 * u + 1], hw[4 * u + 2], hw[4 * u + 3]);
                    if (SPLIT)
                        *reinterpret_cast<uint4 *>(qh + C::ROWB + o) =
                            make_uint4(lw[4 * u], lw[4 * u + 1], lw[4 * u + 2], lw[4 * u + 3]);
                }
            }
        }
        fence_async_smem();
        lfk::mbar_arrive(&b->q_ready);
        const int klo = key_lo(a.pos, tok, a.win), khi = min(key_hi(a.pos, tok, a.len), p1);
        float ref = -INFINITY, l = 0.f;
        bool run = true;
        const int mine = mt < ntile ? nc : 0;
        for (int i = 0; i < mine && run; ++i) {
            const int w = ntile == 2 ? 2 * i + mt : i, s = w & 1;
            const unsigned ph = (unsigned)(w >> 1) & 1u;
            run = __all_sync(0xffffffffu, wait_phase(&b->s_full[s], ph, b, 707));
            if (!run) break;
            fence_after_sync();
            const uint32_t ts = tl + (uint32_t)s * BN;
            const int key0 = p0 + i * BN;
            const bool whole = __all_sync(0xffffffffu, key0 >= klo && key0 + BN <= khi);
            // ---- the chunk's maximum
            const float top = whole ? row_max<true>(ts, 0, BN) : row_max<false>(ts, klo - key0, khi - key0);
            float mx = fmaf(top, f, -TC_EXP);                // -inf stays
            if (f == 0.f) mx = top == -INFINITY ? top : -TC_EXP;
            const bool up = mx > ref + SLACK;                // also from -inf
            if (__any_sync(0xffffffffu, up)) {
                const float alpha = up ? ex2(ref - mx) : 1.f;   // 0 from -inf
                if (up) {
                    l *= alpha;
                    ref = mx;
                }
                if (i > 0) {
                    // O must hold every earlier product of this tile
                    if (ntile == 1) {
                        run = __all_sync(0xffffffffu, wait_phase(&b->pv_done[s ^ 1], (unsigned)((w - 1) >> 1) & 1u, b, 708));
                        if (!run) break;
                        fence_after_sync();
                    }
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        const uint32_t oc = tl + C::T_O + (uint32_t)(mt * HD + 32 * c);
                        uint32_t o[32];
                        tmem_ld32(oc, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(oc, o);
                    }
                    tmem_st_wait();
                }
            }
            // ---- P, over S
            const float neg = ref == -INFINITY ? 0.f : -ref;
            l += whole ? row_probs<true, SPLIT>(ts, f, neg, 0, BN) : row_probs<false, SPLIT>(ts, f, neg, klo - key0, khi - key0);
            tmem_st_wait();
            fence_before_sync();
            lfk::mbar_arrive(&b->p_full[s]);
        }
        // ---- output: O / l, or the partial state of a split
        if (run && mine > 0) {
            const int w = ntile == 2 ? 2 * (nc - 1) + mt : nc - 1;
            run = __all_sync(0xffffffffu, wait_phase(&b->pv_done[w & 1], (unsigned)(w >> 1) & 1u, b, 709));
            fence_after_sync();
        }
        if (run) {
            float *part = a.part ? a.part + ((size_t)((size_t)(kvh * a.tiles + tile) * a.splits + split) * a.rt + row) * (HD + PAD)
                                 : nullptr;
            const float inv = part ? 1.f : (l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l));   // a row that saw nothing is 0
            const size_t at = (size_t)tok * a.o.ts + (size_t)head * a.o.hs;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t o[32];
                if (mine > 0) {
                    tmem_ld32(tl + C::T_O + (uint32_t)(mt * HD + 32 * c), o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float x = __uint_as_float(o[e]) * inv, y = __uint_as_float(o[e + 1]) * inv,
                                    z = __uint_as_float(o[e + 2]) * inv, v = __uint_as_float(o[e + 3]) * inv;
                        if (part) *reinterpret_cast<float4 *>(part + 32 * c + e) = make_float4(x, y, z, v);
                        else store4(a.o, at + 32 * c + e, x, y, z, v);
                    }
                }
                __syncwarp();
            }
            if (part && live) *reinterpret_cast<float2 *>(part + HD) = make_float2(ref, l);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == C::W_MMA) {
        if (lane == 0 && b->abort && W > 0) {
            // nothing may still write TMEM: one more commit covers every MMA issued
            commit(&b->drained);
            settle_phase(&b->drained, 0u);
        }
        __syncwarp();
        fence_after_sync();
        tmem_dealloc(tmem, C::T_COLS);
    }
}

template <int HD, bool SPLIT>
static cudaError_t run_tiles(const Attn &a, cudaStream_t s)
{
    constexpr int smem = (int)tc_smem<HD, SPLIT>();
    static_assert(smem <= 232448, "shared memory of the tiles kernel");
    static bool ready[64] = {};   // the attribute is per device; setting it again is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev]) {
        e = cudaFuncSetAttribute(attn_tiles<HD, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev] = true;
    }
    attn_tiles<HD, SPLIT>
        <<<dim3((unsigned)(a.tiles * a.splits), (unsigned)a.c.Hkv), TcCfg<HD, SPLIT>::NTHR, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attn_tiles(const Attn &a, cudaStream_t s)
{
    const bool split = a.q.dtype == F32;
    if (a.c.hd == 128) return split ? run_tiles<128, true>(a, s) : run_tiles<128, false>(a, s);
    return split ? run_tiles<64, true>(a, s) : run_tiles<64, false>(a, s);
}

cudaError_t tiles_status(unsigned out[4], cudaStream_t s)
{
    void *p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_status);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemcpy(out, p, 4 * sizeof(unsigned), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && out[0]) e = cudaMemset(p, 0, 8 * sizeof(unsigned));
    return e;
}

}  // namespace lfq
