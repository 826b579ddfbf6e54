// lf_kv4_tc.cu -- attention of many query rows over the 4-bit KV cache, on the
// sm_103a tensor cores.
//
// One CTA takes 128 query rows that share a KV head (row r = token r / G, head
// r % G of the group) and walks its positions in chunks of 128:
//
//   dequantise  four warps for K and four for V, one thread per position: the
//               row's codes and scales (prefetched one chunk ahead into
//               registers) -> FP16, written to shared memory in the
//               128-byte-swizzle layout, K as a K-major operand, V (the same row
//               layout) as an MN-major one
//   S = Q K^T   tcgen05.mma, Q from TMEM, FP32 scores in TMEM (two buffers)
//   P           two groups of four warps take the chunks in turn, one thread per
//               query row: mask, maximum, 2^x, running sum, FP16 into TMEM
//   O += P V    tcgen05.mma, P from TMEM, FP32 in TMEM
//
// Shared memory's 128 bytes per cycle are the second limit after the tensor
// cores: a 128 x 128 x 16 product that reads both operands there takes all of
// them.  With Q and P in TMEM a chunk moves 128 KB (K and V written once and read
// once) in the 1,024 cycles of its products at peak rate.  P lies beside
// S, not over it: S(i + 2) needs only that the scores of chunk i were read, so
// that the tensor cores find the next product queued.
//
// A chunk's softmax takes longer than its two products, so two chunks are in
// flight, and no maximum is taken on the common path.  P is formed relative to the
// row's reference as last known; 128 values whose sum is at most 2^15 cannot have
// left FP16's range, so the sum, which is needed anyway, is the check.  At the end
// of a chunk the groups hand the reference on in chunk order; only where it has
// moved, the sum was too large, or the row saw its first position, is the maximum
// taken, the reference put 2^TC_EXP below it, O and l rescaled and P formed
// again.  The quotient O / l does not depend on the reference.
//
// FP32 queries (SPLIT): q and P as an FP16 head and remainder, each product
// formed twice; Q then lies in shared memory (TMEM is full).
//
// What bounds it: the hand-overs between softmax, issue and tensor cores (about 1,600
// cycles a chunk of 128 x 128, 3,000 with FP32 queries; the products take 1,024 and
// 2,048), and about 20,000 cycles to begin and end a tile.  1,024 queries over 32,768
// positions, 20/5 heads x 128, FP16: 255 us, 1.33 PFLOP/s or 69 % of the
// measured rate (692 us with a maximum per chunk and packed conversions only, 372
// with one chunk in flight, 320 with two issuing warps and no maximum, 253
// with even shares, before scales were cut).  511 queries from 0, FP32: 20 us.
//
// Every wait is bounded by %globaltimer; on expiry the CTA records a timeout
// in the status word, settles its MMAs, frees TMEM and returns; its outputs are not
// valid then.
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

// Waits that ran out in launches that name no record, and how many of them tiles_status has told of.  The first is
// only ever added to: none is lost to a status that is asked for meanwhile.
__device__ unsigned g_expired[2];

constexpr int BM = 128, BN = 128;
constexpr float TC_EXP = 7.f;                    // a new reference puts the row's largest P at 2^7 (a sum of at most 2^14)
constexpr float TC_SUM = 32768.f;                // a chunk's sum that shows every P in range

constexpr int NSM = 256;                         // softmax threads: two per query row
constexpr int W_DQ = 8, W_MMA = 16, NTHR = 640;  // warps: 0-7 softmax, 8-15 dequantisation (K, V), 16 S, 17 P V (18, 19 idle)
// Registers per thread after the split; the launch has 96 for each of its five warpgroups
constexpr int REG_SM = 152, REG_DQ = 64, REG_MMA = 40;
static_assert(2 * REG_SM + 2 * REG_DQ + REG_MMA <= 5 * 96, "the warpgroups' registers come out of the launch's");

template <int HD, bool SPLIT>
struct TcCfg {
    static constexpr uint32_t ATOM = 128 * 128;             // 128 rows x 64 FP16
    static constexpr uint32_t ROWB = (HD / 64) * ATOM;      // a 128-row operand
    static constexpr uint32_t OFF_K = 0, OFF_V = 2 * ROWB;  // two stages each
    static constexpr uint32_t OFF_Q = 4 * ROWB;             // staging of q on its way to TMEM (SPLIT: q itself,
    static constexpr uint32_t OFF_BAR = OFF_Q + 2 * ROWB;   // head and remainder), then of the output, FP32
    // TMEM columns: scores (two buffers), O, P (head, remainder), Q
    static constexpr uint32_t T_O = 2 * BN, T_P = T_O + HD, T_Q = T_P + BN / 2 * (SPLIT ? 2 : 1), T_COLS = 512;
    static_assert(T_Q + (SPLIT ? 0 : HD / 2) <= T_COLS, "TMEM columns");
};

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], s_free[2], pv_done[2], p_full, q_ready, drained[2];
    uint32_t tmem;
    int abort;
    long long wait_ns;  // bound of every wait
    unsigned *status;   // error record (null: g_expired)
    float x[2][BM];     // exchanged between the two threads of a row
    float ref[BM];      // the row's reference, handed on from chunk to chunk
    long long qrow[BM], orow[BM];   // the rows' element offsets in q and in the output
    float fac[BM];      // the power of two that q was multiplied with
};
// (a descriptor's start address has 14 bits of 16 bytes: adding offsets to it never carries out of 256 KB)
template <int HD, bool SPLIT>
constexpr uint32_t tc_smem() { return TcCfg<HD, SPLIT>::OFF_BAR + (uint32_t)sizeof(Bars) + 1024u; }

// Sets error record `status` and its abort word, which a handle's later launches look at, or counts.
// (Out of line: in every wait it costs the loops 1.8 % at 1,024 queries over 32,768 positions.)
__device__ __noinline__ void record(unsigned *status, unsigned where)
{
    if (!status) {
        atomicAdd(g_expired, 1u);
        return;
    }
    if (atomicCAS(status, 0u, (unsigned)lfk::STATUS_TIMEOUT) == 0u) {
        status[1] = where;
        status[2] = blockIdx.x;
        status[3] = blockIdx.y;
    }
    atomicExch(status + 4, 1u);
}
// (The timer is read from the 64th poll on: reading it before costs a wait several times its own length.)
__device__ bool wait_phase(uint64_t *bar, unsigned parity, Bars *b, unsigned where)
{
    unsigned long long t0 = 0;
    for (unsigned it = 1;; ++it) {
        if (lfk::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*reinterpret_cast<volatile int *>(&b->abort)) return false;
            const unsigned long long now = lfk::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if ((long long)(now - t0) > b->wait_ns) {
                *reinterpret_cast<volatile int *>(&b->abort) = 1;
                record(b->status, where);
                return false;
            }
        }
    }
}
// Both of two barriers; asked together, since an answer takes its time.
__device__ __forceinline__ bool wait_both(uint64_t *x, unsigned px, uint64_t *y, unsigned py, Bars *b, unsigned where)
{
    const bool okx = lfk::mbar_try_wait(x, px), oky = lfk::mbar_try_wait(y, py);
    return (okx || wait_phase(x, px, b, where)) && (oky || wait_phase(y, py, b, where + 50));
}
__device__ void settle_phase(uint64_t *bar, unsigned parity)
{
    const unsigned long long t0 = lfk::globaltimer_ns();
    while (!lfk::mbar_try_wait(bar, parity))
        if ((long long)(lfk::globaltimer_ns() - t0) > WAIT_NS) return;
}
// One arrival for a warp whose lanes have each fenced their own writes (256 single arrivals queue up on the
// barrier's word for longer than a product takes).
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane)
{
    __syncwarp();
    if (lane == 0) lfk::mbar_arrive(bar);
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
// D[tmem] (+)= A . B[smem], A in TMEM or (SS) in shared memory.  The descriptors' low words come as a base and a
// constant offset that is added beside the instruction: with descriptors computed ahead, 32 of them live in
// registers that the MMA warp does not have, and an MMA every 117 cycles instead of 64.
template <uint32_t OFF>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 l;\n\t.reg .b64 q;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "add.u32 l, %2, %6;\n\t"
        "mov.b64 q, {l, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], q, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(blo), "r"(bhi), "r"(id), "r"(accum), "n"(OFF)
        : "memory");
}
template <uint32_t AOFF, uint32_t OFF>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 l;\n\t.reg .b64 q, r;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "add.u32 l, %1, %6;\n\t"
        "mov.b64 r, {l, %3};\n\t"
        "add.u32 l, %2, %7;\n\t"
        "mov.b64 q, {l, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], r, q, %4, p;\n\t}"
        ::"r"(d), "r"(alo), "r"(blo), "r"(hi), "r"(id), "r"(accum), "n"(AOFF), "n"(OFF)
        : "memory");
}
template <uint32_t N>
struct Int {
    static constexpr uint32_t value = N;
};
// f(Int<0>), f(Int<1>), .. f(Int<N - 1>)
template <uint32_t N, class F>
__device__ __forceinline__ void unroll(F &&f)
{
    if constexpr (N > 0) {
        unroll<N - 1>(f);
        f(Int<N - 1>{});
    }
}

// One position's row: HD / 2 code bytes and HD / 16 scales, held in registers.
template <int HD>
struct RawRow {
    uint4 c[HD / 32];
    uint2 s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales)
    {
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) c[j] = ld(reinterpret_cast<const uint4 *>(codes) + j);
        if (HD == 128) s = ld(reinterpret_cast<const uint2 *>(scales));
        else s = make_uint2(ld(reinterpret_cast<const unsigned *>(scales)), 0u);
    }
    // One row of an operand tile: 16-byte group c of its 64-dim half h to at[c] + h * 16,384 (the shared-memory
    // addresses of the row's eight swizzled groups) + off.
    __device__ __forceinline__ void store(const uint32_t (&at)[8], uint32_t off) const
    {
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {            // 32 values: two blocks
            const unsigned sw = j < 2 ? s.x : s.y;
            const unsigned sc = scales_h2(j & 1 ? sw >> 16 : sw);   // (K's too: one instruction for 32 values)
            const __half2 s2 = *reinterpret_cast<const __half2 *>(&sc);
            const __half2 lo = __low2half2(s2), hi = __high2half2(s2);
            const unsigned w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {              // 8 values: 16 bytes of FP16
                unsigned h[4];
                e2m1x8_h2(w[u], h[0], h[1], h[2], h[3]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&h[q]), u < 2 ? lo : hi);
                    h[q] = *reinterpret_cast<const unsigned *>(&v);
                }
                const int c16 = 4 * j + u;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at[c16 % 8] + off + (uint32_t)(c16 / 8) * 16384u),
                             "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                             : "memory");
            }
        }
    }
};

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one()
{
    unsigned r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// The two warps that share 32 rows (w and w + 4): OR of a predicate, a barrier, and the hand-over from one
// group to the other (arrive by the one, sync by the other).
__device__ __forceinline__ bool pair_or(int warp, bool pred)
{
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.or.pred q, %1, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(1 + (warp & 3)), "r"((unsigned)pred)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void pair_sync(int warp) { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory"); }
__device__ __forceinline__ void all_rows_sync() { asm volatile("bar.sync 13, 256;" ::: "memory"); }   // the softmax warps
__device__ __forceinline__ void hand_over(int warp)
{
    asm volatile("bar.arrive %0, 64;" ::"r"(5 + (warp & 7)) : "memory");
}
__device__ __forceinline__ void take_over(int warp)
{
    asm volatile("bar.sync %0, 64;" ::"r"(5 + ((warp ^ 4) & 7)) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void load64(uint32_t ts, uint32_t (&u)[2][32])
{
    tmem_ld32(ts, u[0]);
    tmem_ld32(ts + 32u, u[1]);
    tmem_ld_wait();
}

// 2^(f s + neg) of 64 scores (0 outside columns lo .. hi - 1 unless WHOLE) as FP16 pairs hw (SPLIT: and the
// remainders lw), and their sum.
template <bool WHOLE, bool SPLIT>
__device__ __forceinline__ float probs(const uint32_t (&u)[2][32], float f, float neg, int lo, int hi, uint32_t (&hw)[32],
                                       uint32_t (&lw)[32])
{
    const uint64_t ff = pack2(f, f), nn = pack2(neg, neg);
    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        float2 y = unpack2(fma2(pack2u(u[e / 32][e % 32], u[e / 32][e % 32 + 1]), ff, nn));
        if (!WHOLE) {
            if (e < lo || e >= hi) y.x = -INFINITY;
            if (e + 1 < lo || e + 1 >= hi) y.y = -INFINITY;
        }
        const float x0 = ex2(y.x), x1 = ex2(y.y);
        acc[e / 2 & 1] = add2(acc[e / 2 & 1], pack2(x0, x1));
        const __half2 h = __floats2half2_rn(x0, x1);
        hw[e / 2] = *reinterpret_cast<const unsigned *>(&h);
        if (SPLIT) {
            const float2 b = __half22float2(h);
            const __half2 r = __floats2half2_rn(x0 - b.x, x1 - b.y);
            lw[e / 2] = *reinterpret_cast<const unsigned *>(&r);
        }
    }
    const float2 t = unpack2(add2(acc[0], acc[1]));
    return t.x + t.y;
}
// The largest of m and 64 scores of columns lo .. hi - 1.
__device__ __forceinline__ float row_max(float m, const uint32_t (&u)[2][32], int lo, int hi)
{
#pragma unroll
    for (int e = 0; e < 64; ++e)
        if (e >= lo && e < hi) m = fmaxf(m, __uint_as_float(u[e / 32][e % 32]));
    return m;
}

template <int HD, bool SPLIT>
__global__ void __launch_bounds__(NTHR, 1) attn_tiles(const __grid_constant__ Attn a, const __grid_constant__ Shares sh)
{
    using C = TcCfg<HD, SPLIT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~uintptr_t(1023));
    Bars *b = reinterpret_cast<Bars *>(smem + C::OFF_BAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA's share of the tiles, tile by tile
    Share begin, end;
    if (a.per == 0) {                                     // one tile, the longest (latest) ones first
        begin = {(int)(blockIdx.x % a.c.Hkv) * a.tiles + a.tiles - 1 - (int)(blockIdx.x / a.c.Hkv), 0, 0};
        end = {begin.tile + 1, 0, 0};
    } else {
        begin = sh.at[blockIdx.x];
        end = sh.at[blockIdx.x + 1];
    }
    struct Walk {
        int tile, skip, piece, kvh, t;   // t: the tile within KV head kvh
    };
    const Walk start = {begin.tile, begin.skip, begin.piece, begin.tile / a.tiles, begin.tile % a.tiles};
    struct Seg {
        int gt, kvh, r0, rows, lo, p0, p1, nc, piece;
        bool first, last;       // the tile's first chunks, its last ones
    };
    auto next = [&](Walk &w, Seg &s) -> bool {
        if (w.tile > end.tile || (w.tile == end.tile && w.skip >= end.skip)) return false;
        s.gt = w.tile;
        s.kvh = w.kvh;
        const int tile = w.t;
        s.r0 = tile * BM;
        s.rows = min(BM, a.n * a.G - s.r0);
        const int t_first = row_token(a, s.r0), t_last = row_token(a, s.r0 + s.rows - 1);
        const int hi = key_hi(a.pos, t_last, a.len);
        int c0;
        const int all = tile_chunks(a, tile, c0), stop = w.tile == end.tile ? end.skip : all;
        s.lo = key_lo(a.pos, t_first, a.win);
        s.p0 = max((c0 + w.skip) * BN, s.lo / BN * BN);
        s.p1 = hi > s.lo ? min((c0 + stop) * BN, hi) : 0;     // no position at all: an empty range
        s.nc = s.p1 > s.p0 ? (s.p1 - s.p0 + BN - 1) / BN : 0;
        s.first = w.skip == 0;
        s.last = stop == all;
        s.piece = w.piece;
        w = tile + 1 < a.tiles ? Walk{w.tile + 1, 0, 0, w.kvh, tile + 1} : Walk{w.tile + 1, 0, 0, w.kvh + 1, 0};
        return true;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            lfk::mbar_init(&b->k_full[i], 4);
            lfk::mbar_init(&b->k_empty[i], 1);
            lfk::mbar_init(&b->v_full[i], 4);
            lfk::mbar_init(&b->v_empty[i], 1);
            lfk::mbar_init(&b->s_full[i], 1);
            lfk::mbar_init(&b->s_free[i], SPLIT ? 5 : 4);
            lfk::mbar_init(&b->drained[i], 1);
            lfk::mbar_init(&b->pv_done[i], 1);
        }
        lfk::mbar_init(&b->p_full, a.fault ? 5 : 4);      // the test hook: a fifth arrival that never comes
        lfk::mbar_init(&b->q_ready, NSM / 32);
        b->abort = 0;
        b->wait_ns = a.wait_ns;
        b->status = a.status;
        lfk::mbar_fence_init();
    }
    if (warp == W_MMA) {
        tmem_alloc(&b->tmem, C::T_COLS);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    // All 512 columns are this CTA's, so the allocation starts at column 0: constant addresses keep the MMA
    // warp's operands out of the vector registers.  (Anything else would be a broken allocation: nothing runs.)
    constexpr uint32_t tmem = 0;
    dependents_may_launch();
    wait_for_prerequisites();
    if (threadIdx.x == 0 && b->tmem != 0u) {
        b->abort = 1;
        record(a.status, 711);
    }
    __syncthreads();
    const bool dead = b->abort != 0;

    if (warp >= W_MMA) {
        setmaxnreg_dec<REG_MMA>();
        // One warp issues the S products, another the P V products: a wait takes as long as a third of a product
        // even when what it waits for is there.  Each warp walks its loop with uniform values; one elected lane
        // issues.
        const bool one = elect_one();
        const uint32_t sb = lfk::smem_u32(smem);
        Walk walk = start;
        Seg g;
        unsigned use0 = 0, use1 = 0;                      // chunks so far in each stage: a barrier's phases
        if (warp == W_MMA && !dead) {
            const uint64_t kd = sdesc_kmajor_sw128(sb + C::OFF_K);
            const uint32_t klo = (uint32_t)kd, khi = (uint32_t)(kd >> 32);
            const uint32_t qlo = (uint32_t)sdesc_kmajor_sw128(sb + C::OFF_Q);
            auto step = [&](int i, auto stage) -> bool {
                constexpr uint32_t S = decltype(stage)::value, D = tmem + S * BN;
                const unsigned ph = ((S ? use1 : use0) + (unsigned)(i >> 1)) & 1u;
                if (!__all_sync(0xffffffffu, wait_both(&b->s_free[S], ph ^ 1u, &b->k_full[S], ph, b, 701))) return false;
                fence_after_sync();
                if (one) {
                    unroll<HD / 16>([&](auto kc) {
                        constexpr uint32_t kk = decltype(kc)::value, off = (kk / 4 * C::ATOM + kk % 4 * 32u) >> 4;
                        constexpr uint32_t id = idesc(BM, BN, false);
                        if constexpr (SPLIT) {
                            mma_ss<off, off + (S * C::ROWB >> 4)>(D, qlo, klo, khi, id, kk != 0);
                            mma_ss<off + (C::ROWB >> 4), off + (S * C::ROWB >> 4)>(D, qlo, klo, khi, id, 1u);
                        } else {
                            mma_ts<off + (S * C::ROWB >> 4)>(D, tmem + C::T_Q + kk * 8u, klo, khi, id, kk != 0);
                        }
                    });
                    commit(&b->k_empty[S]);
                    commit(&b->s_full[S]);
                }
                __syncwarp();
                return true;
            };
            bool ok = true;
            for (unsigned n = 0; ok && next(walk, g); ++n) {
                ok = __all_sync(0xffffffffu, wait_phase(&b->q_ready, n & 1u, b, 700));
                for (int i = 0; ok && i < g.nc; i += 2) ok = step(i, Int<0>{}) && (i + 1 >= g.nc || step(i + 1, Int<1>{}));
                use0 += (unsigned)(g.nc + 1) / 2;
                use1 += (unsigned)g.nc / 2;
            }
        } else if (warp == W_MMA + 1 && !dead) {
            const uint64_t vd = sdesc_mn_sw128(sb + C::OFF_V, C::ATOM);
            const uint32_t vlo = (uint32_t)vd, vhi = (uint32_t)(vd >> 32);
            auto step = [&](int i, auto stage) -> bool {
                constexpr uint32_t S = decltype(stage)::value;
                if (!__all_sync(0xffffffffu, wait_both(&b->v_full[S], ((S ? use1 : use0) + (unsigned)(i >> 1)) & 1u, &b->p_full,
                                                       (use0 + use1 + (unsigned)i) & 1u, b, 702)))
                    return false;
                fence_after_sync();
                if (one) {
                    unroll<BN / 16>([&](auto kc) {
                        constexpr uint32_t kk = decltype(kc)::value, off = (S * C::ROWB >> 4) + kk * 128u;
                        constexpr uint32_t id = idesc(BM, HD, true);
                        mma_ts<off>(tmem + C::T_O, tmem + C::T_P + kk * 8u, vlo, vhi, id, kk != 0 ? 1u : (uint32_t)(i != 0));
                        if constexpr (SPLIT)
                            mma_ts<off>(tmem + C::T_O, tmem + C::T_P + BN / 2 + kk * 8u, vlo, vhi, id, 1u);
                    });
                    commit(&b->v_empty[S]);
                    commit(&b->pv_done[S]);
                    // its scores are free with P (SPLIT): the next S goes behind this product, not before it
                    if (SPLIT) lfk::mbar_arrive(&b->s_free[S]);
                }
                __syncwarp();
                return true;
            };
            bool ok = true;
            while (ok && next(walk, g)) {
                for (int i = 0; ok && i < g.nc; i += 2) ok = step(i, Int<0>{}) && (i + 1 >= g.nc || step(i + 1, Int<1>{}));
                use0 += (unsigned)(g.nc + 1) / 2;
                use1 += (unsigned)g.nc / 2;
            }
        }
    } else if (warp >= W_DQ) {
        // ---- dequantisation: one warpgroup takes K, the other V; thread j position j of every chunk
        setmaxnreg_dec<REG_DQ>();
        const int j = threadIdx.x & 127;
        const bool isv = warp >= W_DQ + 4;
        uint64_t *full = isv ? b->v_full : b->k_full, *empty = isv ? b->v_empty : b->k_empty;
        uint32_t at[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) at[c] = lfk::smem_u32(smem) + (isv ? C::OFF_V : C::OFF_K) + sw128(j, c);
        RawRow<HD> raw;
        Walk walk = start;
        Seg g;
        unsigned use0 = 0, use1 = 0;
        // A lane whose wait ran out stays with its warp to the end, doing nothing: the others' barriers count on it
        // (0.4 % faster at 1,024 queries over 32,768 positions than a vote on who goes on).
        bool ok = !dead;
        while (next(walk, g)) {
            const size_t row0 = (size_t)g.kvh * a.c.cap;
            const uint8_t *codes = (isv ? a.c.vc : a.c.kc) + row0 * code_bytes(HD);
            const uint8_t *scales = (isv ? a.c.vs : a.c.ks) + row0 * scale_bytes(HD);
            auto fetch = [&](int i) {
                const size_t r = (size_t)max(min(g.p0 + i * BN + j, g.p1 - 1), g.lo);   // outside: a seen row, masked
                raw.load(codes + r * code_bytes(HD), scales + r * scale_bytes(HD));
            };
            auto step = [&](int i, auto stage) {
                constexpr uint32_t S = decltype(stage)::value;
                ok = ok && wait_phase(&empty[S], (((S ? use1 : use0) + (unsigned)(i >> 1)) & 1u) ^ 1u, b, 705);
                if (ok) {
                    raw.store(at, S * C::ROWB);
                    fence_async_smem();
                }
                warp_arrive(&full[S], lane);
                if (i + 1 < g.nc) fetch(i + 1);
            };
            if (g.nc > 0) fetch(0);
            for (int i = 0; i < g.nc; i += 2) {
                step(i, Int<0>{});
                if (i + 1 < g.nc) step(i + 1, Int<1>{});
            }
            use0 += (unsigned)(g.nc + 1) / 2;
            use1 += (unsigned)g.nc / 2;
        }
    } else {
        // ---- softmax and output: thread (r, hf) takes chunks hf, hf + 2, .. for row r, and half of its q and of
        // its output
        setmaxnreg_inc<REG_SM>();
        const int hf = warp >> 2, r = (warp & 3) * 32 + lane;
        Walk walk = start;
        Seg g;
        unsigned use0 = 0, use1 = 0;
        bool run = true;
        while (next(walk, g)) {
        const int nc = g.nc, p0 = g.p0;
        const bool live = r < g.rows;
        const int tok = row_token(a, g.r0 + min(r, g.rows - 1)), head = row_head(a, g.kvh, g.r0 + min(r, g.rows - 1), tok);
        if (hf == 0) b->qrow[r] = (long long)tok * a.q.ts + (long long)head * a.q.hs;
        else b->orow[r] = (long long)tok * a.o.ts + (long long)head * a.o.hs;
        all_rows_sync();                                  // the rows' places
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // ---- q: a row's lanes side by side, so that the loads are whole lines; a power of two brings BF16 and FP32
        // rows into FP16's range, a negative scale turns them
        {
            constexpr int V = SPLIT ? 4 : 8, L = HD / V, P = 128 * L / NSM;   // values per lane, lanes per row, passes
            uint4 raw[P];
            const int c = threadIdx.x % L;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int row = i * (NSM / L) + threadIdx.x / L;
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if (row < g.rows)
                    raw[i] = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.q.p) + (b->qrow[row] + c * V) * (16 / V));
            }
            uint8_t *qs = smem + C::OFF_Q;
            auto place = [&](int i) { return i * (NSM / L) + (int)threadIdx.x / L; };
            if (!SPLIT && a.q.dtype == F16 && a.scale > 0.f) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    *reinterpret_cast<uint4 *>(qs + place(i) * (HD * 2) + ((c ^ (place(i) & 7)) << 4)) = raw[i];
                    if (c == 0) b->fac[place(i)] = 1.f;
                }
            } else {
                float fac[P];
                if (a.q.dtype == F16) {
#pragma unroll
                    for (int i = 0; i < P; ++i) fac[i] = 1.f;
                } else {
                    // the largest magnitude's bits (FP32's; BF16's lie in their upper half)
                    unsigned m[P];
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const unsigned w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                        m[i] = 0u;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            m[i] = max(m[i], w[u] & (SPLIT ? 0x7fffffffu : 0x7fff0000u));
                            if (!SPLIT) m[i] = max(m[i], (w[u] << 16) & 0x7fff0000u);
                        }
                    }
#pragma unroll
                    for (int o = L / 2; o; o >>= 1)
#pragma unroll
                        for (int i = 0; i < P; ++i) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
                    for (int i = 0; i < P; ++i) fac[i] = range_factor(__uint_as_float(m[i]));
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (c == 0) b->fac[place(i)] = fac[i];
                    const float fc = a.scale < 0.f ? -fac[i] : fac[i];
                    const unsigned w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                    if constexpr (SPLIT) {                    // to its place in the K-major operand
                        __half h[4], m[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) lfk::split_h(__uint_as_float(w[u]) * fc, h[u], m[u]);
                        const int d = c * V;
                        uint8_t *at = qs + (d / 64) * C::ATOM + sw128(place(i), d % 64 / 8) + d % 8 * 2;
                        *reinterpret_cast<uint2 *>(at) = make_uint2(lfk::pack_h2(h[0], h[1]), lfk::pack_h2(h[2], h[3]));
                        *reinterpret_cast<uint2 *>(at + C::ROWB) = make_uint2(lfk::pack_h2(m[0], m[1]), lfk::pack_h2(m[2], m[3]));
                    } else {
                        uint32_t hw[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 y = a.q.dtype == F16 ? h2_f2(w[u])
                                                              : make_float2(__uint_as_float(w[u] << 16), __uint_as_float(w[u] & 0xffff0000u));
                            const __half2 v = __floats2half2_rn(y.x * fc, y.y * fc);
                            hw[u] = *reinterpret_cast<const unsigned *>(&v);
                        }
                        *reinterpret_cast<uint4 *>(qs + place(i) * (HD * 2) + ((c ^ (place(i) & 7)) << 4)) =
                            make_uint4(hw[0], hw[1], hw[2], hw[3]);
                    }
                }
            }
        }
        if (SPLIT) fence_async_smem();
        all_rows_sync();
        const float f = fabsf(a.scale) * 1.4426950408889634f / b->fac[r];   // score factor
        if (!SPLIT && 64 * hf < HD) {
            uint32_t hw[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4 *>(smem + C::OFF_Q + r * (HD * 2) + (((8 * hf + c) ^ (r & 7)) << 4));
                hw[4 * c] = v.x, hw[4 * c + 1] = v.y, hw[4 * c + 2] = v.z, hw[4 * c + 3] = v.w;
            }
            tmem_st32(tl + C::T_Q + (uint32_t)(32 * hf), hw);
            tmem_st_wait();
        }
        if (!SPLIT) fence_before_sync();
        warp_arrive(&b->q_ready, lane);
        const int klo = key_lo(a.pos, tok, a.win), khi = min(key_hi(a.pos, tok, a.len), g.p1);
        float ref = -INFINITY, l = 0.f;
        const unsigned mine = hf ? use1 : use0, other = hf ? use0 : use1;
        for (int i = hf; i < nc; i += 2) {
            run = __all_sync(0xffffffffu, run && !dead && wait_phase(&b->s_full[hf], (mine + (unsigned)(i >> 1)) & 1u, b, 707));
            fence_after_sync();
            const uint32_t ts = tl + (uint32_t)hf * BN;
            const int key0 = p0 + i * BN, lo = klo - key0, hi = khi - key0;
            const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= BN);
            uint32_t u[2][32], hw[2][32], lw[32];
            float sum = 0.f, now = -INFINITY;
            // P of one half of the chunk; put: into its columns
            auto half = [&](int h, float neg, auto all) {
                constexpr bool WHOLE = decltype(all)::value != 0;
                sum += probs<WHOLE, SPLIT>(u, f, neg, lo - 64 * h, hi - 64 * h, hw[h], lw);
            };
            auto put = [&](int h) {
                tmem_st32(tl + C::T_P + (uint32_t)(32 * h), hw[h]);
                if (SPLIT) tmem_st32(tl + C::T_P + BN / 2 + (uint32_t)(32 * h), lw);
            };
            // P's columns are free once the previous chunk's product has read them: FP16 P waits in registers
            // for that until the chunk's end; head and remainder do not fit there, their first half waits midway.
            // (One barrier per parity: this warp waited for PV(i - 3) in its chunk before, so that the phase it waits
            // for now is PV(i - 1)'s and no earlier one.)
            auto p_free = [&] {
                if (i == 0) return;
                run = __all_sync(0xffffffffu, run && wait_phase(&b->pv_done[hf ^ 1], (other + (unsigned)((i - 1) >> 1)) & 1u, b, 708));
                fence_after_sync();
            };
            if (i == 1) {                                     // nothing known of the row yet: the first chunk's reference
                take_over(warp);
                ref = now = b->ref[r];
            }
            if (i > 0 && run) {
                const float neg = ref == -INFINITY ? 0.f : -ref;
                load64(ts + 64u, u);
                if (whole) half(1, neg, Int<1>{});
                else half(1, neg, Int<0>{});
                load64(ts, u);
                if (SPLIT) {
                    p_free();
                    put(1);
                }
                if (whole) half(0, neg, Int<1>{});
                else half(0, neg, Int<0>{});
                if (SPLIT) put(0);
            }
            // ---- the reference after the chunk before (the hand-over also runs after a failed wait)
            if (i > 1) {
                take_over(warp);
                now = b->ref[r];
            }
            const bool again = now != ref || now == -INFINITY || !(sum <= TC_SUM);
            if (run && __any_sync(0xffffffffu, again)) {
                float m = -INFINITY, alpha = 1.f;
                load64(ts + 64u, u);
                m = row_max(m, u, lo - 64, hi - 64);
                load64(ts, u);
                m = row_max(m, u, lo, hi);
                m = m == -INFINITY ? m : m * f;
                const bool up = m > now && (now == -INFINITY || m - now > TC_EXP + 1.f);
                if (up) {
                    float n = m - TC_EXP;
                    if (!(m - n <= 15.f)) n = m;              // scores so large that their steps are
                    alpha = ex2(now - n);                     // 0 from -inf
                    now = n;
                }
                if (i > 0 && __any_sync(0xffffffffu, up)) {
                    if (!SPLIT) p_free();                     // and O holds every earlier product
#pragma unroll 1
                    for (int c = 0; c < HD / 16; ++c) {
                        const uint32_t oc = tl + C::T_O + (uint32_t)(16 * c);
                        uint32_t o[16];
                        tmem_ld16(oc, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(oc, o);
                    }
                }
                const float neg = now == -INFINITY ? 0.f : -now;
                sum = 0.f;
                half(0, neg, Int<0>{});
                if (SPLIT) put(0);
                load64(ts + 64u, u);
                half(1, neg, Int<0>{});
                if (SPLIT) put(1);
            }
            if (i + 1 < nc) {
                b->ref[r] = now;
                hand_over(warp);
            }
            if (now != ref) {                                 // moved since this thread's last chunk
                l *= ex2(ref - now);
                ref = now;
            }
            l += sum;
            if (!SPLIT) {
                fence_before_sync();
                warp_arrive(&b->s_free[hf], lane);            // the scores are read: the next product may replace them
                p_free();
                if (!run) continue;
                put(1);
                put(0);
            }
            if (!run) continue;
            tmem_st_wait();
            fence_before_sync();
            if (SPLIT) warp_arrive(&b->s_free[hf], lane);
            warp_arrive(&b->p_full, lane);
        }
        // ---- output: O / l, or the partial state of a split
        if (run && nc > 0) {
            run = __all_sync(0xffffffffu, wait_phase(&b->pv_done[(nc - 1) & 1], (((nc - 1) & 1 ? use1 : use0) + (unsigned)((nc - 1) >> 1)) & 1u, b, 710));
            fence_after_sync();
        }
        // the reference of the last chunk is its group's; the other group's sum follows it
        if (nc > 0 && ((nc - 1) & 1) == hf) b->ref[r] = ref;
        pair_sync(warp);
        const float last = nc > 0 ? b->ref[r] : -INFINITY;
        if (last != ref) l *= ex2(ref - last);
        ref = last;
        b->x[hf][r] = l;
        const bool good = !pair_or(warp, !run);
        l = b->x[0][r] + b->x[1][r];
        // a whole tile: its output; a piece of one: a partial state (and the last piece says where they are)
        const bool whole_tile = g.first && g.last;
        float *part = whole_tile ? nullptr : a.part + (size_t)(2 * blockIdx.x + (g.first ? 1 : 0)) * BM * (HD + PAD);
        if (a.pieces && g.last && threadIdx.x == 0)
            a.pieces[g.gt] = whole_tile ? make_int2(0, 0) : make_int2((int)blockIdx.x - g.piece, g.piece + 1);
        // through shared memory (q's staging, read by now), so that the stores are whole lines
        if (good) {
            const float inv = part ? 1.f : (l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l));   // a row that saw nothing is 0
#pragma unroll 1
            for (int c = 0; c < HD / 64; ++c) {
                uint32_t o[32];
                if (nc > 0) {
                    tmem_ld32(tl + C::T_O + (uint32_t)(HD / 2 * hf + 32 * c), o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const int c16 = (HD / 2 * hf + 32 * c + e) / 4;
                    *reinterpret_cast<float4 *>(smem + C::OFF_Q + r * (HD * 4) + ((c16 ^ (r & 7)) << 4)) =
                        make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                    __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                }
            }
            if (part && live && hf == 0) *reinterpret_cast<float2 *>(part + (size_t)r * (HD + PAD) + HD) = make_float2(ref, l);
        }
        fence_before_sync();                              // O is read: the next tile's first product overwrites it
        all_rows_sync();
        {
            // V values per lane: 16 bytes in the staging's FP32, or in a 16-bit output
            auto copy = [&](auto lanes, auto put) {
                constexpr int L = decltype(lanes)::value, V = HD / L;
                const int c = threadIdx.x % L;
#pragma unroll 2
                for (int row = threadIdx.x / L; row < g.rows; row += NSM / L) {
                    float4 v[V / 4];
#pragma unroll
                    for (int u = 0; u < V / 4; ++u)
                        v[u] = *reinterpret_cast<const float4 *>(smem + C::OFF_Q + row * (HD * 4) + (((c * (V / 4) + u) ^ (row & 7)) << 4));
                    put(row, c * V, v);
                }
            };
            if (part)
                copy(Int<HD / 4>{}, [&](int row, int d, const float4 *v) {
                    *reinterpret_cast<float4 *>(part + (size_t)row * (HD + PAD) + d) = v[0];
                });
            else if (a.o.dtype == F16 || a.o.dtype == BF16)
                copy(Int<HD / 8>{}, [&](int row, int d, const float4 *v) {
                    uint4 w;
                    if (a.o.dtype == F16) {
                        const __half2 x[4] = {__floats2half2_rn(v[0].x, v[0].y), __floats2half2_rn(v[0].z, v[0].w),
                                              __floats2half2_rn(v[1].x, v[1].y), __floats2half2_rn(v[1].z, v[1].w)};
                        w = *reinterpret_cast<const uint4 *>(x);
                    } else {
                        w = make_uint4(pack_bf2(v[0].x, v[0].y), pack_bf2(v[0].z, v[0].w), pack_bf2(v[1].x, v[1].y),
                                       pack_bf2(v[1].z, v[1].w));
                    }
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o.p) + b->orow[row] + d) = w;
                });
            else
                copy(Int<HD / 4>{}, [&](int row, int d, const float4 *v) {
                    store4(a.o, (size_t)b->orow[row] + d, v[0].x, v[0].y, v[0].z, v[0].w);
                });
        }
        all_rows_sync();                                  // the staging is free for the next tile's q
        use0 += (unsigned)(nc + 1) / 2;
        use1 += (unsigned)nc / 2;
        }
        tmem_st_wait();                                   // P that no product waited for
    }
    fence_before_sync();
    __syncthreads();
    // After a wait that ran out, products may be under way that nothing waited for.  Every role has ended, so none
    // follows: one more commit by each of the lanes that issued, and TMEM goes when they are done.
    if (b->abort) {
        if (warp == W_MMA || warp == W_MMA + 1) {
            if (elect_one()) {
                commit(&b->drained[warp - W_MMA]);
                settle_phase(&b->drained[warp - W_MMA], 0u);
            }
            __syncwarp();
        }
        __syncthreads();
    }
    if (warp == W_MMA) {
        __syncwarp();
        fence_after_sync();
        tmem_dealloc(b->tmem, C::T_COLS);
    }
}

template <int HD, bool SPLIT>
static cudaError_t run_tiles(const Attn &a, const Shares &sh, cudaStream_t s)
{
    constexpr int smem = (int)tc_smem<HD, SPLIT>();
    static_assert(smem <= 232448, "shared memory of the tiles kernel");
    static bool ready[64] = {};   // the attribute is per device; setting it again is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev]) {
        // the register split waits for ever unless the launch holds what it hands out
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, attn_tiles<HD, SPLIT>);
        if (e != cudaSuccess) return e;
        if ((fa.numRegs + 7) / 8 * 8 * 5 < 2 * REG_SM + 2 * REG_DQ + REG_MMA) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(attn_tiles<HD, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.splits);
    cfg.blockDim = dim3(NTHR);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tiles<HD, SPLIT>, a, sh);
}

cudaError_t launch_attn_tiles(const Attn &a, cudaStream_t s)
{
    Shares sh;
    if (a.per > 0 && (a.per > MAX_CTAS || share_tiles(a, a.per, sh) != a.splits)) return cudaErrorInvalidConfiguration;
    const bool split = a.q.dtype == F32;
    if (a.c.hd == 128) return split ? run_tiles<128, true>(a, sh, s) : run_tiles<128, false>(a, sh, s);
    return split ? run_tiles<64, true>(a, sh, s) : run_tiles<64, false>(a, sh, s);
}

cudaError_t tiles_status(bool &expired, cudaStream_t s)
{
    void *p = nullptr;
    unsigned w[2] = {0, 0};
    cudaError_t e = cudaGetSymbolAddress(&p, g_expired);
    if (e == cudaSuccess) e = cudaMemcpyAsync(w, p, sizeof(w), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    expired = w[0] != w[1];
    if (e == cudaSuccess && expired) {
        e = cudaMemcpyAsync(static_cast<unsigned *>(p) + 1, w, sizeof(w[0]), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace lfq
