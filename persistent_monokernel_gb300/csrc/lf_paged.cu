// lf_paged.cu -- a KV cache of many sequences in pages: the plan of their pages
// and slots, the append, and the C entry points of these and the attention.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/lf.h"
#include "lf_kv4.cuh"
#include "lf_paged.h"
#include "lf_rows.cuh"

namespace lfpg {

// ---------------------------------------------------------------- plan

// Row i keeps kept = min(lens, keep) positions and gives the pages behind them back, then takes n_new more.  With
// stay, held, want the pages of kept, lens and kept + n_new positions:
//   the pages stay .. held - 1 of all rows, rows in order, are the back entries 0 ..; entry k goes to
//   free[top - 1 - k], top = n_free + (their number);
//   the pages stay .. want - 1 of all rows are the need entries 0 ..; entry k comes from free[top - 1 - k].
// So a plan that takes back exactly what the one before it took finds the same pages again.
//
// Three sums over the rows say where everything lies; after them every page and token finds its row by a search in
// shared memory, however uneven the rows are.  Every CTA of the (only) cluster forms the sums for itself: they are
// a read of a few KB, and nothing has to be handed over.  What is read and what is written overlaps (lens, n_free,
// table entries given back and taken anew), hence one cluster barrier between reading and writing.  Many tokens are
// left to a second launch, which needs no more than the tables and offsets that the first one wrote.
//
// Bound by latency: the loads of the rows, the sums' shuffles, a search and two dependent loads per token.  64 rows of one
// token: 4.1 us; 500 rows, 71,360 tokens: 8.7 us (13.9 with all tokens in the one cluster, 10.0 with clusters of four
// for the 5,000 pages), 8,000 rows: 25 us.
__device__ __forceinline__ int row_of(const int *before, int n, int k)   // the last row with before[row] <= k
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= k) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Position to page: a shift where the page is a power of two.
__device__ __forceinline__ int page_of(const Plan &p, int shift, int x)
{
    return shift >= 0 ? x >> shift : (int)((unsigned)x / (unsigned)p.page);
}

// Slots and positions of tokens t0 .. t0 + 3 (and nothing behind max_tokens).  tok: tokens before each row;
// first(r): position of row r's first; page(r, c): its c-th page.
template <class First, class Page>
__device__ __forceinline__ void four_tokens(const Plan &p, int t0, int tokens, const int *tok, int shift, First first, Page page)
{
    int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0};
    if (t0 < tokens) {
        int r = row_of(tok, p.n, t0), base = first(r), have = -1, id = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i;
            if (t >= tokens) break;
            while (t >= tok[r + 1]) base = first(++r), have = -1;
            const int x = base + t - tok[r], c = page_of(p, shift, x);
            if (c != have) have = c, id = page(r, c);
            slot[i] = id * p.page + x - c * p.page;
            pos[i] = x;
        }
    }
    if (t0 + 4 <= p.max_tokens) {
        *reinterpret_cast<int4 *>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t0 + i < p.max_tokens) {
                p.slots[t0 + i] = slot[i];
                p.positions[t0 + i] = pos[i];
            }
    }
}

__global__ void __launch_bounds__(1024) plan_pages(const __grid_constant__ Plan p, int ctas, int shift, bool with_tokens)
{
    extern __shared__ int smem[];
    int *const kept = smem, *const tok = kept + p.n, *const back = tok + p.n + 1, *const need = back + p.n + 1;
    __shared__ unsigned wsum[4][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    lfq::dependents_may_launch();
    lfq::wait_for_prerequisites();
    auto pages = [&](int x) { return x ? page_of(p, shift, x - 1) + 1 : 0; };

    // ---- the rows' numbers (new tokens, pages back, pages needed), and their sums up to each row.  The sums saturate:
    // one that leaves 32 bits is more than any pool or max_tokens.
    const int per = (p.n + blockDim.x - 1) / blockDim.x;
    const int r0 = min(tid * per, p.n), r1 = min(r0 + per, p.n);
    const long long cap = (long long)p.max_pages * p.page;
    const int n_free = lfq::ld(p.n_free);
    unsigned wrong = n_free < 0 || n_free > p.n_pages ? 1u : 0u;         // bit 0: INVALID_ARG, bit 1: CAPACITY
    auto row = [&](int r, unsigned (&x)[3]) {
        const int len = lfq::ld(p.lens + r), n_new = lfq::ld(p.n_new + r);
        const int keep = p.keep ? lfq::ld(p.keep + r) : len, k = min(len, keep);
        x[0] = x[1] = x[2] = 0;
        if (len < 0 || len > cap || keep < 0 || n_new < 0) {
            wrong |= 1u;
            return 0;
        }
        if ((long long)k + n_new > cap) {
            wrong |= 2u;
            return 0;
        }
        x[0] = n_new;
        x[1] = pages(len) - pages(k);
        x[2] = pages(k + n_new) - pages(k);
        return k;
    };
    auto plus = [](unsigned x, unsigned y) { return x + y < x ? 0xffffffffu : x + y; };
    unsigned x[3] = {0, 0, 0}, mine[3] = {0, 0, 0}, at[3], sum[3];
    int k0 = 0;
    for (int r = r0; r < r1; ++r) {
        k0 = row(r, x);
        for (int i = 0; i < 3; ++i) mine[i] = plus(mine[i], x[i]);
    }
    auto scan = [&](unsigned (&v)[3]) {              // inclusive, over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const unsigned y = __shfl_up_sync(0xffffffffu, v[i], d);
                if (lane >= d) v[i] = plus(v[i], y);
            }
    };
    unsigned incl[3] = {mine[0], mine[1], mine[2]}, all_w[3];
    scan(incl);
    const unsigned some = __reduce_or_sync(0xffffffffu, wrong);
    if (lane == 31) wsum[0][warp] = incl[0], wsum[1][warp] = incl[1], wsum[2][warp] = incl[2], wsum[3][warp] = some;
#pragma unroll
    for (int i = 0; i < 3; ++i) {                    // up to this thread's rows
        const unsigned before = __shfl_up_sync(0xffffffffu, incl[i], 1);
        at[i] = lane ? before : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) all_w[i] = lane < warps ? wsum[i][lane] : 0u;
    const unsigned all_wrong = __reduce_or_sync(0xffffffffu, lane < warps ? wsum[3][lane] : 0u);
    scan(all_w);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const unsigned before = __shfl_sync(0xffffffffu, all_w[i], max(warp - 1, 0));
        at[i] = plus(at[i], warp ? before : 0u);
        sum[i] = __shfl_sync(0xffffffffu, all_w[i], 31);
    }
    for (int r = r0; r < r1; ++r) {
        if (per > 1) k0 = row(r, x);
        kept[r] = k0;
        tok[r] = at[0], back[r] = at[1], need[r] = at[2];
        for (int i = 0; i < 3; ++i) at[i] = plus(at[i], x[i]);
    }
    if (tid == 0) tok[p.n] = sum[0], back[p.n] = sum[1], need[p.n] = sum[2];
    __syncthreads();
    // all or nothing: more pages given back than the pool has (tables that are not a plan's), or too few for the rows
    const long long top64 = (long long)n_free + sum[1];
    const bool invalid = (all_wrong & 1u) || top64 > p.n_pages;
    const bool fails = invalid || (all_wrong & 2u) || sum[2] > top64 || sum[0] > (unsigned)p.max_tokens;
    const int all = ctas * blockDim.x, me = blockIdx.x * blockDim.x + tid;
    const int tokens = fails ? 0 : (int)sum[0], n_back = (int)sum[1], n_need = (int)sum[2], top = (int)top64;

    // ---- pages given back
    if (!fails) {
        for (int k = me; k < n_back; k += all) {
            const int r = row_of(back, p.n, k);
            p.free[top - 1 - k] = lfq::ld(p.tables + r * p.tstride + pages(kept[r]) + k - back[r]);
        }
    }
    if (ctas > 1) lfq::cluster_sync();
    else __syncthreads();
    // ---- pages taken, and the rows; the last threads take these, the first ones the tokens
    const int last = all - 1 - me;
    for (int r = last; r <= p.n; r += all) p.offsets[r] = fails ? 0 : tok[r];
    if (!fails) {
        for (int r = last; r < p.n; r += all) p.lens[r] = kept[r] + tok[r + 1] - tok[r];
        if (last == 0) *p.n_free = top - n_need;
        for (int k = last; k < n_need; k += all) {
            const int r = row_of(need, p.n, k);
            p.tables[r * p.tstride + pages(kept[r]) + k - need[r]] = lfq::ld(p.free + top - 1 - k);
        }
    } else if (last == 0 && lfq::ld(p.status) == 0) {
        *p.status = invalid ? LF_ERR_INVALID_ARG : LF_ERR_CAPACITY;
    }
    if (!with_tokens) return;
    for (int t0 = me * 4; t0 < p.max_tokens; t0 += all * 4)
        four_tokens(p, t0, tokens, tok, shift, [&](int r) { return kept[r]; },
                    [&](int r, int c) {
                        const int stay = pages(kept[r]);
                        return c < stay ? lfq::ld(p.tables + r * p.tstride + c) : lfq::ld(p.free + top - 1 - (need[r] + c - stay));
                    });
}

// The slots and positions of many tokens, from what the first launch wrote.
__global__ void __launch_bounds__(256) plan_tokens(const __grid_constant__ Plan p, int shift)
{
    extern __shared__ int smem[];
    lfq::dependents_may_launch();
    lfq::wait_for_prerequisites();
    for (int r = threadIdx.x; r <= p.n; r += 256) smem[r] = lfq::ld(p.offsets + r);
    __syncthreads();
    const int t0 = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (t0 < p.max_tokens)
        four_tokens(p, t0, smem[p.n], smem, shift, [&](int r) { return lfq::ld(p.lens + r) - (smem[r + 1] - smem[r]); },
                    [&](int r, int c) { return lfq::ld(p.tables + r * p.tstride + c); });
}

// ---------------------------------------------------------------- append

// A thread moves 8 values (16 bytes of the cache); one grid row per KV head and K or V, so that no division but the
// slot's finds a place.  Slots outside the pool store nothing.  Bound by memory (8,191 rows of 5 x 128, FP32 to FP16: 10.6 us,
// 5.9 TB/s), and by the launch for few rows (64 of 8 x 128: 1.2 us).
template <class TI, class TO>
__global__ void __launch_bounds__(256) append_rows(const __grid_constant__ Pool c, const __grid_constant__ Rows k,
                                                   const __grid_constant__ Rows v, int n, const int *slots, int shift)
{
    lfq::dependents_may_launch();
    lfq::wait_for_prerequisites();
    const bool isv = blockIdx.y & 1;
    const int h = blockIdx.y >> 1;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, t = i >> shift;   // 2^shift places per row
    const int b = (int)(i & ((1 << shift) - 1));
    if (t >= n) return;
    const Rows &in = isv ? v : k;
    const TI *src = static_cast<const TI *>(in.p) + t * in.ts + h * in.hs + b * 8;
    const unsigned slot = (unsigned)lfq::ld(slots + t);
    uint4 x;
    if constexpr (sizeof(TI) == 2) {
        x = lfq::ld(reinterpret_cast<const uint4 *>(src));
    } else {
        const float4 f = lfq::ld(reinterpret_cast<const float4 *>(src)), g = lfq::ld(reinterpret_cast<const float4 *>(src) + 1);
        auto two = [](float lo, float hi) {
            if constexpr (std::is_same_v<TO, __half>) {
                const __half2 y = __floats2half2_rn(lo, hi);
                return *reinterpret_cast<const unsigned *>(&y);
            } else {
                const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
                return *reinterpret_cast<const unsigned *>(&y);
            }
        };
        x = make_uint4(two(f.x, f.y), two(f.z, f.w), two(g.x, g.y), two(g.z, g.w));
    }
    const unsigned page = slot / (unsigned)c.page;
    if (page >= (unsigned)c.n_pages) return;
    char *dst = (isv ? c.v : c.k) + page * c.page_b + (long long)(slot - page * c.page) * c.pos_b + h * c.head_b + b * 16;
    *reinterpret_cast<uint4 *>(dst) = x;
}

// ---------------------------------------------------------------- launches

cudaError_t launch_plan(const Plan &p, cudaStream_t s)
{
    // One CTA, or a cluster of them where there may be thousands of pages to move: new tokens' and given back ones.
    const bool with_tokens = p.max_tokens <= 4096;
    const long long moves = (long long)p.max_tokens / p.page + p.n;
    const int ctas = moves <= 1024 ? 1 : moves <= 2048 ? 2 : moves <= 4096 ? 4 : 8, threads = p.n <= 256 && p.max_tokens <= 1024 ? 256 : 1024;
    int shift = -1;
    for (int i = 4; i < 31; ++i)
        if (p.page == 1 << i) shift = i;
    static bool ready[64] = {};
    cudaError_t e = lfr::allow_smem(plan_pages, (4 * MAX_ROWS + 3) * (int)sizeof(int), ready);
    if (e != cudaSuccess) return e;
    e = lfr::launch(plan_pages, dim3((unsigned)ctas), threads, (4 * p.n + 3) * (int)sizeof(int), ctas, s, p, ctas, shift, with_tokens);
    if (e != cudaSuccess || with_tokens) return e;
    return lfr::launch(plan_tokens, dim3((unsigned)((p.max_tokens + 1023) / 1024)), 256, (p.n + 1) * (int)sizeof(int), 1, s, p, shift);
}

cudaError_t launch_append(const Pool &c, const Rows &k, const Rows &v, int n, const int *slots, cudaStream_t s)
{
    const int shift = c.hd == 128 ? 4 : 3;
    const dim3 grid((unsigned)((((long long)n << shift) + 255) / 256), (unsigned)(2 * c.Hkv));
    if (k.dtype != LF_F32) return lfr::launch(append_rows<__half, __half>, grid, 256, 0, 1, s, c, k, v, n, slots, shift);
    if (c.bf16) return lfr::launch(append_rows<float, __nv_bfloat16>, grid, 256, 0, 1, s, c, k, v, n, slots, shift);
    return lfr::launch(append_rows<float, __half>, grid, 256, 0, 1, s, c, k, v, n, slots, shift);
}

}  // namespace lfpg

// ---------------------------------------------------------------- C entry points

namespace {

using namespace lfpg;
using lfr::aligned16;
using lfr::check_rows;
using lfr::status_of;

constexpr int kMaxKvHeads = 1024;
constexpr long long kMaxStride = 1ll << 40;   // elements: keeps every offset far inside 64 bits

bool aligned4(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool page_ok(int page) { return page >= 16 && page % 16 == 0; }

lf_status check_pool(const lf_paged *c)
{
    if (!c || c->n_pages < 1 || c->n_kv_heads < 1 || c->page < 1) return LF_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return LF_ERR_NOT_SUPPORTED;
    if (c->dtype != LF_F16 && c->dtype != LF_BF16) return LF_ERR_NOT_SUPPORTED;
    if (c->n_kv_heads > kMaxKvHeads || !page_ok(c->page) || (long long)c->n_pages * c->page > INT32_MAX) return LF_ERR_NOT_SUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v) || c->k == c->v) return LF_ERR_INVALID_ARG;
    struct Dim {
        long long stride, size;
    } dims[3] = {{c->page_stride, c->n_pages}, {c->head_stride, c->n_kv_heads}, {c->pos_stride, c->page}};
    for (Dim &d : dims) {
        if (d.size == 1) d.stride = 0;                 // (never used)
        if (d.stride < 0 || d.stride % 8 || d.stride > kMaxStride) return LF_ERR_INVALID_ARG;
    }
    // no two rows overlap: each stride spans all that lies within it
    std::sort(dims, dims + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    long long extent = c->head_dim;
    for (const Dim &d : dims) {
        if (d.size == 1) continue;
        if (d.stride < extent || d.stride > (INT64_MAX >> 2) / d.size) return LF_ERR_INVALID_ARG;
        extent += d.stride * (d.size - 1);
    }
    return LF_OK;
}

Pool pool_of(const lf_paged *c)
{
    return {static_cast<char *>(c->k), static_cast<char *>(c->v), 2 * c->page_stride, 2 * c->head_stride, 2 * c->pos_stride,
            c->n_pages, c->page, c->n_kv_heads, c->head_dim, c->dtype == LF_BF16};
}
Rows rows_of(const lf_rows *r) { return {r->data, r->dtype, r->token_stride, r->head_stride}; }

lf_status make_attn(const lf_paged *c, const lf_paged_query *q, Attn *a, size_t *bytes)
{
    lf_status st = check_pool(c);
    if (st != LF_OK) return st;
    if (!q || q->n_seqs < 0 || q->n_heads < 1 || q->table_width < 0 || q->table_stride < 0 || q->table_stride > kMaxStride ||
        q->window < 0 || !std::isfinite(q->scale))
        return LF_ERR_INVALID_ARG;
    if (q->n_heads % c->n_kv_heads) return LF_ERR_NOT_SUPPORTED;
    if (q->q.dtype != LF_F16 && q->q.dtype != LF_BF16 && q->q.dtype != LF_F32) return LF_ERR_NOT_SUPPORTED;
    if (q->q.dtype != LF_F32 && q->q.dtype != c->dtype) return LF_ERR_INVALID_ARG;
    // positions and blocks of a launch (at most 8 per row and head) in 32 bits
    if ((long long)q->table_width * c->page > (1 << 30) || (long long)q->n_seqs * q->n_heads > (1 << 27)) return LF_ERR_NOT_SUPPORTED;
    a->c = pool_of(c);
    a->q = rows_of(&q->q);
    a->tables = q->tables;
    a->tstride = q->table_stride;
    a->lens = q->lens;
    a->width = q->table_width;
    a->n = q->n_seqs;
    a->G = q->n_heads / c->n_kv_heads;
    a->win = q->window;
    a->scale = q->scale != 0.f ? q->scale : 1.0f / std::sqrt((float)c->head_dim);
    *bytes = 0;
    if (a->n == 0) return LF_OK;
    int sms = 0;
    st = lfr::sm_count(&sms);
    if (st == LF_OK) *bytes = plan_attn(*a, sms);
    return st;
}

}  // namespace

extern "C" {

lf_status lf_paged_plan(const lf_page_tables *t, const int32_t *n_new, const int32_t *keep, int32_t *slots,
                        int32_t *positions, int32_t *offsets, int32_t max_tokens, void *stream)
{
    if (!t || t->n_seqs < 0 || t->max_pages < 1 || t->n_pages < 1 || t->page < 1 || max_tokens < 0 || t->table_stride < 0 ||
        t->table_stride > kMaxStride || (t->n_seqs > 1 && t->table_stride < t->max_pages))
        return LF_ERR_INVALID_ARG;
    if (!page_ok(t->page) || t->n_seqs > MAX_ROWS || (long long)t->n_pages * t->page > INT32_MAX ||
        (long long)t->max_pages * t->page > (1 << 30) || max_tokens > (1 << 30))
        return LF_ERR_NOT_SUPPORTED;
    if (!aligned4(t->n_free) || !aligned4(t->status) || !aligned4(t->free_pages) || !aligned4(offsets)) return LF_ERR_INVALID_ARG;
    if (t->n_seqs && (!aligned4(t->tables) || !aligned4(t->lens) || !aligned4(n_new) || (keep && !aligned4(keep)))) return LF_ERR_INVALID_ARG;
    if (max_tokens && (!aligned16(slots) || !aligned16(positions))) return LF_ERR_INVALID_ARG;
    const Plan p = {t->tables, t->table_stride, t->lens, t->free_pages, t->n_free, t->status, t->n_seqs, t->max_pages, t->n_pages,
                    t->page, n_new, keep, slots, positions, offsets, max_tokens};
    return status_of(launch_plan(p, static_cast<cudaStream_t>(stream)));
}

lf_status lf_paged_append(const lf_paged *c, const lf_rows *k, const lf_rows *v, int32_t n, const int32_t *slots, void *stream)
{
    lf_status st = check_pool(c);
    if (st != LF_OK) return st;
    if (n < 0) return LF_ERR_INVALID_ARG;
    if (n == 0) return LF_OK;
    st = check_rows(k, n, c->n_kv_heads, c->head_dim, false);
    if (st == LF_OK) st = check_rows(v, n, c->n_kv_heads, c->head_dim, false);
    if (st != LF_OK) return st;
    if (k->dtype != v->dtype || (k->dtype != LF_F32 && k->dtype != c->dtype) || !aligned4(slots)) return LF_ERR_INVALID_ARG;
    return status_of(launch_append(pool_of(c), rows_of(k), rows_of(v), n, slots, static_cast<cudaStream_t>(stream)));
}

lf_status lf_paged_workspace(const lf_paged *c, const lf_paged_query *q, int64_t *bytes)
{
    if (!bytes) return LF_ERR_INVALID_ARG;
    Attn a = {};
    size_t need = 0;
    const lf_status st = make_attn(c, q, &a, &need);
    if (st == LF_OK) *bytes = (int64_t)need;
    return st;
}

lf_status lf_paged_attend(const lf_paged *c, const lf_paged_query *q, void *workspace, int64_t workspace_bytes, void *stream)
{
    Attn a = {};
    size_t need = 0;
    lf_status st = make_attn(c, q, &a, &need);
    if (st != LF_OK || a.n == 0) return st;
    st = check_rows(&q->q, a.n, q->n_heads, c->head_dim, false);
    if (st == LF_OK) st = check_rows(&q->out, a.n, q->n_heads, c->head_dim, true);
    if (st != LF_OK) return st;
    if (q->q.dtype != q->out.dtype || q->q.data == q->out.data) return LF_ERR_INVALID_ARG;
    if (!aligned4(q->lens) || (a.width && !aligned4(q->tables))) return LF_ERR_INVALID_ARG;
    if (need && (!aligned16(workspace) || workspace_bytes < (int64_t)need)) return LF_ERR_INVALID_ARG;
    a.o = rows_of(&q->out);
    set_workspace(a, need ? workspace : nullptr);
    return status_of(launch_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
