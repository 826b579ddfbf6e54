// lf_paged.h -- internal interface of the paged KV cache operators: the plan of
// a batch's pages and the append (lf_paged.cu), the attention (lf_paged_attn.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace lfpg {

constexpr int MAX_ROWS = 8192;   // rows of a plan: it keeps four numbers per row in shared memory

// Page tables of a batch (lf_page_tables) and one plan's arguments.
struct Plan {
    int *tables;            // [n][max_pages] at element stride tstride
    long long tstride;
    int *lens, *free, *n_free, *status;
    int n, max_pages, n_pages, page;
    const int *n_new, *keep;   // keep: null keeps everything
    int *slots, *positions, *offsets;
    int max_tokens;
};

// K and V pools: byte offsets of page, head and position; V lies at `v`.
struct Pool {
    char *k, *v;
    long long page_b, head_b, pos_b;
    int n_pages, page, Hkv, hd;
    int bf16;               // values are BF16, not FP16
};

// [n][heads][hd] values at element strides ts (token) and hs (head).
struct Rows {
    void *p;
    int dtype;              // LF_F16, LF_BF16, LF_F32
    long long ts, hs;
};

struct Attn {
    Pool c;
    Rows q, o;
    const int *tables;
    long long tstride;
    const int *lens;
    int width;              // table columns
    int n, G;               // sequences; query heads per KV head
    int tiles, ht;          // tiles of rt query heads per KV head; KV heads x tiles
    int rt;                 // 8 or 16
    int win;
    float scale;
    // launch: `parts` clusters of `cl` CTAs of `cw` warps (4 or 8) for each sequence and tile
    int cl, cw, parts;
    int sorted;             // the clusters take long sequences first (parts 1)
    float *part;            // [n * ht][parts] partial states of rt * (hd + 4) floats (parts > 1)
};

constexpr int PADF = 4;           // floats behind a partial state's O per row: m, l, and two that keep rows aligned

// The lengths are known on the device alone, so the launch goes by what the host knows: the items (sequences x tiles)
// and the slabs that the widest row may have (of 8 KB: narrow heads' count half).  Two CTAs of four warps fit an SM (304
// places on 152).
//   * Clusters as large as the items leave places for, with two slabs a warp at least (16 x 5 heads of up to 512 positions:
//     6.7 us in clusters of two, 7.0 in fours, 8.2 in eights, of which most have to wait for places).
//   * More items than places: long ones first, which costs each CTA half a microsecond (up to 256 rows, where one has
//     2,048 positions or more).  Clusters then only up to three rounds of items, and only where a warp still has 40 slabs
//     of a row: 64 x 8 heads of up to 16,384 positions take 296 us in twos (310 in single CTAs, 302 in fours, 315 in row
//     order), of 4,096 81 in single CTAs (87 in twos); 200 x 2 heads of 16 FP32 queries each, skewed to 20,000,
//     160 in fours (196 in twos, 344 in single CTAs, 206 in eights, 191 in row order).
//   * The same of more than 256 rows, in row order: clusters while all their CTAs come in eight rounds.  Where the table is
//     far wider than its rows they are rounds of CTAs that have nothing to do (257 x 8 heads of up to 1,000 positions
//     in a table for 16,384: 81 us in single CTAs, 149 in fours, 224 in eights), and of long rows larger clusters would
//     gain less (1,000 x 8 heads skewed to 16,000: 1,775 us in single CTAs, 1,767 in twos; 257 x 2 heads skewed to 60,000:
//     491 us in fours, 474 in eights, 707 in single CTAs).
//   * Fewer items whose clusters need rounds: as large as leaves 8 cl slabs a warp (16 x 8 heads skewed to 32,768:
//     223 us in single CTAs, 91 in fours, 80 in eights), long ones first from 4,096 positions on (48 x 5 heads of up to
//     4,096: 41.9 us, 45.3 in row order).
//   * Few items of many slabs leave SMs idle in one cluster each: up to 23 items of 12,288 positions or more are cut into
//     parts, as many clusters of four as fit (280 CTAs: the last clusters find no group of SMs that is free), and a second
//     launch joins them (3 us; one sequence of 5 heads at 32,768: 20.4 us in parts, 24.5 in clusters of eight CTAs of
//     eight warps; of 8 heads at 131,071: 81 and 91).
//   * Otherwise, where clusters of eight leave half the places empty, CTAs of eight warps (5 heads at 8,192: 10.1 us,
//     11.2 with four; at 2,048 6.4 either way).
//
// Fills a's choice of launch for `sms` SMs and returns the workspace it needs.
inline size_t plan_attn(Attn &a, int sms)
{
    a.rt = a.G <= 8 ? 8 : 16;
    a.tiles = (a.G + a.rt - 1) / a.rt;
    a.ht = a.c.Hkv * a.tiles;
    const long long items = (long long)a.n * a.ht, places = 2 * sms;
    long long slabs = ((long long)a.width * a.c.page + 15) / 16;
    if (a.win > 0) slabs = std::min<long long>(slabs, a.win / 16 + 2);
    a.cl = 1, a.cw = 4, a.parts = 1;
    const long long wide = slabs * a.c.hd / 128;
    const bool many = items > places, can_sort = a.n > 1 && a.n <= 256;
    a.sorted = many && can_sort && wide >= 128;
    for (int cl = 2; cl <= 8; cl *= 2) {
        const bool few_rounds = !many || (a.sorted ? items * cl < 6 * places : items * cl <= 8 * places);
        const bool long_rows = wide >= (a.sorted ? 160 * cl : 32 * cl * cl);
        if (slabs >= 8 * cl && (items * cl <= places || (few_rounds && long_rows))) a.cl = cl;
    }
    const long long parts = places * 280 / 304 / (4 * items);
    if (slabs >= 768 && parts >= 3) {
        a.cl = 4;
        a.parts = (int)parts;
    } else if (a.cl == 8 && items * 8 <= sms && slabs >= 256) {
        a.cw = 8;
    }
    if (a.parts == 1 && items * a.cl > places && wide >= 256 && can_sort) a.sorted = 1;
    return a.parts > 1 ? (size_t)items * a.parts * a.rt * (a.c.hd + PADF) * sizeof(float) : 0;
}

void set_workspace(Attn &a, void *ws);

cudaError_t launch_plan(const Plan &p, cudaStream_t s);
cudaError_t launch_append(const Pool &c, const Rows &k, const Rows &v, int n, const int *slots, cudaStream_t s);
cudaError_t launch_attn(const Attn &a, cudaStream_t s);

}  // namespace lfpg
