// lf_paged.h -- internal interface of the paged KV cache operators: the plan of
// a batch's pages and the append (lf_paged.cu), the attention (lf_paged_attn.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

// Fills a's choice of launch for `sms` SMs and returns the workspace it needs.
size_t plan_attn(Attn &a, int sms);
void set_workspace(Attn &a, void *ws);

cudaError_t launch_plan(const Plan &p, cudaStream_t s);
cudaError_t launch_append(const Pool &c, const Rows &k, const Rows &v, int n, const int *slots, cudaStream_t s);
cudaError_t launch_attn(const Attn &a, cudaStream_t s);

}  // namespace lfpg
