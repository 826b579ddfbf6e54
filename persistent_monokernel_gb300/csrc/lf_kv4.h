// lf_kv4.h -- internal interface of the 4-bit KV cache operators (lf_kv4.cu):
// launches used by the C entry points and by the decoder's own 4-bit path.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lfq {

constexpr long long WAIT_NS = 2000000000LL;   // bound of a wait where the caller has named none
constexpr int PAD = 4;      // words of a partial row behind O: m, l, and two that keep rows 16-byte aligned

// Element types of the public calls, then those of the decoder's own buffers:
//   TAG32    FP32 with a tag in the lowest mantissa bit; read: FP16 values (whose own bit there is 0); written: the
//            value with Rows::aux there
//   SWZ16    read: FP16 rows whose 16-byte groups are XOR-ed with the position (Rows::aux: position of token 0) mod 8
//   SPLIT16  written: an FP16 head to p and remainder to p2
enum DType { F16 = 0, BF16 = 1, F32 = 2, TAG32 = 3, SWZ16 = 4, SPLIT16 = 5 };

// Bytes of one row of head_dim values: codes (two per byte) and scales (one per 16).
__host__ __device__ constexpr int code_bytes(int hd) { return hd / 2; }
__host__ __device__ constexpr int scale_bytes(int hd) { return hd / 16; }

// Cache of one layer: [Hkv][cap] rows of codes and of scales, for K and V.
struct Cache {
    uint8_t *kc, *ks, *vc, *vs;
    int Hkv, hd, cap;
};

// [n][heads][hd] values at element strides ts (token) and hs (head).
struct Rows {
    void *p;
    int dtype;
    long long ts, hs;
    int aux;
    void *p2;
};

struct Attn {
    Cache c;
    Rows q, o;
    int Hq, G;              // query heads; per KV head
    int gsh;                // log2 G, or -1 (set by the plan)
    int n, pos;             // query rows at positions pos .. pos + n - 1
    int len, win;           // keys 0 .. len - 1; window (0: all)
    float scale;
    // plan: row tiles of rt query rows (n * G rows per KV head, row r = token r / G, head r % G).
    // rt 8 or 16: each over `splits` ranges of `per` positions from lo on; `cl` ranges in a row are one cluster,
    // which joins them into one of splits / cl partial states.
    // rt 128: `splits` CTAs share all chunks of all tiles (share_tiles of `per` CTAs), or (per 0) take a tile each.
    int rt, tiles, splits, cl, per, lo;
    int sl;                 // rt 8 or 16: slabs of 16 positions that a warp takes at a time, 1 or 2
    // partial states [..][rt][hd + PAD]: O, then m and l (null: none).  rt 8 or 16: [Hkv * tiles * splits / cl];
    // rt 128: two per CTA, for the tile it goes on with and the tile it leaves unfinished, and where a tile's are:
    // pieces[Hkv * tiles] = (first CTA, number of pieces or 0).
    float *part;
    int2 *pieces;
    unsigned *status;       // [8]: error record [0..3] and abort word [4] of a handle; null: counted for the device
    long long wait_ns;      // bound of every wait of the tiles kernel
    int fault;              // test hook: the tiles kernel's products wait for a P that is never complete
};

// Keys that query row t (position pos + t) sees: [key_lo, key_hi).
__host__ __device__ inline int key_hi(int pos, int t, int len) { return pos + t + 1 < len ? pos + t + 1 : len; }
__host__ __device__ inline int key_lo(int pos, int t, int win)
{
    return (win > 0 && pos + t + 1 > win) ? pos + t + 1 - win : 0;
}

// Token of row x (of a KV head's n * G rows); a division costs 30 instructions, and G is mostly a power of two.
__host__ __device__ inline int row_token(const Attn &a, int x) { return a.gsh >= 0 ? x >> a.gsh : x / a.G; }
// Query head of row x of token t.
__host__ __device__ inline int row_head(const Attn &a, int kvh, int x, int t) { return kvh * a.G + x - t * a.G; }

// Chunks of 128 positions that some row of tile `tile` (of 128 rows) sees: their count, at least 1, and the first.
__host__ __device__ inline int tile_chunks(const Attn &a, int tile, int &first)
{
    const int r0 = tile * 128, last = r0 + 127 < a.n * a.G ? r0 + 127 : a.n * a.G - 1;
    const int lo = key_lo(a.pos, row_token(a, r0), a.win), hi = key_hi(a.pos, row_token(a, last), a.len);
    first = lo / 128;
    return hi > lo ? (hi + 127) / 128 - first : 1;
}
// Where CTA c of the tiles kernel begins: tile (KV head * tiles + tile), chunks and pieces of it that are earlier CTAs'.
struct Share {
    int tile, skip, piece;
};
constexpr int MAX_CTAS = 256;
struct Shares {
    Share at[MAX_CTAS + 1];
};
// Deals the chunks of all tiles out to at most `ctas` CTAs and returns how many have any.
int share_tiles(const Attn &a, int ctas, Shares &sh);

// Fills a's plan for `sms` SMs (a.q.dtype is set) and returns the workspace bytes it needs, at most
// max_workspace for blocks of up to n rows.
size_t plan_attn(Attn &a, int sms);
size_t max_workspace(const Cache &c, int Hq, int n, int sms);
// Points a at its workspace (null where the plan needs none).
void set_workspace(Attn &a, void *ws);

cudaError_t launch_append(const Cache &c, const Rows &k, const Rows &v, int n, int pos, cudaStream_t s);
cudaError_t launch_read(const Cache &c, const Rows &k, const Rows &v, int n, int pos, cudaStream_t s);
cudaError_t launch_attn(const Attn &a, cudaStream_t s);
// Tiles of 128 query rows on tcgen05 (lf_kv4_tc.cu); launch_attn calls it by the plan's rt.
cudaError_t launch_attn_tiles(const Attn &a, cudaStream_t s);
// Synchronises s; expired: whether a wait that is counted for the device ran out since this last said so.
cudaError_t tiles_status(bool &expired, cudaStream_t s);

}  // namespace lfq
