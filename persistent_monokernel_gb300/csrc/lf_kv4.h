// lf_kv4.h -- internal interface of the 4-bit KV cache operators (lf_kv4.cu):
// launches used by the C entry points and by the decoder's own 4-bit path.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lfq {

constexpr int PAD = 4;      // words of a partial row behind O: m, l, and two that keep rows 16-byte aligned

// Element types of the public calls, then those of the decoder's own buffers:
//   TAG32    FP32 with a tag in the lowest mantissa bit; read: FP16 values (the tag is rounded away); written: the
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
    int n, pos;             // query rows at positions pos .. pos + n - 1
    int len, win;           // keys 0 .. len - 1; window (0: all)
    float scale;
    // plan: row tiles of rt query rows (n * G rows per KV head, row r = token r / G, head r % G), each over
    // `splits` ranges of `per` positions from lo on; `cl` ranges in a row are one cluster, which joins them into
    // one of splits / cl partial states
    int rt, tiles, splits, cl, per, lo;
    float *part;            // [Hkv * tiles * splits / cl][rt][hd + PAD]: O, then m and l; null: one partial state
};

// Keys that query row t (position pos + t) sees: [key_lo, key_hi).
__host__ __device__ inline int key_hi(int pos, int t, int len) { return pos + t + 1 < len ? pos + t + 1 : len; }
__host__ __device__ inline int key_lo(int pos, int t, int win)
{
    return (win > 0 && pos + t + 1 > win) ? pos + t + 1 - win : 0;
}

// Fills a's plan for `sms` SMs (a.q.dtype is set) and returns the workspace floats it needs, at most `limit`
// (which is at least min_workspace).
size_t plan_attn(Attn &a, int sms, size_t limit = SIZE_MAX);
size_t min_workspace(const Cache &c, int sms);

cudaError_t launch_append(const Cache &c, const Rows &k, const Rows &v, int n, int pos, cudaStream_t s);
cudaError_t launch_read(const Cache &c, const Rows &k, const Rows &v, int n, int pos, cudaStream_t s);
cudaError_t launch_attn(const Attn &a, cudaStream_t s);
// Tiles of 128 query rows on tcgen05 (lf_kv4_tc.cu); launch_attn calls it by the plan's rt.
cudaError_t launch_attn_tiles(const Attn &a, cudaStream_t s);
// Error record of that kernel (out[0] = 0: none), read after synchronising s, and cleared.
cudaError_t tiles_status(unsigned out[4], cudaStream_t s);

}  // namespace lfq
