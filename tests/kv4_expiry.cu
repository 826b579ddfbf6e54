// The attention of many rows with a hand-over withheld (lfq::Attn::fault), in launches that name no error record:
// each ends by its waits' limit, lf_kv4_status tells of it once, and the launch behind it is right.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <vector>

#include "../include/lf.h"
#include "../persistent_monokernel_gb300/csrc/lf_kv4.h"

using namespace lfq;

static int failures = 0;
static void expect(bool ok, const char *what, int hd, int dtype, int n)
{
    if (ok) return;
    std::printf("head_dim %d, type %d, %d rows: %s\n", hd, dtype, n, what);
    ++failures;
}

int main()
{
    const int Hkv = 2, Hq = 8, cap = 4600, pos = 1500;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, 0) != cudaSuccess) return 2;
    cudaStream_t side;
    if (cudaStreamCreate(&side) != cudaSuccess) return 2;
    for (int hd : {64, 128})
        for (int dtype : {F16, BF16, F32})
            for (int n : {600, 3000}) {
                const size_t rows = (size_t)Hkv * cap, es = dtype == F32 ? 4 : 2, bytes = (size_t)n * Hq * hd * es;
                std::vector<uint8_t> host(bytes);
                Cache c = {nullptr, nullptr, nullptr, nullptr, Hkv, hd, cap};
                void *q = nullptr, *o = nullptr, *ws = nullptr;
                Attn a = {};
                a.Hq = Hq;
                a.G = Hq / Hkv;
                a.n = n;
                a.pos = pos;
                a.len = pos + n;
                a.scale = 0.125f;
                a.wait_ns = 20000000;
                a.q.dtype = a.o.dtype = dtype;
                a.c = c;
                const size_t need = plan_attn(a, sms);
                expect(a.rt == 128, "another kernel", hd, dtype, n);
                bool ok = cudaMalloc((void **)&c.kc, rows * code_bytes(hd)) == cudaSuccess &&
                          cudaMalloc((void **)&c.vc, rows * code_bytes(hd)) == cudaSuccess &&
                          cudaMalloc((void **)&c.ks, rows * scale_bytes(hd)) == cudaSuccess &&
                          cudaMalloc((void **)&c.vs, rows * scale_bytes(hd)) == cudaSuccess && cudaMalloc(&q, bytes) == cudaSuccess &&
                          cudaMalloc(&o, bytes) == cudaSuccess && cudaMalloc(&ws, need + 16) == cudaSuccess;
                // K of 0.5 and -0.5, every value of V 1 (code 2, scale 1), q 0
                ok = ok && cudaMemset(c.kc, 0x91, rows * code_bytes(hd)) == cudaSuccess &&
                     cudaMemset(c.vc, 0x22, rows * code_bytes(hd)) == cudaSuccess &&
                     cudaMemset(c.ks, 0x38, rows * scale_bytes(hd)) == cudaSuccess &&
                     cudaMemset(c.vs, 0x38, rows * scale_bytes(hd)) == cudaSuccess && cudaMemset(q, 0, bytes) == cudaSuccess;
                if (!ok) return 2;
                a.c = c;
                a.q = {q, dtype, (long long)Hq * hd, hd, 0, nullptr};
                a.o = {o, dtype, (long long)Hq * hd, hd, 0, nullptr};
                set_workspace(a, need ? ws : nullptr);
                for (cudaStream_t s : {(cudaStream_t) nullptr, side}) {
                    if (cudaDeviceSynchronize() != cudaSuccess) return 2;
                    expect(lf_kv4_status(s) == LF_OK, "an error before", hd, dtype, n);
                    a.fault = 1;
                    expect(launch_attn(a, s) == cudaSuccess, "not launched", hd, dtype, n);
                    expect(lf_kv4_status(s) == LF_ERR_TIMEOUT, "the wait that ran out is not told of", hd, dtype, n);
                    expect(lf_kv4_status(s) == LF_OK, "told of twice", hd, dtype, n);
                    a.fault = 0;
                    expect(launch_attn(a, s) == cudaSuccess, "not launched again", hd, dtype, n);
                    expect(lf_kv4_status(s) == LF_OK, "an error behind", hd, dtype, n);
                    if (cudaMemcpy(host.data(), o, bytes, cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
                    // sums of equal powers of two are exact; 1 / l and its product are off by 2^-24 each
                    bool right = true;
                    for (size_t i = 0; i < bytes; i += es) {
                        uint16_t h = 0;
                        float f = 1.f;
                        if (dtype == F32) std::memcpy(&f, &host[i], es);
                        else std::memcpy(&h, &host[i], es);
                        right = right && (dtype == F32 ? std::fabs(f - 1.f) <= 0x1p-23f : h == (dtype == F16 ? 0x3c00 : 0x3f80));
                    }
                    expect(right, "the next launch is wrong", hd, dtype, n);
                }
                for (void *p : {(void *)c.kc, (void *)c.vc, (void *)c.ks, (void *)c.vs, q, o, ws}) cudaFree(p);
            }
    cudaStreamDestroy(side);
    std::printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
