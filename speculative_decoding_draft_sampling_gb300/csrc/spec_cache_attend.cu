// spec_cache_attend.cu -- attention of drafted rows over the paged 4-bit cache.
//
// [SD-survey] = "大模型投机解码：Medusa、MTP、EAGLE、DFlash、DDTree 与 DSpark"
// (Speculative decoding for LLMs: Medusa, MTP, EAGLE, DFlash, DDTree and
// DSpark), chzhyang.github.io, §5 "DDTree": drafted nodes take position id =
// depth and see only their ancestors.
//
// One warp per (request, row, q head) walks the keys one at a time with a
// running maximum and sum (all fp32): m' = max(m, x), l' = l e^(m-m') +
// e^(x-m'), o' = o e^(m-m') + e^(x-m') v.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "../../include/spec_cache.h"
#include "spec_cache.cuh"

namespace spec {

namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) cache_attend_kernel(const CacheAttendArgs A) {
    using Blk = CacheBlock<D>;
    constexpr int kE = D / 32;                  // values a lane
    const int lane = threadIdx.x & 31;
    const long long unit = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int h = static_cast<int>(unit % A.hq);
    const int i = static_cast<int>(unit / A.hq % A.n);
    const int b = static_cast<int>(unit / A.hq / A.n);
    if (b >= A.B) return;
    const int P = A.pool.P;
    const long long room = static_cast<long long>(A.tab.width) * P;
    const int ctx = static_cast<int>(min(static_cast<long long>(max(A.ctx[b], 0)), room));
    const int rows = A.rows ? min(max(A.rows[b], 0), A.n) : A.n;
    float q[kE], o[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        q[e] = __uint_as_float(static_cast<uint32_t>(A.q[b * A.q_bs + i * A.q_rs + h * A.q_hs + lane * kE + e]) << 16);
        o[e] = 0.0f;
    }
    float m = -CUDART_INF_F, l = 0.0f;
    int bits = 0;
    if (i < rows) {
        const int W = (A.n + 63) / 64;
        const int* depth = A.depth ? A.depth + static_cast<long long>(b) * A.n : nullptr;
        const long long pos = static_cast<long long>(ctx) + (depth ? depth[i] : i);
        const unsigned char* head = A.pool.base + (h / A.G) * A.pool.head_stride;
        for (int t = 0; t < ctx + rows; ++t) {
            long long key = t;
            const int j = t - ctx;
            if (j >= 0) {
                const bool seen = A.mask ? (A.mask[(static_cast<long long>(b) * A.n + i) * W + (j >> 6)] >> (j & 63)) & 1
                                         : j <= i;
                if (!seen) continue;
                key = static_cast<long long>(ctx) + (depth ? depth[j] : j);
            }
            if (A.window > 0 && pos - key >= A.window && key >= A.sinks) continue;
            const int page = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, t);
            if (page < 0) { bits |= SPEC_ST_BAD_PAGE; continue; }
            const int slot = t & (P - 1);
            const unsigned char* blk = head + page * A.pool.page_stride;
            float kv[2][kE];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const unsigned char* x = blk + (s ? Blk::v_codes(P) : 0);
                const float scl = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(
                    x + P * Blk::kRow + slot * Blk::kScl)[lane * kE / kCacheGroup]) << 16);
#pragma unroll
                for (int e = 0; e < kE; e += 2) {
                    const uint32_t c = x[slot * Blk::kRow + (lane * kE + e) / 2];
                    kv[s][e] = (static_cast<float>(c & 15u) - 8.0f) * scl;
                    kv[s][e + 1] = (static_cast<float>(c >> 4) - 8.0f) * scl;
                }
            }
            float x = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) x = fmaf(q[e], kv[0][e], x);
#pragma unroll
            for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
            x *= A.scale;
            const float mn = fmaxf(m, x);
            const float f = m == -CUDART_INF_F ? 0.0f : __expf(m - mn), p = __expf(x - mn);
            m = mn;
            l = fmaf(l, f, p);
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = fmaf(o[e], f, p * kv[1][e]);
        }
    }
    const long long row = (static_cast<long long>(b) * A.n + i) * A.hq + h;
    const bool none = l == 0.0f;                // NaN scores are not "nothing seen"
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        A.out[row * D + lane * kE + e] = __bfloat16_as_ushort(__float2bfloat16_rn(none ? 0.0f : o[e] / l));
    }
    if (lane == 0) {
        if (A.lse) A.lse[row] = none ? -CUDART_INF_F : m + logf(l);
        if (bits && A.status) atomicOr(A.status + b, bits);
    }
}

}  // namespace

size_t cache_attend_ws(int, int, int, int, int) { return 0; }

cudaError_t cache_attend_run(const CacheAttendArgs& A, cudaStream_t st) {
    const long long blocks = (static_cast<long long>(A.B) * A.n * A.hq + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (A.pool.D == 128) cache_attend_kernel<128><<<grid, kThreads, 0, st>>>(A);
    else cache_attend_kernel<64><<<grid, kThreads, 0, st>>>(A);
    return cudaGetLastError();
}

}  // namespace spec
