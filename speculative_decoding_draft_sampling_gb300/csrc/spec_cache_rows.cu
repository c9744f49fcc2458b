// spec_cache_rows.cu -- rows of the paged 4-bit cache: writing them
// (quantisation), reading them back, and keeping an accepted path's.
//
// [SD-survey] = "大模型投机解码：Medusa、MTP、EAGLE、DFlash、DDTree 与 DSpark"
// (Speculative decoding for LLMs: Medusa, MTP, EAGLE, DFlash, DDTree and
// DSpark), chzhyang.github.io, §5 "DDTree": only the accepted path's KV is kept.
//
// Quantisation of a group of 32 bf16 values x: scale s = rn5(max|x| / 7),
// where rn5 rounds to five significant bits, code = 8 + rn(x / s), both ties
// to even.  It is exact to the definition in real numbers although it works
// in fp32 and multiplies by 1/s: x has 8 significant bits and s five, so x/s
// is either exactly k + 1/2 or at least 2^-4/31 away from it, and the product
// x * (1/s) is off by at most 7.3 * 2^-22.  Rounding the product to a multiple
// of 2^-13 first (one fused multiply-add with 1.5 * 2^10) turns the exact ties
// back into ties and moves nothing else across a half.
#include <cuda_bf16.h>

#include "../../include/spec_cache.h"
#include "spec_cache.cuh"

namespace spec {

namespace {

constexpr int kRowThreads = 256;

// Eight bf16 of a row into registers, as four words.
template <bool kAligned>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
    if constexpr (kAligned) {
        return __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// five significant bits, ties to even; 0 below 2^-120
__device__ __forceinline__ float round5(float x) {
    uint32_t u = __float_as_uint(x);
    u = (u + 0x3FFFFu + ((u >> 19) & 1u)) & ~0x7FFFFu;
    return u < 0x03800000u ? 0.0f : __uint_as_float(u);
}

// code of x under a scale of reciprocal r
__device__ __forceinline__ uint32_t code_of(float x, float r) {
    const float t = __fadd_rn(__fmaf_rn(x, r, 1536.0f), -1536.0f);   // a multiple of 2^-13
    return __float_as_uint(__fadd_rn(t, 12582912.0f + 8.0f)) & 15u;
}

// Quantises a thread's eight values (four neighbouring lanes share a group, the
// whole warp takes part).  Returns the eight codes, the scale's bf16 bits, and
// reports a value that is not finite.
__device__ __forceinline__ uint32_t quantise8(uint4 x, uint32_t& scale, bool& bad) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                          __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (__any_sync(0xffffffffu, m >= 0x7f80u)) {
        // a NaN or an infinity in the warp: the maximum is over finite values,
        // NaN becomes 0 and an infinity the largest code
        uint32_t f = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
            if (h < 0x7f80u) f = max(f, h);
        }
        f = max(f, __shfl_xor_sync(0xffffffffu, f, 1));
        f = max(f, __shfl_xor_sync(0xffffffffu, f, 2));
        if (m >= 0x7f80u) {
            bad = true;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int sh = 16 * (i & 1);
                const uint32_t h = (w[i >> 1] >> sh) & 0xffffu;
                uint32_t g = h;
                if ((h & 0x7fffu) > 0x7f80u) g = 0;
                else if ((h & 0x7fffu) == 0x7f80u) g = (h & 0x8000u) | f;
                w[i >> 1] = (w[i >> 1] & ~(0xffffu << sh)) | (g << sh);
            }
            m = f;
        }
    }
    const float s = round5(__fdiv_rn(__uint_as_float(m << 16), 7.0f));
    scale = __float_as_uint(s) >> 16;
    const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        out |= code_of(__uint_as_float(w[i] << 16), r) << (8 * i);
        out |= code_of(__uint_as_float(w[i] & 0xffff0000u), r) << (8 * i + 4);
    }
    return out;
}

// D/8 threads quantise a row; rows go K heads, V heads of a token, token by
// token.  Every thread of a warp takes part in the shuffles, live or not.
template <int D, bool kAligned>
__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const CacheRowsArgs A) {
    constexpr int kT = D / 8;                               // threads a row
    const int H = A.pool.heads;
    const long long item = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) / kT;
    const int c = threadIdx.x % kT;
    const long long tok = item / (2 * H);                   // b * n + i
    const int hk = static_cast<int>(item % (2 * H));
    const bool isv = hk >= H;
    const int h = isv ? hk - H : hk;
    const int b = static_cast<int>(tok / A.n), i = static_cast<int>(tok % A.n);
    const bool live = b < A.B && i < (A.count ? A.count[b] : A.n);
    uint4 x = make_uint4(0, 0, 0, 0);
    int page = -1;
    long long pos = 0;
    if (live) {
        pos = static_cast<long long>(A.start[b]) + i;
        page = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, pos);
        const uint16_t* src = isv ? A.v + b * A.v_bs + i * A.v_rs + h * A.v_hs
                                  : A.k + b * A.k_bs + i * A.k_rs + h * A.k_hs;
        x = load8<kAligned>(src + c * 8);
    }
    bool bad = false;
    uint32_t scale;
    const uint32_t codes = quantise8(x, scale, bad);
    if (!live) return;
    if (A.status && (bad || page < 0))
        atomicOr(A.status + b, (bad ? SPEC_ST_BAD_ROW : 0) | (page < 0 ? SPEC_ST_BAD_PAGE : 0));
    if (page < 0) return;
    const int P = A.pool.P, slot = static_cast<int>(pos & (P - 1));
    unsigned char* blk = A.pool.base + page * A.pool.page_stride + h * A.pool.head_stride +
                         (isv ? CacheBlock<D>::v_codes(P) : 0);
    reinterpret_cast<uint32_t*>(blk + slot * CacheBlock<D>::kRow)[c] = codes;
    if ((c & 3) == 0)
        reinterpret_cast<uint16_t*>(blk + P * CacheBlock<D>::kRow + slot * CacheBlock<D>::kScl)[c >> 2] =
            static_cast<uint16_t>(scale);
}

// (code - 8) * scale of two neighbouring codes, as bf16 bits
__device__ __forceinline__ uint32_t values2(uint32_t two, float s) {
    const float lo = (static_cast<float>(two & 15u) - 8.0f) * s;
    const float hi = (static_cast<float>((two >> 4) & 15u) - 8.0f) * s;
    return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const CacheRowsArgs A) {
    constexpr int kT = D / 8;
    const int H = A.pool.heads;
    const long long item = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) / kT;
    const int c = threadIdx.x % kT;
    const long long tok = item / (2 * H);
    const int hk = static_cast<int>(item % (2 * H));
    const bool isv = hk >= H;
    const int h = isv ? hk - H : hk;
    const int b = static_cast<int>(tok / A.n), i = static_cast<int>(tok % A.n);
    if (b >= A.B) return;
    uint4 out = make_uint4(0, 0, 0, 0);
    if (i < (A.count ? A.count[b] : A.n)) {
        const long long pos = static_cast<long long>(A.start[b]) + i;
        const int page = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, pos);
        if (page >= 0) {
            const int P = A.pool.P, slot = static_cast<int>(pos & (P - 1));
            const unsigned char* blk = A.pool.base + page * A.pool.page_stride + h * A.pool.head_stride +
                                       (isv ? CacheBlock<D>::v_codes(P) : 0);
            const uint32_t w = reinterpret_cast<const uint32_t*>(blk + slot * CacheBlock<D>::kRow)[c];
            const uint32_t sb = reinterpret_cast<const uint16_t*>(blk + P * CacheBlock<D>::kRow +
                                                                  slot * CacheBlock<D>::kScl)[c >> 2];
            const float s = __uint_as_float(sb << 16);
            out = make_uint4(values2(w, s), values2(w >> 8, s), values2(w >> 16, s), values2(w >> 24, s));
        } else if (A.status) {
            atomicOr(A.status + b, SPEC_ST_BAD_PAGE);
        }
    }
    uint16_t* dst = (isv ? A.v_out : A.k_out) + ((tok * H) + h) * D + c * 8;
    __stcs(reinterpret_cast<uint4*>(dst), out);
}

cudaError_t row_grid(const CacheRowsArgs& A, int D, dim3& grid) {
    const long long threads = static_cast<long long>(A.B) * A.n * A.pool.heads * 2 * (D / 8);
    const long long blocks = (threads + kRowThreads - 1) / kRowThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    grid = dim3(static_cast<unsigned>(blocks));
    return cudaSuccess;
}

}  // namespace

cudaError_t cache_append_run(const CacheRowsArgs& A, cudaStream_t st) {
    dim3 grid;
    const cudaError_t e = row_grid(A, A.pool.D, grid);
    if (e != cudaSuccess) return e;
    if (A.pool.D == 128) {
        if (A.aligned) cache_append_kernel<128, true><<<grid, kRowThreads, 0, st>>>(A);
        else cache_append_kernel<128, false><<<grid, kRowThreads, 0, st>>>(A);
    } else {
        if (A.aligned) cache_append_kernel<64, true><<<grid, kRowThreads, 0, st>>>(A);
        else cache_append_kernel<64, false><<<grid, kRowThreads, 0, st>>>(A);
    }
    return cudaGetLastError();
}

cudaError_t cache_read_run(const CacheRowsArgs& A, cudaStream_t st) {
    dim3 grid;
    const cudaError_t e = row_grid(A, A.pool.D, grid);
    if (e != cudaSuccess) return e;
    if (A.pool.D == 128) cache_read_kernel<128><<<grid, kRowThreads, 0, st>>>(A);
    else cache_read_kernel<64><<<grid, kRowThreads, 0, st>>>(A);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// accepted-path compaction, in place
// ---------------------------------------------------------------------------
namespace {

constexpr int kCompactThreads = 256;
constexpr int kCompactBatch = 8;                // rows whose loads are in flight together

// A CTA takes a range of (layer, head) pairs of one request; a thread owns one
// piece of a row (16 bytes of codes, or one of the scale runs) and moves it
// along the whole path.  The path ascends, so a row is only ever overwritten
// by a later row of the path: with each batch's loads before its stores, and
// batches in order, the copy is right in place, and threads never meet.
template <int D>
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const CacheCompactArgs A, int pairs_per_cta) {
    extern __shared__ int2 moves[];             // (page * P + slot) from, to
    __shared__ int count;
    using Blk = CacheBlock<D>;
    constexpr int kCode = Blk::kRow / 16;       // 16-byte pieces of a row's codes
    constexpr int kPieces = 2 * (kCode + 1);
    const int b = blockIdx.y, P = A.pool.P;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const long long ctx = A.ctx[b];
    int last = A.accepted[b];
    if (last >= A.path_width) last = A.path_width - 1;
    // the moves, in path order (one warp; a path has few entries)
    if (threadIdx.x < 32) {
        int bits = 0, base = 0;
        for (int j0 = 0; j0 <= last; j0 += 32) {
            const int j = j0 + static_cast<int>(threadIdx.x);
            bool move = false;
            int2 m = make_int2(0, 0);
            if (j <= last) {
                const int node = A.path[static_cast<long long>(b) * A.path_width + j];
                if (node < j) {
                    bits |= SPEC_ST_BAD_NODE;
                } else if (node > j) {
                    const int fp = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, ctx + node);
                    const int tp = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, ctx + j);
                    move = fp >= 0 && tp >= 0;
                    if (!move) bits |= SPEC_ST_BAD_PAGE;
                    m = make_int2(fp * P + static_cast<int>((ctx + node) & (P - 1)),
                                  tp * P + static_cast<int>((ctx + j) & (P - 1)));
                }
            }
            const unsigned who = __ballot_sync(0xffffffffu, move);
            if (move) moves[base + __popc(who & ((1u << threadIdx.x) - 1u))] = m;
            base += __popc(who);
        }
        if (bits && A.status && blockIdx.x == 0) atomicOr(A.status + b, bits);
        if (threadIdx.x == 0) count = base;
    }
    __syncthreads();
    const int n = count;
    if (n == 0) return;
    const int pairs = A.pool.layers * A.pool.heads;
    const int first = blockIdx.x * pairs_per_cta;
    const int mine = min(pairs_per_cta, pairs - first) * kPieces;
    for (int w = threadIdx.x; w < mine; w += kCompactThreads) {
        const int pair = first + w / kPieces, piece = w % kPieces;
        const int layer = pair / A.pool.heads, head = pair % A.pool.heads;
        const int half = piece % (kCode + 1);
        // where the piece lies: its offset in a block and the row pitch
        const int sec = (piece > kCode ? Blk::v_codes(P) : 0) + (half < kCode ? half * 16 : P * Blk::kRow);
        const int pitch = half < kCode ? Blk::kRow : Blk::kScl;
        unsigned char* base = A.pool.base + layer * A.pool.layer_stride + head * A.pool.head_stride + sec;
        auto at = [&](int row) {
            return base + (row >> A.pool.p_shift) * A.pool.page_stride + (row & (P - 1)) * pitch;
        };
        for (int j0 = 0; j0 < n; j0 += kCompactBatch) {
            uint4 r[kCompactBatch];
#pragma unroll
            for (int q = 0; q < kCompactBatch; ++q) {
                if (j0 + q >= n) break;
                const unsigned char* p = at(moves[j0 + q].x);
                if (half < kCode) r[q] = *reinterpret_cast<const uint4*>(p);
                else if constexpr (Blk::kScl == 8) {
                    const uint2 t = *reinterpret_cast<const uint2*>(p);
                    r[q].x = t.x; r[q].y = t.y;
                } else r[q].x = *reinterpret_cast<const uint32_t*>(p);
            }
#pragma unroll
            for (int q = 0; q < kCompactBatch; ++q) {
                if (j0 + q >= n) break;
                unsigned char* p = at(moves[j0 + q].y);
                if (half < kCode) *reinterpret_cast<uint4*>(p) = r[q];
                else if constexpr (Blk::kScl == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r[q].x, r[q].y);
                else *reinterpret_cast<uint32_t*>(p) = r[q].x;
            }
        }
    }
}

}  // namespace

cudaError_t cache_compact_run(const CacheCompactArgs& A, cudaStream_t st) {
    const int pairs = A.pool.layers * A.pool.heads;
    const int kPieces = A.pool.D == 128 ? 10 : 6;
    // a few passes a thread at most, and no more CTAs than pairs fill
    const int per = max(1, kCompactThreads / kPieces);
    const dim3 grid(static_cast<unsigned>((pairs + per - 1) / per), static_cast<unsigned>(A.B));
    const size_t smem = static_cast<size_t>(A.path_width) * sizeof(int2);
    if (A.pool.D == 128) cache_compact_kernel<128><<<grid, kCompactThreads, smem, st>>>(A, per);
    else cache_compact_kernel<64><<<grid, kCompactThreads, smem, st>>>(A, per);
    return cudaGetLastError();
}

}  // namespace spec
