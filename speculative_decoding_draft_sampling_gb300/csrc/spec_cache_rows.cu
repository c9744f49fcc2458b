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
// in fp32 and multiplies by 1/7 and 1/s: x has 8 significant bits and s five,
// so x/s is either exactly k + 1/2 or at least 2^-4/31 away from it, and the
// product x * (1/s) is off by less than 2^-18.  Rounding the product to a
// multiple of 2^-13 first (one fused multiply-add with 1.5 * 2^10) turns the
// exact ties back into ties and moves nothing else across a half; one more add
// rounds to the integer.  Likewise max|x| / 7 is a five-bit tie or at least
// 1/(7 * 64) of it away from one, and is rounded to 13 bits first.
//
// Append and read move 4 bytes of codes or 16 of values a thread with four heads
// in flight.  8 prompts of 8192 tokens each, 8 heads of 128 (268 MB of bf16, 75 MB of
// cache), take 62 us to append (5.6 TB/s) and 54 to read (6.3).  Reading is bound by
// HBM; writing by its instructions as well (four fifths of the issue slots), so its
// products come in pairs and its addresses by steps (4 us).  Eight heads in
// flight cost 8 % more, two 3 %; registers cut for more warps an SM cost 8 % too.
#include <cuda_bf16.h>

#include "../../include/spec_cache.h"
#include "spec_cache.cuh"

namespace spec {

namespace {

// Append, then read of 8 prompts of 8192 to 4608 tokens (of 8192 rows given): 101 us at
// 128 threads; at 64 the same, at 256 4 more, at 512 10.
constexpr int kRowThreads = 128;

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

// max|x| / 7 to five significant bits, ties to even; 0 below 2^-120
__device__ __forceinline__ float scale_of(float top) {
    uint32_t u = __float_as_uint(__fmul_rn(top, 1.0f / 7.0f));
    u = (u + 0x400u) & ~0x7FFu;                             // 13 bits: what 1/7 lost
    u = (u + 0x3FFFFu + ((u >> 19) & 1u)) & ~0x7FFFFu;
    return u < 0x03800000u ? 0.0f : __uint_as_float(u);
}

// Two neighbours' codes under a scale of reciprocal r, in the low byte: each result
// is an integer whose low four bits are a code.
__device__ __forceinline__ uint32_t codes_of(uint32_t w, float r) {
    unsigned long long y;
    asm("{\n\t.reg .b64 x, a, c;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 a, {%3, %3};\n\tmov.b64 c, {%4, %4};\n\t"
        "fma.rn.f32x2 x, x, a, c;\n\tmov.b64 c, {%5, %5};\n\tadd.rn.f32x2 %0, x, c;\n\t}"
        : "=l"(y)
        : "f"(__uint_as_float(w << 16)), "f"(__uint_as_float(w & 0xffff0000u)), "f"(r), "f"(1536.0f),
          "f"(12582912.0f + 8.0f - 1536.0f));
    return static_cast<uint32_t>(y >> 32) * 16u + static_cast<uint32_t>(y);
}

// Quantises a thread's eight values (four neighbouring lanes share a group, the
// whole warp takes part).  Returns the eight codes, the scale's bf16 bits, and
// reports a value that is not finite.
__device__ __forceinline__ uint32_t quantise8(uint4 x, uint32_t& scale, bool& bad) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                          __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m & 0xffffu, m >> 16);
    if (__any_sync(0xffffffffu, m >= 0x7f80u)) {
        // a NaN or an infinity in the warp: the maximum is over finite values,
        // NaN becomes 0 and an infinity the largest code
        uint32_t f = 0;
        bool mine = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
            if (h < 0x7f80u) f = max(f, h);
            else mine = true;
        }
        f = max(f, __shfl_xor_sync(0xffffffffu, f, 1));
        f = max(f, __shfl_xor_sync(0xffffffffu, f, 2));
        bad |= mine;
        if (m >= 0x7f80u) {
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
    const float s = scale_of(__uint_as_float(m << 16));
    scale = __float_as_uint(s) >> 16;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    if (s == 0.0f) r = 0.0f;
    uint32_t two[4];                                        // low byte: the codes of two neighbours
#pragma unroll
    for (int i = 0; i < 4; ++i) two[i] = codes_of(w[i], r);
    return __byte_perm(__byte_perm(two[0], two[1], 0x0040), __byte_perm(two[2], two[3], 0x0040), 0x5410);
}

// How the rows are dealt out: blockIdx.x takes 4 (D = 128) or 8 tokens,
// blockIdx.y a request, blockIdx.z a range of heads; D/8 threads take K or V of
// one token and go through the heads, four at a time.
template <int D>
struct RowPlace {
    static constexpr int kT = D / 8;                        // threads a row
    static constexpr int kTokens = kRowThreads / kT / 2;
    int i, c;
    bool isv;
    __device__ __forceinline__ RowPlace() {
        const int group = threadIdx.x / kT;
        c = threadIdx.x % kT;
        isv = group & 1;
        i = blockIdx.x * kTokens + group / 2;
    }
};

constexpr int kFly = 4;                                     // heads in flight

// Every thread of a warp takes part in the shuffles, live or not.
template <int D, bool kAligned>
__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const CacheRowsArgs A, int heads_per) {
    after_earlier();
    using Blk = CacheBlock<D>;
    const RowPlace<D> at;
    const int c = at.c, P = A.pool.P;
    const int h0 = blockIdx.z * heads_per, h1 = min(h0 + heads_per, A.pool.heads);
    for (int b = blockIdx.y; b < A.B; b += gridDim.y) {
        const bool live = at.i < (A.count ? min(A.count[b], A.n) : A.n);
        int page = -1;
        long long pos = 0;
        if (live) {
            pos = static_cast<long long>(A.start[b]) + at.i;
            page = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, pos);
        }
        const long long hs = at.isv ? A.v_hs : A.k_hs;
        const uint16_t* src = (at.isv ? A.v + b * A.v_bs + at.i * A.v_rs : A.k + b * A.k_bs + at.i * A.k_rs) + h0 * hs + c * 8;
        const int slot = static_cast<int>(pos & (P - 1));
        // this thread's codes and, P rows of codes on, its row's scales
        unsigned char* to = A.pool.base + page * A.pool.page_stride + h0 * A.pool.head_stride + (at.isv ? Blk::v_codes(P) : 0);
        unsigned char* to_s = to + P * Blk::kRow + slot * Blk::kScl + (c >> 2) * 2;
        to += slot * Blk::kRow + c * 4;
        bool bad = false;
        for (int h = h0; h < h1; h += kFly, src += kFly * hs, to += kFly * A.pool.head_stride, to_s += kFly * A.pool.head_stride) {
            uint4 x[kFly];
#pragma unroll
            for (int q = 0; q < kFly; ++q) {
                x[q] = make_uint4(0, 0, 0, 0);
                if (live && h + q < h1) x[q] = load8<kAligned>(src + q * hs);
            }
#pragma unroll
            for (int q = 0; q < kFly; ++q) {
                if (h + q >= h1) break;
                uint32_t scale;
                const uint32_t codes = quantise8(x[q], scale, bad);
                if (page >= 0) {
                    *reinterpret_cast<uint32_t*>(to + q * A.pool.head_stride) = codes;
                    if ((c & 3) == 0)
                        *reinterpret_cast<uint16_t*>(to_s + q * A.pool.head_stride) = static_cast<uint16_t>(scale);
                }
            }
        }
        if (A.status && live && (bad || page < 0))
            atomicOr(A.status + b, (bad ? SPEC_ST_BAD_ROW : 0) | (page < 0 ? SPEC_ST_BAD_PAGE : 0));
    }
}

// Eight codes under scale s as bf16, in order: two codes 16 bits apart become
// 1 + code/16, then (code - 8)/16 * s by one exact fused multiply-add with
// (s, -1.5 s), and 16 times that (16 s itself may be out of range).
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t s2, uint32_t c2) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t t = ((i == 0 ? w << 3 : w >> (4 * i - 3)) & 0x00780078u) | 0x3F803F80u;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(t), "r"(s2), "r"(c2));
        asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(0x41804180u));
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const CacheRowsArgs A, int heads_per) {
    after_earlier();
    using Blk = CacheBlock<D>;
    const RowPlace<D> at;
    const int c = at.c, P = A.pool.P, H = A.pool.heads;
    const int h0 = blockIdx.z * heads_per, h1 = min(h0 + heads_per, H);
    if (at.i >= A.n) return;
    for (int b = blockIdx.y; b < A.B; b += gridDim.y) {
        const bool live = at.i < (A.count ? A.count[b] : A.n);
        int page = -1;
        long long pos = 0;
        if (live) {
            pos = static_cast<long long>(A.start[b]) + at.i;
            page = cache_page(A.tab, A.pool.num_pages, A.pool.p_shift, b, pos);
            if (page < 0 && A.status) atomicOr(A.status + b, SPEC_ST_BAD_PAGE);
        }
        const int slot = static_cast<int>(pos & (P - 1));
        const unsigned char* blk = A.pool.base + page * A.pool.page_stride + (at.isv ? Blk::v_codes(P) : 0);
        uint16_t* dst = (at.isv ? A.v_out : A.k_out) + (static_cast<long long>(b) * A.n + at.i) * H * D + c * 8;
        for (int h = h0; h < h1; h += kFly) {
            uint32_t w[kFly], s[kFly];
#pragma unroll
            for (int q = 0; q < kFly; ++q) {
                w[q] = 0x88888888u;
                s[q] = 0;
                if (page >= 0 && h + q < h1) {
                    const unsigned char* from = blk + (h + q) * A.pool.head_stride;
                    w[q] = reinterpret_cast<const uint32_t*>(from + slot * Blk::kRow)[c];
                    s[q] = reinterpret_cast<const uint16_t*>(from + P * Blk::kRow + slot * Blk::kScl)[c >> 2];
                }
            }
#pragma unroll
            for (int q = 0; q < kFly; ++q) {
                if (h + q >= h1) break;
                const uint32_t s2 = s[q] * 0x10001u;
                uint32_t c2;
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(c2) : "r"(s2), "r"(0xBFC0BFC0u));
                __stcs(reinterpret_cast<uint4*>(dst + static_cast<long long>(h + q) * D), values8(w[q], s2, c2));
            }
        }
    }
}

// Heads are split over blockIdx.z where there are few rows: a step's rows then
// cost one round of loads instead of H / 4.
template <int D>
dim3 row_grid(const CacheRowsArgs& A, int& heads_per) {
    const int x = (A.n + RowPlace<D>::kTokens - 1) / RowPlace<D>::kTokens, y = A.B < 65535 ? A.B : 65535;
    const long long blocks = static_cast<long long>(x) * y;
    heads_per = A.pool.heads;
    if (blocks < 1216 && heads_per > kFly) heads_per = kFly;
    const int z = (A.pool.heads + heads_per - 1) / heads_per;
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y), static_cast<unsigned>(z));
}

}  // namespace

cudaError_t cache_append_run(const CacheRowsArgs& A, cudaStream_t st) {
    int per;
    if (A.pool.D == 128) {
        const dim3 grid = row_grid<128>(A, per);
        if (A.aligned) return launch_early(cache_append_kernel<128, true>, grid, kRowThreads, 0, st, A, per);
        else return launch_early(cache_append_kernel<128, false>, grid, kRowThreads, 0, st, A, per);
    } else {
        const dim3 grid = row_grid<64>(A, per);
        if (A.aligned) return launch_early(cache_append_kernel<64, true>, grid, kRowThreads, 0, st, A, per);
        else return launch_early(cache_append_kernel<64, false>, grid, kRowThreads, 0, st, A, per);
    }
}

cudaError_t cache_read_run(const CacheRowsArgs& A, cudaStream_t st) {
    int per;
    if (A.pool.D == 128) {
        const dim3 grid = row_grid<128>(A, per);
        return launch_early(cache_read_kernel<128>, grid, kRowThreads, 0, st, A, per);
    } else {
        const dim3 grid = row_grid<64>(A, per);
        return launch_early(cache_read_kernel<64>, grid, kRowThreads, 0, st, A, per);
    }
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
// Its time is a chain of three dependent reads (path, page, row) and a store, not
// bytes: 128 requests of 32 layers and 8 heads of 128, trees of 64 (31 MB moved), take
// 11 us, 2.8 TB/s in pieces of 16 and 8 bytes; 4 requests of 4 layers 3 us.
template <int D>
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const CacheCompactArgs A, int pairs_per_cta) {
    after_earlier();
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
    if (A.pool.D == 128) return launch_early(cache_compact_kernel<128>, grid, kCompactThreads, smem, st, A, per);
    else return launch_early(cache_compact_kernel<64>, grid, kCompactThreads, smem, st, A, per);
}

}  // namespace spec
