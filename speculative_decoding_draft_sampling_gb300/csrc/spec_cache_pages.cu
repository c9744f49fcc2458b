// spec_cache_pages.cu -- which request holds which page of the paged cache:
// growing requests, forking them and freeing what nothing holds.
//
// The decisions are made by one CTA: they are a scan over the requests (who
// gets how many pages off the stack) and a pass over the pages held, a few
// kilobytes, and every order that a caller can see is fixed by request and
// page numbers, never by the order in which threads arrive.  64 requests of
// 500 to 131 tokens, each forked twice: reserve 5 us, fork 7, release 8, all latency (a
// launch, the scan's barriers, dependent reads of table and counts).  What costs
// bandwidth, the copy of a forked request's last partial page in every layer
// and head, is a second kernel over the whole device.
#include <type_traits>

#include "../../include/spec_cache.h"
#include "spec_cache.cuh"

namespace spec {

namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kCopyThreads = 256;

// Exclusive scan of v over the CTA; `total` gets the sum.  Every thread calls.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) warp_sums[w] = inc;
    __syncthreads();
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    const int before = w ? __shfl_sync(0xffffffffu, s, w - 1) : 0;
    total = __shfl_sync(0xffffffffu, s, kPageWarps - 1);
    __syncthreads();                            // the sums may be written again
    return before + inc - v;
}

__device__ __forceinline__ int pages_for(int length, int p_shift) {
    return length <= 0 ? 0 : static_cast<int>((static_cast<unsigned>(length) + (1u << p_shift) - 1u) >> p_shift);
}

__device__ __forceinline__ int clamp_held(int held, int width) { return min(max(held, 0), width); }

// The i-th page off the stack, or -1 where the stack's entry is no page.
__device__ __forceinline__ int take_page(const CachePagesArgs& A, int num_free, int i) {
    const int page = A.free_list[num_free - 1 - i];
    return static_cast<unsigned>(page) < static_cast<unsigned>(A.num_pages) ? page : -1;
}

__device__ __forceinline__ int stack_size(const CachePagesArgs& A) {
    return min(max(A.num_free[0], 0), A.num_pages);
}

__global__ void __launch_bounds__(kPageThreads) cache_reserve_kernel(const CachePagesArgs A) {
    after_earlier();
    __shared__ int sums[kPageWarps];
    __shared__ int4 grant[kPageThreads];        // a request's pages: first of the taken, where in its row, how many
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int have = stack_size(A);
    long long asked = 0;                        // pages of all requests before this chunk
    int taken = 0;
    for (int r0 = 0; r0 < A.R; r0 += kPageThreads) {
        const int r = r0 + static_cast<int>(threadIdx.x);
        int held = 0, need = 0, bits = 0;
        if (r < A.R) {
            held = clamp_held(A.held[r], A.width);
            need = pages_for(A.length[r], A.p_shift);
            if (need > A.width) { bits = SPEC_ST_BAD_PAGE; need = 0; }
            need = max(0, need - held);
            need = min(need, A.num_pages + 1);  // more than any stack holds; keeps the sums in range
        }
        // 1024 needs of at most 2^20 + 1 pages: the chunk's sum fits 31 bits
        int total;
        const int off = block_scan(need, sums, total);
        const bool ok = need > 0 && asked + off + need <= have;
        if (need > 0 && !ok) bits = SPEC_ST_NO_PAGE;
        if (bits && A.status) atomicOr(A.status + r, bits);
        if (ok) A.held[r] = held + need;
        grant[threadIdx.x] = make_int4(static_cast<int>(asked) + off, held, ok ? need : 0, 0);
        int got;
        block_scan(ok ? need : 0, sums, got);   // (and a barrier)
        // the warps write the requests' pages in turn
        for (int l = w; l < min(kPageThreads, A.R - r0); l += kPageWarps) {
            const int4 g = grant[l];
            for (int j = lane; j < g.z; j += 32) {
                const int page = take_page(A, have, g.x + j);
                if (page >= 0) A.ref[page] = 1;
                A.table[(r0 + l) * A.stride + g.y + j] = page;
            }
        }
        __syncthreads();
        taken += got;
        asked += total;
        if (asked > have) asked = static_cast<long long>(have) + 1;   // nobody behind gets a page
    }
    if (threadIdx.x == 0) A.num_free[0] = have - taken;
}

// References first, then the pages that nothing holds any more, marked in a
// bitmap in shared memory: reading it in order gives the stack its order.
__global__ void __launch_bounds__(kPageThreads) cache_release_kernel(const CachePagesArgs A) {
    after_earlier();
    extern __shared__ uint32_t freed[];         // one bit a page
    __shared__ int sums[kPageWarps];
    __shared__ int2 spans[kPageThreads];
    constexpr int kFly = 4;                     // requests that a warp looks at together
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int words = (A.num_pages + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kPageThreads) freed[i] = 0;
    __syncthreads();
    for (int r0 = 0; r0 < A.R; r0 += kPageThreads) {
        const int r = r0 + static_cast<int>(threadIdx.x);
        int2 span = make_int2(0, 0);            // the pages that go: [x, y) of the request's
        if (r < A.R) {
            span.y = clamp_held(A.held[r], A.width);
            span.x = min(span.y, pages_for(A.length[r], A.p_shift));
            if (span.x < span.y) A.held[r] = span.x;
        }
        spans[threadIdx.x] = span;
        __syncthreads();
        // a warp has pages of several requests in flight: each is a read, an
        // update of the page's count and a look at what it was
        const int rows = min(kPageThreads, A.R - r0);
        for (int l0 = w; l0 < rows; l0 += kFly * kPageWarps) {
            int most = 0;
#pragma unroll
            for (int q = 0; q < kFly; ++q) {
                const int l = l0 + q * kPageWarps;
                if (l < rows) most = max(most, spans[l].y - spans[l].x);
            }
            for (int j = lane; j < most; j += 32) {
                int page[kFly], before[kFly];
#pragma unroll
                for (int q = 0; q < kFly; ++q) {
                    const int l = l0 + q * kPageWarps;
                    page[q] = -2;
                    if (l < rows && spans[l].x + j < spans[l].y) page[q] = A.table[(r0 + l) * A.stride + spans[l].x + j];
                }
#pragma unroll
                for (int q = 0; q < kFly; ++q) {
                    before[q] = 2;
                    if (static_cast<unsigned>(page[q]) < static_cast<unsigned>(A.num_pages))
                        before[q] = atomicSub(A.ref + page[q], 1);
                }
#pragma unroll
                for (int q = 0; q < kFly; ++q) {
                    const int l = l0 + q * kPageWarps;
                    if (page[q] == -2 && !(l < rows && spans[l].x + j < spans[l].y)) continue;
                    A.table[(r0 + l) * A.stride + spans[l].x + j] = -1;
                    bool bad = static_cast<unsigned>(page[q]) >= static_cast<unsigned>(A.num_pages);
                    if (!bad && before[q] == 1) {
                        atomicOr(freed + (page[q] >> 5), 1u << (page[q] & 31));
                    } else if (!bad && before[q] <= 0) {    // nobody held it: left as it was
                        atomicAdd(A.ref + page[q], 1);
                        bad = true;
                    }
                    if (bad && A.status) atomicOr(A.status + r0 + l, SPEC_ST_BAD_PAGE);
                }
            }
        }
        __syncthreads();
    }
    // Requests that were cut back into a page which others hold as well: whoever writes
    // there writes the others' rows.  Looked for only where somebody asks; all
    // references are dropped by now.
    if (A.status)
        for (int r = threadIdx.x; r < A.R; r += kPageThreads) {
            const int length = A.length[r], last = pages_for(length, A.p_shift) - 1;
            if (length <= 0 || !(length & ((1 << A.p_shift) - 1)) || last >= clamp_held(A.held[r], A.width)) continue;
            const int page = A.table[r * A.stride + last];
            if (static_cast<unsigned>(page) < static_cast<unsigned>(A.num_pages) && __ldcg(A.ref + page) > 1)
                atomicOr(A.status + r, SPEC_ST_SHARED_PAGE);
        }
    int top = stack_size(A);
    for (int i0 = 0; i0 < words; i0 += kPageThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        uint32_t m = i < words ? freed[i] : 0;
        int total;
        int at = top + block_scan(__popc(m), sums, total);
        for (; m; m &= m - 1, ++at)
            if (at < A.num_pages) A.free_list[at] = i * 32 + __ffs(m) - 1;
        top += total;
    }
    if (threadIdx.x == 0) A.num_free[0] = min(top, A.num_pages);
}

__global__ void __launch_bounds__(kPageThreads) cache_fork_kernel(const CachePagesArgs A) {
    after_earlier();
    let_next_start();                           // the copy
    __shared__ int sums[kPageWarps];
    __shared__ int4 shares[kPageThreads];       // parent, child, full pages shared
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int have = stack_size(A);
    int asked = 0, taken = 0;
    for (int f0 = 0; f0 < A.F; f0 += kPageThreads) {
        const int f = f0 + static_cast<int>(threadIdx.x);
        int src = -1, dst = -1, full = 0, bits = 0, own = 0;
        bool ok = false;
        if (f < A.F) {
            src = A.src[f];
            dst = A.dst[f];
            ok = src >= 0 && src < A.R && dst >= 0 && dst < A.R && src != dst;
            if (ok) {
                const int len = max(A.length[src], 0);
                full = len >> A.p_shift;
                own = (len & ((1 << A.p_shift) - 1)) ? 1 : 0;
                ok = A.held[dst] == 0 && full + own <= clamp_held(A.held[src], A.width);
            }
            if (!ok) { bits = SPEC_ST_BAD_PAGE; own = 0; }
        }
        int total;
        const int off = asked + block_scan(own, sums, total);
        if (ok && own && off + 1 > have) { ok = false; bits = SPEC_ST_NO_PAGE; }
        if (f < A.F) {
            int page = -1;
            if (ok && own) {
                page = take_page(A, have, off);
                if (page >= 0) A.ref[page] = 1;
                A.table[dst * A.stride + full] = page;
            }
            A.new_page[f] = page;
            if (ok) A.held[dst] = full + own;
            if (bits && A.status) atomicOr(A.status + f, bits);
        }
        shares[threadIdx.x] = make_int4(src, dst, ok ? full : 0, 0);
        int got;
        block_scan(ok ? own : 0, sums, got);    // (and a barrier)
        // the shared pages: the warps take the children in turn
#pragma unroll 4
        for (int l = w; l < min(kPageThreads, A.F - f0); l += kPageWarps) {
            const int4 g = shares[l];
            for (int j = lane; j < g.z; j += 32) {
                const int page = A.table[g.x * A.stride + j];
                A.table[g.y * A.stride + j] = page;
                if (static_cast<unsigned>(page) < static_cast<unsigned>(A.num_pages)) atomicAdd(A.ref + page, 1);
            }
        }
        __syncthreads();
        taken += got;
        asked += total;
    }
    if (threadIdx.x == 0) A.num_free[0] = have - taken;
}

// A CTA copies one fork's rows in a few (layer, head) blocks: four runs a block,
// codes in 16-byte pieces and scales a row at a time, a piece of each of kBlocks
// blocks in flight a thread.  It may be launched while the fork's decisions are
// still being made.  128 forks at 500 to 131 tokens (0 to 63 rows each), 32 layers, 8 heads
// of 128, 301 MB read and written: 53 us, 5.7 TB/s, reads in flight; one block in flight a
// thread is slower.
constexpr int kBlocks = 2;

template <int D>
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const CachePagesArgs A) {
    using Blk = CacheBlock<D>;
    using Scl = typename std::conditional<D == 128, uint2, uint32_t>::type;    // a row's scales
    after_earlier();
    const int f = blockIdx.y, P = A.pool.P;
    const int to = A.new_page[f];
    if (to < 0) return;
    const int src = A.src[f];
    const int len = A.length[src];
    const int rows = len & (P - 1);
    const int from = A.table[src * A.stride + (len >> A.p_shift)];
    if (static_cast<unsigned>(from) >= static_cast<unsigned>(A.num_pages)) return;
    const int codes = rows * Blk::kRow / 16, half = codes + rows;
    const int pairs = A.pool.layers * A.pool.heads;
    const long long move = (static_cast<long long>(to) - from) * A.pool.page_stride;
    const int p0 = blockIdx.x * kBlocks;
    unsigned char* blk[kBlocks];
#pragma unroll
    for (int q = 0; q < kBlocks; ++q) {
        const int layer = (p0 + q) / A.pool.heads, head = (p0 + q) % A.pool.heads;
        blk[q] = A.pool.base + layer * A.pool.layer_stride + head * A.pool.head_stride + from * A.pool.page_stride;
    }
    for (int w = threadIdx.x; w < 2 * half; w += kCopyThreads) {
        const int x = w >= half ? w - half : w;
        int at = w >= half ? Blk::v_codes(P) : 0;
        if (x < codes) {
            at += x * 16;
            uint4 r[kBlocks];
#pragma unroll
            for (int q = 0; q < kBlocks; ++q)
                if (p0 + q < pairs) r[q] = __ldcs(reinterpret_cast<const uint4*>(blk[q] + at));
#pragma unroll
            for (int q = 0; q < kBlocks; ++q)
                if (p0 + q < pairs) *reinterpret_cast<uint4*>(blk[q] + at + move) = r[q];
        } else {
            at += P * Blk::kRow + (x - codes) * Blk::kScl;
            Scl r[kBlocks];
#pragma unroll
            for (int q = 0; q < kBlocks; ++q)
                if (p0 + q < pairs) r[q] = *reinterpret_cast<const Scl*>(blk[q] + at);
#pragma unroll
            for (int q = 0; q < kBlocks; ++q)
                if (p0 + q < pairs) *reinterpret_cast<Scl*>(blk[q] + at + move) = r[q];
        }
    }
}

}  // namespace

cudaError_t cache_reserve_run(const CachePagesArgs& A, cudaStream_t st) {
    return launch_early(cache_reserve_kernel, 1, kPageThreads, 0, st, A);
}

cudaError_t cache_release_run(const CachePagesArgs& A, cudaStream_t st) {
    const size_t smem = static_cast<size_t>((A.num_pages + 31) / 32) * 4;
    if (smem > 32 * 1024) {                     // (beside the static arrays)
        const cudaError_t e = cudaFuncSetAttribute(cache_release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kCacheMaxPages / 8);
        if (e != cudaSuccess) return e;
    }
    return launch_early(cache_release_kernel, 1, kPageThreads, smem, st, A);
}

cudaError_t cache_fork_run(const CachePagesArgs& A, cudaStream_t st) {
    const cudaError_t e = launch_early(cache_fork_kernel, 1, kPageThreads, 0, st, A);
    if (e != cudaSuccess) return e;
    // the copy waits for the decisions on the device, not for their launch's end
    const int pairs = A.pool.layers * A.pool.heads;
    const dim3 grid(static_cast<unsigned>((pairs + kBlocks - 1) / kBlocks), static_cast<unsigned>(A.F));
    return launch_early(A.pool.D == 128 ? cache_copy_kernel<128> : cache_copy_kernel<64>, grid, kCopyThreads, 0, st, A);
}

}  // namespace spec
