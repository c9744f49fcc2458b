// spec_cache_pages.cu -- which request holds which page of the paged cache:
// growing requests, forking them and freeing what nothing holds.
//
// The decisions are made by one CTA: they are a scan over the requests (who
// gets how many pages off the stack) and a pass over the pages held, a few
// kilobytes, and every order that a caller can see is fixed by request and
// page numbers, never by the order in which threads arrive.  What costs
// bandwidth, the copy of a forked request's last partial page in every layer
// and head, is a second kernel over the whole device.
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
    __shared__ int sums[kPageWarps];
    const int lane = threadIdx.x & 31;
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
        // a warp writes the pages of its 32 requests, one request at a time
        const int first = static_cast<int>(asked) + off;
#pragma unroll 1
        for (unsigned todo = __ballot_sync(0xffffffffu, ok); todo; todo &= todo - 1) {
            const int l = __ffs(todo) - 1;
            const int rr = r0 + static_cast<int>(threadIdx.x) - lane + l;
            const int cnt = __shfl_sync(0xffffffffu, need, l);
            const int at = __shfl_sync(0xffffffffu, first, l);
            const int h = __shfl_sync(0xffffffffu, held, l);
            for (int j = lane; j < cnt; j += 32) {
                const int page = take_page(A, have, at + j);
                if (page >= 0) A.ref[page] = 1;
                A.table[rr * A.stride + h + j] = page;
            }
        }
        int got;
        block_scan(ok ? need : 0, sums, got);
        taken += got;
        asked += total;
        if (asked > have) asked = static_cast<long long>(have) + 1;   // nobody behind gets a page
    }
    if (threadIdx.x == 0) A.num_free[0] = have - taken;
}

// References first, then the pages that nothing holds any more, marked in a
// bitmap in shared memory: reading it in order gives the stack its order.
__global__ void __launch_bounds__(kPageThreads) cache_release_kernel(const CachePagesArgs A) {
    extern __shared__ uint32_t freed[];         // one bit a page
    __shared__ int sums[kPageWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int words = (A.num_pages + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kPageThreads) freed[i] = 0;
    __syncthreads();
    for (int r = w; r < A.R; r += kPageWarps) {
        const int held = clamp_held(A.held[r], A.width);
        const int keep = min(held, pages_for(A.length[r], A.p_shift));
        int bits = 0;
        for (int j = keep + lane; j < held; j += 32) {
            int* entry = A.table + r * A.stride + j;
            const int page = *entry;
            *entry = -1;
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(A.num_pages)) {
                bits = SPEC_ST_BAD_PAGE;
                continue;
            }
            const int before = atomicSub(A.ref + page, 1);
            if (before == 1) {
                atomicOr(freed + (page >> 5), 1u << (page & 31));
            } else if (before <= 0) {           // nobody held it: left as it was
                atomicAdd(A.ref + page, 1);
                bits = SPEC_ST_BAD_PAGE;
            }
        }
        if (bits && A.status) atomicOr(A.status + r, bits);
        __syncwarp();
        if (lane == 0 && keep < held) A.held[r] = keep;
    }
    __syncthreads();
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
    __shared__ int sums[kPageWarps];
    const int lane = threadIdx.x & 31;
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
        // the shared pages, one child at a time a warp
#pragma unroll 1
        for (unsigned todo = __ballot_sync(0xffffffffu, ok && full > 0); todo; todo &= todo - 1) {
            const int l = __ffs(todo) - 1;
            const int s = __shfl_sync(0xffffffffu, src, l), d = __shfl_sync(0xffffffffu, dst, l);
            const int cnt = __shfl_sync(0xffffffffu, full, l);
            for (int j = lane; j < cnt; j += 32) {
                const int page = A.table[s * A.stride + j];
                A.table[d * A.stride + j] = page;
                if (static_cast<unsigned>(page) < static_cast<unsigned>(A.num_pages)) atomicAdd(A.ref + page, 1);
            }
        }
        int got;
        block_scan(ok ? own : 0, sums, got);
        taken += got;
        asked += total;
    }
    if (threadIdx.x == 0) A.num_free[0] = have - taken;
}

// One CTA copies the rows of one (fork, layer, range of heads): four runs a
// block, codes in 16-byte vectors and scales in 4-byte words.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const CachePagesArgs A) {
    using Blk = CacheBlock<D>;
    const int f = blockIdx.y, P = A.pool.P;
    const int to = A.new_page[f];
    if (to < 0) return;
    const int src = A.src[f];
    const int len = A.length[src];
    const int rows = len & (P - 1);
    const int from = A.table[src * A.stride + (len >> A.p_shift)];
    if (static_cast<unsigned>(from) >= static_cast<unsigned>(A.num_pages)) return;
    const int codes = rows * Blk::kRow / 16, scales = rows * Blk::kScl / 4;
    const int per = 2 * (codes + scales);
    const int pairs = A.pool.layers * A.pool.heads;
    for (int pair = blockIdx.x; pair < pairs; pair += gridDim.x) {
        const int layer = pair / A.pool.heads, head = pair % A.pool.heads;
        unsigned char* base = A.pool.base + layer * A.pool.layer_stride + head * A.pool.head_stride;
        const unsigned char* a = base + from * A.pool.page_stride;
        unsigned char* z = base + to * A.pool.page_stride;
        for (int w = threadIdx.x; w < per; w += kCopyThreads) {
            const int half = w >= codes + scales ? w - (codes + scales) : w;
            int at = half == w ? 0 : Blk::v_codes(P);
            if (half < codes) {
                at += half * 16;
                *reinterpret_cast<uint4*>(z + at) = *reinterpret_cast<const uint4*>(a + at);
            } else {
                at += P * Blk::kRow + (half - codes) * 4;
                *reinterpret_cast<uint32_t*>(z + at) = *reinterpret_cast<const uint32_t*>(a + at);
            }
        }
    }
}

}  // namespace

cudaError_t cache_reserve_run(const CachePagesArgs& A, cudaStream_t st) {
    cache_reserve_kernel<<<1, kPageThreads, 0, st>>>(A);
    return cudaGetLastError();
}

cudaError_t cache_release_run(const CachePagesArgs& A, cudaStream_t st) {
    const size_t smem = static_cast<size_t>((A.num_pages + 31) / 32) * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(cache_release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kCacheMaxPages / 8);
        if (e != cudaSuccess) return e;
    }
    cache_release_kernel<<<1, kPageThreads, smem, st>>>(A);
    return cudaGetLastError();
}

cudaError_t cache_fork_run(const CachePagesArgs& A, cudaStream_t st) {
    cache_fork_kernel<<<1, kPageThreads, 0, st>>>(A);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(A.pool.layers * A.pool.heads), static_cast<unsigned>(A.F));
    if (A.pool.D == 128) cache_copy_kernel<128><<<grid, kCopyThreads, 0, st>>>(A);
    else cache_copy_kernel<64><<<grid, kCopyThreads, 0, st>>>(A);
    return cudaGetLastError();
}

}  // namespace spec
