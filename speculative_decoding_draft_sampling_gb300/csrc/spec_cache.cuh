// spec_cache.cuh -- the paged 4-bit KV cache: block layout, page lookup and
// the argument records that the C API hands to the kernels.
//
// A block holds one page (P tokens) of one kv head:
//   K codes [P][D/2] | K scales bf16 [P][D/32] | V codes [P][D/2] | V scales bf16 [P][D/32]
// Element d of a row: low (even d) or high (odd d) half of byte d/2, value
// (code - 8) * scale[d / 32].  |code - 8| <= 7 has three significant bits and a
// scale five, so a value has at most eight: exact in bf16, and the tensor
// cores multiply exactly what the cache stands for.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace spec {

constexpr int kCacheGroup = 32;                 // values that share a scale
constexpr int kCacheMaxPages = 1 << 20;

// offsets inside a block, in bytes
template <int D>
struct CacheBlock {
    static constexpr int kRow = D / 2;          // bytes of a row's codes
    static constexpr int kScl = D / 16;         // bytes of a row's scales
    static constexpr int kTok = 2 * (kRow + kScl);
    __host__ __device__ static constexpr int v_codes(int P) { return P * (kRow + kScl); }
    __host__ __device__ static constexpr int bytes(int P) { return P * kTok; }
};

// A step is a row of short kernels.  They are launched so that a kernel's blocks may
// be set up while the kernel before it in the stream ends; every thread waits for that
// end, and for all that was written, before it reads anything (and reads nothing as
// constant: it may have been written after the launch).  A call takes 2 us less: one
// request's attention 12.4 to 10.0, a batch's reserve, forks and release 93 to 86 when it
// was made.
#ifdef __CUDACC__
__device__ __forceinline__ void after_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// lets the next kernel's blocks be set up now
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

struct CachePool {
    unsigned char* base;
    long long layer_stride, page_stride, head_stride;   // bytes
    int layers, num_pages, heads, D, P, p_shift;        // P = 1 << p_shift
};

struct CacheTable {
    const int* table;
    long long stride;
    int width;
};

// The page that holds position t of request b, or -1 (out of the table, no
// page, or an id outside the pool).
__device__ __forceinline__ int cache_page(const CacheTable& T, int num_pages, int p_shift, int b, long long t) {
    if (t < 0 || (t >> p_shift) >= T.width) return -1;
    const int page = T.table[b * T.stride + (t >> p_shift)];
    return static_cast<unsigned>(page) < static_cast<unsigned>(num_pages) ? page : -1;
}

struct CacheRowsArgs {                          // append and read
    CachePool pool;
    CacheTable tab;
    const uint16_t* k; long long k_bs, k_rs, k_hs;      // elements (append)
    const uint16_t* v; long long v_bs, v_rs, v_hs;
    uint16_t* k_out; uint16_t* v_out;                   // read
    const int* start; const int* count;
    int B, n;
    int aligned;                                // 16-byte rows of k and v
    int* status;
};
cudaError_t cache_append_run(const CacheRowsArgs& A, cudaStream_t st);
cudaError_t cache_read_run(const CacheRowsArgs& A, cudaStream_t st);

struct CacheCompactArgs {
    CachePool pool;
    CacheTable tab;
    const int* ctx; const int* path; int path_width; const int* accepted;
    int B;
    int* status;
};
cudaError_t cache_compact_run(const CacheCompactArgs& A, cudaStream_t st);

struct CachePagesArgs {                         // reserve, release, fork
    CachePool pool;                             // fork: the pages' bytes
    int* table; long long stride; int width;
    int* held; int* ref; int* free_list; int* num_free;
    const int* length;
    const int* src; const int* dst; int* new_page;      // fork
    int R, F, num_pages, p_shift;
    int* status;
};
cudaError_t cache_reserve_run(const CachePagesArgs& A, cudaStream_t st);
cudaError_t cache_release_run(const CachePagesArgs& A, cudaStream_t st);
cudaError_t cache_fork_run(const CachePagesArgs& A, cudaStream_t st);

struct CacheAttendArgs {
    CachePool pool;
    CacheTable tab;
    const uint16_t* q; long long q_bs, q_rs, q_hs;      // elements
    const int* ctx; const int* rows;
    const unsigned long long* mask; const int* depth;   // mask words: ceil(n / 64)
    int window, sinks;
    float scale;
    int B, n, hq, G;                            // G = q heads per kv head
    int aligned;                                // 16-byte rows of q
    uint16_t* out; float* lse; int* status;
    void* ws;
};
size_t cache_attend_ws(int B, int n, int hq, int hkv, int D);
// tiles that a request of this many positions may come to, over all kv heads and blocks of rows
long long cache_attend_tiles(int n, int hq, int hkv, long long positions);
cudaError_t cache_attend_run(const CacheAttendArgs& A, cudaStream_t st);

}  // namespace spec
