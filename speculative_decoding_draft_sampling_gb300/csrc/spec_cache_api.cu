// spec_cache_api.cu -- the C ABI of the paged 4-bit cache: argument checks and
// launches.  Nothing here allocates, synchronises or throws.
#include "../../include/spec_cache.h"
#include "spec_cache.cuh"
#include "spec_host.cuh"

namespace {

using spec::cuda_fail;
using spec::fail;

int shift_of(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : -1; }

// Pools (bulk copies) and the pages' state (atomics) must be device memory.
spec_status device_only(const char* who, const char* name, const void* p) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) == cudaSuccess &&
        (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged))
        return SPEC_OK;
    cudaGetLastError();
    return fail(SPEC_INVALID_ARG, "%s: %s must be device memory", who, name);
}

#define CACHE_TRY(call)                           \
    do {                                          \
        const spec_status try_s_ = (call);        \
        if (try_s_ != SPEC_OK) return try_s_;     \
    } while (0)

spec_status pool_of(const char* who, const void* pool, int layers, int64_t layer_stride, int64_t page_stride,
                    int64_t head_stride, int num_pages, int kv_heads, int head_dim, int page_size,
                    spec::CachePool& out) {
    const size_t block = spec_cache_block_bytes(head_dim, page_size);
    if (block == 0)
        return fail(SPEC_UNSUPPORTED, "%s: head_dim is 64 or 128 and page_size 16, 32 or 64 (got %d and %d)", who,
                    head_dim, page_size);
    if (kv_heads < 1 || layers < 1 || num_pages < 0)
        return fail(SPEC_INVALID_ARG, "%s: need kv_heads >= 1, layers >= 1, num_pages >= 0", who);
    if (num_pages > spec::kCacheMaxPages || kv_heads > 65535 || layers > 65535)
        return fail(SPEC_UNSUPPORTED, "%s: at most 2^20 pages, 65535 kv heads and 65535 layers", who);
    if (!pool) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    const int64_t least = static_cast<int64_t>(block);
    if (reinterpret_cast<uintptr_t>(pool) % 16 || page_stride % 16 || head_stride % 16 || layer_stride % 16)
        return fail(SPEC_INVALID_ARG, "%s: the pool and its strides must be multiples of 16 bytes", who);
    if (page_stride < least || head_stride < least || (layers > 1 && layer_stride < least))
        return fail(SPEC_INVALID_ARG, "%s: strides below a block's %lld bytes", who, static_cast<long long>(least));
    CACHE_TRY(device_only(who, "pool", pool));
    out.base = static_cast<unsigned char*>(const_cast<void*>(pool));
    out.layer_stride = layer_stride;
    out.page_stride = page_stride;
    out.head_stride = head_stride;
    out.layers = layers;
    out.num_pages = num_pages;
    out.heads = kv_heads;
    out.D = head_dim;
    out.P = page_size;
    out.p_shift = shift_of(page_size);
    return SPEC_OK;
}

spec_status table_of(const char* who, const int32_t* table, int64_t stride, int width, spec::CacheTable& out) {
    if (!table) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    if (width < 1 || stride < width)
        return fail(SPEC_INVALID_ARG, "%s: need table_width >= 1 and table_stride >= table_width", who);
    SPEC_MAP(table);
    out.table = table;
    out.stride = stride;
    out.width = width;
    return SPEC_OK;
}

bool rows16(const void* p, int64_t a, int64_t b, int64_t c) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0;
}

spec_status done(const char* who, cudaError_t e) { return e == cudaSuccess ? SPEC_OK : cuda_fail(e, who); }

}  // namespace

extern "C" {

size_t spec_cache_block_bytes(int head_dim, int page_size) {
    if ((head_dim != 64 && head_dim != 128) || shift_of(page_size) < 0) return 0;
    return static_cast<size_t>(head_dim) * page_size * 9 / 8;
}

spec_status spec_cache_append(
    const void* k, int64_t k_bs, int64_t k_rs, int64_t k_hs,
    const void* v, int64_t v_bs, int64_t v_rs, int64_t v_hs,
    void* pool, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* start, const int32_t* count,
    int B, int n, int kv_heads, int head_dim, int page_size, int32_t* status, void* stream) {
    const char* who = "spec_cache_append";
    if (B < 0 || n < 0) return fail(SPEC_INVALID_ARG, "%s: need B >= 0 and n >= 0", who);
    if (B == 0 || n == 0) return SPEC_OK;
    spec::CacheRowsArgs A{};
    CACHE_TRY(pool_of(who, pool, 1, 0, page_stride, head_stride, num_pages, kv_heads, head_dim, page_size, A.pool));
    CACHE_TRY(table_of(who, page_table, table_stride, table_width, A.tab));
    if (!k || !v || !start) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    if (reinterpret_cast<uintptr_t>(k) % 2 || reinterpret_cast<uintptr_t>(v) % 2)
        return fail(SPEC_INVALID_ARG, "%s: k and v must be 2-byte aligned", who);
    SPEC_MAP(k);
    SPEC_MAP(v);
    SPEC_MAP(start);
    SPEC_MAP(count);
    SPEC_MAP(status);
    A.k = static_cast<const uint16_t*>(k); A.k_bs = k_bs; A.k_rs = k_rs; A.k_hs = k_hs;
    A.v = static_cast<const uint16_t*>(v); A.v_bs = v_bs; A.v_rs = v_rs; A.v_hs = v_hs;
    A.start = start; A.count = count; A.B = B; A.n = n; A.status = status;
    A.aligned = rows16(k, k_bs, k_rs, k_hs) && rows16(v, v_bs, v_rs, v_hs);
    return done(who, spec::cache_append_run(A, static_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_read(
    const void* pool, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* start, const int32_t* count,
    int B, int n, int kv_heads, int head_dim, int page_size,
    void* k, void* v, int32_t* status, void* stream) {
    const char* who = "spec_cache_read";
    if (B < 0 || n < 0) return fail(SPEC_INVALID_ARG, "%s: need B >= 0 and n >= 0", who);
    if (B == 0 || n == 0) return SPEC_OK;
    spec::CacheRowsArgs A{};
    CACHE_TRY(pool_of(who, pool, 1, 0, page_stride, head_stride, num_pages, kv_heads, head_dim, page_size, A.pool));
    CACHE_TRY(table_of(who, page_table, table_stride, table_width, A.tab));
    if (!k || !v || !start) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    if (reinterpret_cast<uintptr_t>(k) % 16 || reinterpret_cast<uintptr_t>(v) % 16)
        return fail(SPEC_INVALID_ARG, "%s: k and v must be 16-byte aligned", who);
    SPEC_MAP(k);
    SPEC_MAP(v);
    SPEC_MAP(start);
    SPEC_MAP(count);
    SPEC_MAP(status);
    A.k_out = static_cast<uint16_t*>(k); A.v_out = static_cast<uint16_t*>(v);
    A.start = start; A.count = count; A.B = B; A.n = n; A.status = status;
    return done(who, spec::cache_read_run(A, static_cast<cudaStream_t>(stream)));
}

size_t spec_cache_attend_workspace_size(int B, int n, int q_heads, int kv_heads, int head_dim) {
    if (B < 1 || n < 1 || n > 1024 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return spec::cache_attend_ws(B, n, q_heads, kv_heads, head_dim);
}

spec_status spec_cache_attend(
    const void* q, int64_t q_bs, int64_t q_rs, int64_t q_hs,
    const void* pool, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* ctx_len, const int32_t* num_rows,
    const uint64_t* anc_mask, const int32_t* depth, int window, int sinks, float scale,
    int B, int n, int q_heads, int kv_heads, int head_dim, int page_size,
    void* out, float* lse, int32_t* status, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "spec_cache_attend";
    if (B < 0 || n < 0) return fail(SPEC_INVALID_ARG, "%s: need B >= 0 and n >= 0", who);
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads)
        return fail(SPEC_INVALID_ARG, "%s: q_heads must be a multiple of kv_heads (got %d and %d)", who, q_heads,
                    kv_heads);
    if (window < 0 || sinks < 0) return fail(SPEC_INVALID_ARG, "%s: need window >= 0 and sinks >= 0", who);
    // the kernels multiply by 16 scale log2 e
    if (!(scale > 0.0f) || !(scale < 1.4e37f)) return fail(SPEC_INVALID_ARG, "%s: need a scale > 0 and < 1.4e37", who);
    if (depth && !anc_mask) return fail(SPEC_INVALID_ARG, "%s: depth goes with anc_mask", who);
    if (n > 1024) return fail(SPEC_UNSUPPORTED, "%s: at most 1024 rows a request (got %d)", who, n);
    if (B > 65535 || q_heads > 65535) return fail(SPEC_UNSUPPORTED, "%s: at most 65535 requests and q heads", who);
    if (B == 0 || n == 0) return SPEC_OK;
    spec::CacheAttendArgs A{};
    // positions, and a request's tiles over all kv heads and blocks of rows, are counted in 32 bits
    if (static_cast<long long>(table_width) * page_size > 0x7fff0000LL)
        return fail(SPEC_UNSUPPORTED, "%s: a table of more than 2^31 positions", who);
    if (table_width > 0 && shift_of(page_size) >= 0 &&
        spec::cache_attend_tiles(n, q_heads, kv_heads, static_cast<long long>(table_width) * page_size) > 0x7fffffffLL)
        return fail(SPEC_UNSUPPORTED, "%s: %d pages of %d tokens a request are too many for %d rows of %d q heads", who,
                    table_width, page_size, n, q_heads);
    CACHE_TRY(pool_of(who, pool, 1, 0, page_stride, head_stride, num_pages, kv_heads, head_dim, page_size, A.pool));
    CACHE_TRY(table_of(who, page_table, table_stride, table_width, A.tab));
    if (!q || !ctx_len || !out) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    if (reinterpret_cast<uintptr_t>(q) % 2 || reinterpret_cast<uintptr_t>(out) % 16)
        return fail(SPEC_INVALID_ARG, "%s: q must be 2-byte and out 16-byte aligned", who);
    const size_t need = spec::cache_attend_ws(B, n, q_heads, kv_heads, head_dim);
    if (need > 0) {
        if (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16)
            return fail(SPEC_INVALID_ARG, "%s: the workspace needs %zu bytes, 16-byte aligned", who, need);
        SPEC_WS_DEVICE(ws);
    }
    SPEC_MAP(q);
    SPEC_MAP(ctx_len);
    SPEC_MAP(num_rows);
    SPEC_MAP(anc_mask);
    SPEC_MAP(depth);
    SPEC_MAP(out);
    SPEC_MAP(lse);
    SPEC_MAP(status);
    A.q = static_cast<const uint16_t*>(q); A.q_bs = q_bs; A.q_rs = q_rs; A.q_hs = q_hs;
    A.ctx = ctx_len; A.rows = num_rows;
    A.mask = reinterpret_cast<const unsigned long long*>(anc_mask);
    A.depth = depth;
    A.window = window; A.sinks = sinks; A.scale = scale;
    A.B = B; A.n = n; A.hq = q_heads; A.G = q_heads / kv_heads;
    A.aligned = rows16(q, q_bs, q_rs, q_hs);
    A.out = static_cast<uint16_t*>(out); A.lse = lse; A.status = status; A.ws = ws;
    return done(who, spec::cache_attend_run(A, static_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_compact(
    void* pool, int layers, int64_t layer_stride, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* ctx_len, const int32_t* path, int path_width, const int32_t* num_accepted,
    int B, int kv_heads, int head_dim, int page_size, int32_t* status, void* stream) {
    const char* who = "spec_cache_compact";
    if (B < 0 || path_width < 1) return fail(SPEC_INVALID_ARG, "%s: need B >= 0 and path_width >= 1", who);
    if (path_width > 1024 || B > 65535)
        return fail(SPEC_UNSUPPORTED, "%s: at most 1024 path entries and 65535 requests", who);
    if (B == 0) return SPEC_OK;
    spec::CacheCompactArgs A{};
    CACHE_TRY(pool_of(who, pool, layers, layer_stride, page_stride, head_stride, num_pages, kv_heads, head_dim,
                      page_size, A.pool));
    CACHE_TRY(table_of(who, page_table, table_stride, table_width, A.tab));
    if (!ctx_len || !path || !num_accepted) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    SPEC_MAP(ctx_len);
    SPEC_MAP(path);
    SPEC_MAP(num_accepted);
    SPEC_MAP(status);
    A.ctx = ctx_len; A.path = path; A.path_width = path_width; A.accepted = num_accepted;
    A.B = B; A.status = status;
    return done(who, spec::cache_compact_run(A, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// the checks that the three page calls share
spec_status pages_of(const char* who, int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
                     int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages, const int32_t* length, int R,
                     int page_size, int32_t* status, spec::CachePagesArgs& A) {
    if (shift_of(page_size) < 0)
        return fail(SPEC_UNSUPPORTED, "%s: page_size is 16, 32 or 64 (got %d)", who, page_size);
    if (num_pages < 1) return fail(SPEC_INVALID_ARG, "%s: need num_pages >= 1", who);
    if (num_pages > spec::kCacheMaxPages) return fail(SPEC_UNSUPPORTED, "%s: at most 2^20 pages", who);
    if (!num_held || !ref || !free_list || !num_free || !length)
        return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    spec::CacheTable T;
    CACHE_TRY(table_of(who, page_table, table_stride, table_width, T));
    CACHE_TRY(device_only(who, "page_table", page_table));
    CACHE_TRY(device_only(who, "num_held", num_held));
    CACHE_TRY(device_only(who, "ref", ref));
    CACHE_TRY(device_only(who, "free_list", free_list));
    CACHE_TRY(device_only(who, "num_free", num_free));
    SPEC_MAP(length);
    SPEC_MAP(status);
    A.table = const_cast<int*>(T.table); A.stride = table_stride; A.width = table_width;
    A.held = num_held; A.ref = ref; A.free_list = free_list; A.num_free = num_free;
    A.length = length; A.R = R; A.num_pages = num_pages; A.p_shift = shift_of(page_size); A.status = status;
    return SPEC_OK;
}

}  // namespace

extern "C" {

spec_status spec_cache_reserve(
    int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
    int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages,
    const int32_t* length, int R, int page_size, int32_t* status, void* stream) {
    const char* who = "spec_cache_reserve";
    if (R < 0) return fail(SPEC_INVALID_ARG, "%s: need R >= 0", who);
    if (R == 0) return SPEC_OK;
    spec::CachePagesArgs A{};
    CACHE_TRY(pages_of(who, page_table, table_stride, table_width, num_held, ref, free_list, num_free, num_pages,
                       length, R, page_size, status, A));
    return done(who, spec::cache_reserve_run(A, static_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_release(
    int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
    int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages,
    const int32_t* length, int R, int page_size, int32_t* status, void* stream) {
    const char* who = "spec_cache_release";
    if (R < 0) return fail(SPEC_INVALID_ARG, "%s: need R >= 0", who);
    if (R == 0) return SPEC_OK;
    spec::CachePagesArgs A{};
    CACHE_TRY(pages_of(who, page_table, table_stride, table_width, num_held, ref, free_list, num_free, num_pages,
                       length, R, page_size, status, A));
    return done(who, spec::cache_release_run(A, static_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_fork(
    void* pool, int layers, int64_t layer_stride, int64_t page_stride, int64_t head_stride,
    int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
    int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages,
    const int32_t* src, const int32_t* dst, const int32_t* length, int R, int F,
    int kv_heads, int head_dim, int page_size, int32_t* new_page, int32_t* status, void* stream) {
    const char* who = "spec_cache_fork";
    if (R < 0 || F < 0) return fail(SPEC_INVALID_ARG, "%s: need R >= 0 and F >= 0", who);
    if (F > 65535) return fail(SPEC_UNSUPPORTED, "%s: at most 65535 forks a call", who);
    if (F == 0) return SPEC_OK;
    spec::CachePagesArgs A{};
    CACHE_TRY(pool_of(who, pool, layers, layer_stride, page_stride, head_stride, num_pages, kv_heads, head_dim,
                      page_size, A.pool));
    CACHE_TRY(pages_of(who, page_table, table_stride, table_width, num_held, ref, free_list, num_free, num_pages,
                       length, R, page_size, status, A));
    if (!src || !dst || !new_page) return fail(SPEC_INVALID_ARG, "%s: null pointer argument", who);
    SPEC_MAP(src);
    SPEC_MAP(dst);
    SPEC_MAP(new_page);
    A.src = src; A.dst = dst; A.new_page = new_page; A.F = F;
    return done(who, spec::cache_fork_run(A, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
