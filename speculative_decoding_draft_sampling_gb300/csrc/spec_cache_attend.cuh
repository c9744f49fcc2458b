// spec_cache_attend.cuh -- what the attention kernels over the paged 4-bit cache
// share: the deal of the work, which keys a row sees, codes to bf16.
//
// The work.  A unit is (request, kv head, block of rows); its keys are cut into
// tiles of kTile tokens.  All tiles of all units, in order, are dealt out in
// equal contiguous shares to a grid that fills the device once, whatever the
// requests' lengths; a unit that several CTAs share is joined by the last of
// them to finish, in CTA order (so the bits do not depend on timing).
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "../../include/spec_cache.h"
#include "spec_cache.cuh"
#include "spec_common.cuh"

namespace spec {

// Failure-path test builds (-DSPEC_TEST_HOOKS): when set, CTA 0 leaves out its first
// copy (spec_cache_attend.cu) or the commit of its first scores
// (spec_cache_attend_tc.cu), so that every wait that depends on it runs into its
// limit and the kernel must leave with the workspace error set.
#ifdef SPEC_TEST_HOOKS
static __device__ int g_test_drop;
#endif

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.0e38f;              // the maximum before any key
constexpr float kSlack = 8.0f;                  // how far (in powers of two) a score may pass the maximum

// ---------------------------------------------------------------------------
// the workspace and the shares of the work
// ---------------------------------------------------------------------------
// control words (zero before the first call; every call leaves `arrived` zero)
struct AttendCtrl {
    uint32_t pad0;
    uint32_t error;                             // SPEC_WS_ERR_WAIT, where spec_workspace_error reads it
    uint32_t pad1[62];
    uint32_t arrived[(SPEC_CACHE_WS_CONTROL - 256) / 4];   // per CTA: parts done of the unit that starts in it
};

static_assert(sizeof(AttendCtrl) == SPEC_CACHE_WS_CONTROL, "the control words");
constexpr int kMaxGrid = (SPEC_CACHE_WS_CONTROL - 256) / 4;

struct AttendPlan {
    uint32_t one2;                              // 0x3F803F80 (codes2)
    int row_tiles;                              // blocks of rows a (request, kv head)
    int min_tiles;                              // tiles worth a CTA
    float* ml;                                  // [2 * grid][rows of a block][4]: m, l, l of the rounded weights
    float* part;                                // [2 * grid][rows of a block][D]
    AttendCtrl* ctrl;
};

// What a request asks for.
template <int kTile>
struct Req {
    int ctx, rows, len;                         // len = ctx + rows
    int first;                                  // tiles [0, sink_tiles) and [first, tiles) hold visible keys
    int sink_tiles, tiles;                      // tiles: of the whole context
    int low;                                    // positions below are outside every row's window (sinks aside)

    Req() = default;
    __device__ __forceinline__ Req(const CacheAttendArgs& A, int2 given) {
        const long long room = static_cast<long long>(A.tab.width) << A.pool.p_shift;
        ctx = static_cast<int>(min(static_cast<long long>(max(given.x, 0)), room));
        rows = min(max(given.y, 0), A.n);
        len = rows ? ctx + rows : 0;
        tiles = (len + kTile - 1) / kTile;
        low = 0;
        sink_tiles = 0;
        first = 0;
        if (A.window > 0) {
            low = max(0, ctx - A.window + 1);
            sink_tiles = min(tiles, (min(A.sinks, len) + kTile - 1) / kTile);
            first = min(max(low / kTile, sink_tiles), tiles);
        }
    }
    __device__ __forceinline__ int visited() const { return max(1, sink_tiles + tiles - first); }
    __device__ __forceinline__ int real(int v) const { return v < sink_tiles ? v : first + (v - sink_tiles); }
    // tiles of one kv head: blocks of rows that hold no row cost one
    __device__ __forceinline__ int head_work(const CacheAttendArgs& A, int row_tiles, int rows_a_block) const {
        const int live = (rows * A.G + rows_a_block - 1) / rows_a_block;
        return live * visited() + (row_tiles - live);
    }
    // whether a position of the cache may be seen (it lies before the end, and
    // in some row's window or among the sinks): others are not looked up
    __device__ __forceinline__ bool needs(const CacheAttendArgs& A, int t0, int t1) const {
        return t0 < len && (A.window == 0 || t0 < A.sinks || t1 > low);
    }
    // Visited tiles [from, to) are such that every row sees every key (there may be
    // others: a range that costs nothing to look up).
    __device__ __forceinline__ void plain(const CacheAttendArgs& A, int& from, int& to) const {
        from = A.window > 0 ? sink_tiles + max(0, (low + A.n + kTile - 1) / kTile - first) : 0;
        to = sink_tiles + ctx / kTile - first;
    }
    // whether some row may not see some key of the tile at t0
    __device__ __forceinline__ bool partial(const CacheAttendArgs& A, int t0) const {
        return t0 + kTile > ctx || (A.window > 0 && t0 + kTile > A.sinks && t0 < low + A.n);
    }
};

// its context and rows as given
__device__ __forceinline__ int2 request_len(const CacheAttendArgs& A, int b) {
    return make_int2(A.ctx[b], A.rows ? A.rows[b] : A.n);
}

// A unit, or the part of it that falls into a CTA's share.
struct Segment {
    int b, h, row0, live_rows;                  // request, kv head, first row, rows that are there
    int v0, v1, tiles_u;                        // tiles [v0, v1) of the unit's
    int tiles;                                  // v1 - v0, or 0 where no row is there
    long long u_from;                           // the unit's first tile among all
    __device__ __forceinline__ bool whole() const { return v0 == 0 && v1 == tiles_u; }
};

template <int kWarps>
struct ShareScratch {                           // in shared memory
    long long sum[kWarps], found[2];
    long long total, lo, hi;                    // all tiles, and this CTA's share of them
    int active;                                 // CTAs that have work
    int2 len[32 * kWarps];                      // the first requests' lengths
};

// A CTA's share [lo, hi) of all tiles, and a cursor over its segments.
template <int kTile, int kWarps>
struct Share {
    const CacheAttendArgs& A;
    const AttendPlan& L;
    const ShareScratch<kWarps>& S;
    const int rows_a_block;
    // the share's limits: in registers where the CTA is small, else in shared memory
    static constexpr bool kRegs = kWarps <= 4;
    long long total_, lo_, hi_;
    int active_;
    int b;                                      // the cursor's request, and where its tiles start
    long long b_from;
    Req<kTile> rq;

    // quotients of 64 bits only where the work needs them
    static __device__ __forceinline__ long long quotient(long long x, long long y) {
        return (x | y) >> 32 ? x / y : static_cast<long long>(static_cast<unsigned>(x) / static_cast<unsigned>(y));
    }
    __device__ __forceinline__ long long start_of(long long c) const { return quotient(c * total(), active()); }
    // the CTA whose share holds tile x
    __device__ __forceinline__ int cta_of(long long x) const {
        int c = static_cast<int>(quotient(x * active(), total()));
        while (start_of(c + 1) <= x) ++c;
        while (start_of(c) > x) --c;
        return c;
    }
    __device__ __forceinline__ Req<kTile> req_at(int i) const {
        return Req<kTile>(A, i < 32 * kWarps ? S.len[i] : request_len(A, i));
    }

    __device__ __forceinline__ long long total() const { return kRegs ? total_ : S.total; }
    __device__ __forceinline__ long long lo() const { return kRegs ? lo_ : S.lo; }
    __device__ __forceinline__ long long hi() const { return kRegs ? hi_ : S.hi; }
    __device__ __forceinline__ int active() const { return kRegs ? active_ : S.active; }

    // Every thread of the CTA takes part.  A CTA without work has lo == hi.
    __device__ __forceinline__ Share(const CacheAttendArgs& A_, const AttendPlan& L_, ShareScratch<kWarps>& scratch,
                                     int rows_a_block_)
        : A(A_), L(L_), S(scratch), rows_a_block(rows_a_block_) {
        constexpr int kThreads = 32 * kWarps;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int H = A.pool.heads;
        int2 given = make_int2(0, 0);
        auto work_of = [&](int i) {
            if (i >= A.B) return 0ll;
            given = request_len(A, i);
            return static_cast<long long>(H) * Req<kTile>(A, given).head_work(A, L.row_tiles, rows_a_block);
        };
        // Sums of all requests' tiles, a chunk of threads at a time; the chunk of the
        // first requests, the only one in the usual case, is scanned as it is summed.
        auto scan = [&](long long v, long long& before) {   // tiles before this thread's, and of the chunk
            long long inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            if (lane == 31) scratch.sum[warp] = inc;
            __syncthreads();
            long long all = 0;
            before = inc - v;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += scratch.sum[w];
                all += scratch.sum[w];
            }
            __syncthreads();
            return all;
        };
        const long long first_work = work_of(tid);
        scratch.len[tid] = given;
        long long first_before, unused;
        const long long first_all = scan(first_work, first_before);
        long long total = first_all;                        // (as the member, while it is counted)
        for (int b0 = kThreads; b0 < A.B; b0 += kThreads) total += scan(work_of(b0 + tid), unused);
        const long long units = static_cast<long long>(A.B) * H * L.row_tiles;
        long long want = quotient(total, L.min_tiles);
        if (want > units * 64) want = units * 64;           // what joins a unit must stay small beside it
        const int active = static_cast<int>(min(static_cast<long long>(gridDim.x), max(want, 1ll)));
        const int cta = blockIdx.x;
        b = 0;
        b_from = 0;
        const long long lo = cta < active ? quotient(cta * total, active) : 0;
        const long long hi = cta < active ? quotient((cta + 1) * total, active) : 0;
        if constexpr (kRegs) {
            total_ = total;
            active_ = active;
            lo_ = lo;
            hi_ = hi;
        } else {
            if (tid == 0) {
                scratch.total = total;
                scratch.active = active;
                scratch.lo = lo;
                scratch.hi = hi;
            }
            __syncthreads();
        }
        if (cta >= active) return;
        // the request that holds tile lo, and where its tiles start
        long long base = 0, v = first_work, before = first_before, all = first_all;
        for (int b0 = 0;;) {
            const long long from = base + before;
            if (v > 0 && from <= lo && lo < from + v) {
                scratch.found[0] = b0 + tid;
                scratch.found[1] = from;
            }
            base += all;
            b0 += kThreads;
            if (lo < base || b0 >= A.B) break;
            v = work_of(b0 + tid);
            all = scan(v, before);
        }
        __syncthreads();
        b = static_cast<int>(scratch.found[0]);
        b_from = scratch.found[1];
        rq = req_at(b);
    }

    // The unit that holds tile pos, which does not go back; rq becomes its request.
    __device__ __forceinline__ Segment segment(long long pos) {
        Segment g;
        const int H = A.pool.heads;
        int per_head = rq.head_work(A, L.row_tiles, rows_a_block);
        while (pos - b_from >= static_cast<long long>(per_head) * H) {
            b_from += static_cast<long long>(per_head) * H;
            rq = req_at(++b);
            per_head = rq.head_work(A, L.row_tiles, rows_a_block);
        }
        const unsigned in_req = static_cast<unsigned>(pos - b_from);
        g.b = b;
        g.h = in_req / static_cast<unsigned>(per_head);
        const int in_head = in_req - static_cast<unsigned>(g.h) * per_head;
        const int live = (rq.rows * A.G + rows_a_block - 1) / rows_a_block;
        const int visited = rq.visited();
        int rt;
        if (in_head < live * visited) {
            rt = static_cast<unsigned>(in_head) / static_cast<unsigned>(visited);
            g.tiles_u = visited;
            g.v0 = in_head - rt * visited;
        } else {
            rt = live + in_head - live * visited;
            g.tiles_u = 1;
            g.v0 = 0;
        }
        g.u_from = pos - g.v0;
        g.v1 = static_cast<int>(min(static_cast<long long>(g.tiles_u), hi() - g.u_from));
        g.row0 = rt * rows_a_block;
        g.live_rows = min(max(rq.rows * A.G - g.row0, 0), rows_a_block);
        g.tiles = g.live_rows > 0 ? g.v1 - g.v0 : 0;
        return g;
    }
    // the CTA that holds a segment's unit's first tile, and how many share it
    __device__ __forceinline__ void sharers(const Segment& g, int& c0, int& parts) const {
        const int cta = blockIdx.x;
        c0 = g.v0 == 0 ? cta : cta_of(g.u_from);
        parts = (g.v1 == g.tiles_u ? cta : cta_of(g.u_from + g.tiles_u - 1)) - c0 + 1;
    }
};

// ---------------------------------------------------------------------------
// codes to bf16
// ---------------------------------------------------------------------------
// Two codes that lie 16 bits apart (at 4i and 4i + 16) as bf16: placed at bits
// 3..6 of the significand under the exponent of 1 they are 1 + code/16, and one
// fused multiply-add with (s, -1.5 s) gives (code - 8)/16 * s, exactly (a scale
// has five significant bits, so 1.5 s fits too).  The factor 16 goes into the
// softmax scale (K) and the final division (V).  one2 is 0x3F803F80, the two
// ones' bits, out of the kernel's parameters: as a literal beside the mask's it
// costs a second logic instruction, the pipe that these kernels fill first
// (4 requests of 131072 to 57344 tokens: 144 against 128 us).
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t s2, uint32_t c2, uint32_t one2) {
    uint32_t t;
    if constexpr (I == 0) t = w << 3;
    else t = w >> (4 * I - 3);
    t = (t & 0x00780078u) | one2;
    uint32_t v;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(t), "r"(s2), "r"(c2));
    return v;
}
__device__ __forceinline__ uint32_t minus1_5(uint32_t s2) {
    uint32_t v;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(s2), "r"(0xBFC0BFC0u));
    return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float v;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(x));
    return v;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}
// bits [a, b) of a tile that starts at t0
__device__ __forceinline__ unsigned long long range64(long long a, long long b, long long t0) {
    const int lo = static_cast<int>(min(max(a - t0, 0ll), 64ll)), hi = static_cast<int>(min(max(b - t0, 0ll), 64ll));
    if (hi <= lo) return 0;
    return (hi == 64 ? ~0ull : (1ull << hi) - 1ull) & ~((1ull << lo) - 1ull);
}

// Which of the 64 keys from t0 on row i of request b sees.
template <int kTile>
__device__ __forceinline__ unsigned long long seen64(const CacheAttendArgs& A, const Req<kTile>& r, int b, int i, int t0) {
    const long long at = static_cast<long long>(b) * A.n;
    const int p = r.ctx + (A.depth ? min(max(A.depth[at + i], 0), A.n) : i);
    unsigned long long drafted = 0, context;
    if (!A.mask) {
        context = range64(0, r.ctx + min(i + 1, r.rows), t0);
    } else {
        context = range64(0, r.ctx, t0);
        const int off = t0 - r.ctx;             // drafted row at the tile's first token
        if (off + 64 > 0) {
            const int W = (A.n + 63) >> 6;
            const unsigned long long* m = A.mask + (at + i) * W;
            if (off < 0) {
                drafted = m[0] << -off;
            } else {
                const int w = off >> 6, s = off & 63;
                if (w < W) drafted = m[w] >> s;
                if (s && w + 1 < W) drafted |= m[w + 1] << (64 - s);
            }
            drafted &= range64(r.ctx, r.len, t0);
            if (A.window > 0)
                for (unsigned long long x = drafted; x; x &= x - 1) {
                    const int bit = __ffsll(static_cast<long long>(x)) - 1;
                    const int j = off + bit;
                    const int key = r.ctx + (A.depth ? min(max(A.depth[at + j], 0), A.n) : j);
                    if (p - key >= A.window && key >= A.sinks) drafted &= ~(1ull << bit);
                }
        }
    }
    if (A.window > 0)
        context &= range64(static_cast<long long>(p) - A.window + 1, 1ll << 40, t0) | range64(0, A.sinks, t0);
    return context | drafted;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int attend_device();                            // the current device, 64 where there is none
int attend_sms();                               // its SMs

// the workspace's arrays for `slots` parts of `rows` rows
struct AttendLayout {
    size_t ml, part, bytes;
    AttendLayout(int slots, int rows, int D) {
        auto up = [](size_t x) { return (x + 255) / 256 * 256; };
        ml = SPEC_CACHE_WS_CONTROL;
        part = ml + up(static_cast<size_t>(slots) * rows * 16);
        bytes = part + static_cast<size_t>(slots) * rows * D * 4;
    }
};

// many rows a kv head: tcgen05 (spec_cache_attend_tc.cu)
size_t attend_tc_ws(int D);
long long attend_tc_tiles(int R, int hkv, long long positions);
cudaError_t attend_tc_run(const CacheAttendArgs& A, cudaStream_t st);

}  // namespace spec
