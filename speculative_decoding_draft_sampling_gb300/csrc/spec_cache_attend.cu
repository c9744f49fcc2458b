// spec_cache_attend.cu -- attention of drafted rows over the paged 4-bit cache.
//
// [SD-survey] = "大模型投机解码：Medusa、MTP、EAGLE、DFlash、DDTree 与 DSpark"
// (Speculative decoding for LLMs: Medusa, MTP, EAGLE, DFlash, DDTree and
// DSpark), chzhyang.github.io, §5 "DDTree": drafted nodes take position id =
// depth and see only their ancestors.
//
// Mathematics.  For the R = n * G rows that read one kv head (G q heads each),
// scores x = scale * q.k, running maximum m, sum l = sum 2^((x - m) log2 e) and
// o = sum 2^(...) v, all fp32; parts of the keys are joined by their (m, l, o).
// The maximum is lazy: it moves, and o and l are rescaled, only when a score
// passes it by more than 2^8; until then weights may reach 2^8, which changes
// nothing in fp32 and costs one comparison a score.
//
// Work.  A unit is (request, kv head, block of 8 * NT rows); its keys are cut
// into tiles of 64 tokens.  All tiles of all units, in order, are dealt out in
// equal contiguous shares to a grid that fills the device once, whatever the
// requests' lengths; a unit that several CTAs share is joined by the last of
// them to finish, in CTA order (so the bits do not depend on timing).
//
// A warp takes every fourth tile of its CTA's share and is a pipeline of its
// own: one bulk copy (TMA) per page block into its ring in shared memory, no
// barrier with other warps.  Codes go from there straight into the registers
// of the tensor instruction (mma m16n8k16): scores are computed transposed,
// S^T = K Q^T and O^T = V^T P^T, so that the cache's side is the 16-row operand
// and the few rows of a request fill 8-column blocks instead of padding a
// 16-row tile.  A lane's 32 (D = 128) values of a key are 16 consecutive bytes
// of its row: the order of the k index is free as long as Q is laid out alike.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "../../include/spec_cache.h"
#include "spec_cache.cuh"
#include "spec_common.cuh"

namespace spec {

namespace {

constexpr int kAtWarps = 4;
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kTile = 64;                       // tokens a tile
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
    int grid;                                   // CTAs
    int row_tiles;                              // blocks of 8 * NT rows a (request, kv head)
    int min_tiles;                              // tiles worth a CTA
    float* ml;                                  // [2 * grid][8 * NT][4]: m, l, l of the rounded weights
    float* part;                                // [2 * grid][8 * NT][D]
    AttendCtrl* ctrl;
};

// What a request asks for.
struct Req {
    int ctx, rows, len;                         // len = ctx + rows
    int first;                                  // tiles [0, sink_tiles) and [first, tiles) hold visible keys
    int sink_tiles, tiles;                      // tiles: of the whole context
    int low;                                    // positions below are outside every row's window (sinks aside)
    __device__ __forceinline__ int visited() const { return max(1, sink_tiles + tiles - first); }
    __device__ __forceinline__ int real(int v) const { return v < sink_tiles ? v : first + (v - sink_tiles); }
};

__device__ __forceinline__ Req request(const CacheAttendArgs& A, int b) {
    Req r;
    const long long room = static_cast<long long>(A.tab.width) << A.pool.p_shift;
    r.ctx = static_cast<int>(min(static_cast<long long>(max(A.ctx[b], 0)), room));
    r.rows = A.rows ? min(max(A.rows[b], 0), A.n) : A.n;
    r.len = r.rows ? r.ctx + r.rows : 0;
    r.tiles = (r.len + kTile - 1) / kTile;
    r.low = 0;
    r.sink_tiles = 0;
    r.first = 0;
    if (A.window > 0) {
        r.low = max(0, r.ctx - A.window + 1);
        r.sink_tiles = min(r.tiles, (min(A.sinks, r.len) + kTile - 1) / kTile);
        r.first = min(max(r.low / kTile, r.sink_tiles), r.tiles);
    }
    return r;
}

// tiles of one kv head of a request: blocks of rows that hold no row cost one
__device__ __forceinline__ int head_work(const CacheAttendArgs& A, const Req& r, int row_tiles, int rows_a_tile) {
    const int live = (r.rows * A.G + rows_a_tile - 1) / rows_a_tile;
    return live * r.visited() + (row_tiles - live);
}

// ---------------------------------------------------------------------------
// codes to bf16
// ---------------------------------------------------------------------------
// Two codes that lie 16 bits apart (at 4i and 4i + 16) as bf16: placed at bits
// 3..6 of the significand under the exponent of 1 they are 1 + code/16, and one
// fused multiply-add with (s, -1.5 s) gives (code - 8)/16 * s, exactly (a scale
// has five significant bits, so 1.5 s fits too).  The factor 16 goes into the
// softmax scale (K) and the final division (V).
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t s2, uint32_t c2) {
    uint32_t t;
    if constexpr (I == 0) t = w << 3;
    else t = w >> (4 * I - 3);
    t = (t & 0x00780078u) | 0x3F803F80u;
    uint32_t v;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(t), "r"(s2), "r"(c2));
    return v;
}
__device__ __forceinline__ uint32_t minus1_5(uint32_t s2) {
    uint32_t v;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(s2), "r"(0xBFC0BFC0u));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
template <int kWords>
__device__ __forceinline__ void lds(uint32_t (&w)[kWords], uint32_t a) {
    if constexpr (kWords == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
    else if constexpr (kWords == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t v;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(v) : "r"(x));
    return v;
}

// bits [a, b) of a tile that starts at t0
__device__ __forceinline__ unsigned long long range64(long long a, long long b, long long t0) {
    const int lo = static_cast<int>(min(max(a - t0, 0ll), 64ll)), hi = static_cast<int>(min(max(b - t0, 0ll), 64ll));
    if (hi <= lo) return 0;
    return (hi == 64 ? ~0ull : (1ull << hi) - 1ull) & ~((1ull << lo) - 1ull);
}

// The keys of the tile at t0 that row i of request b sees.
__device__ __forceinline__ unsigned long long seen64(const CacheAttendArgs& A, const Req& r, int b, int i, int t0) {
    const long long at = static_cast<long long>(b) * A.n;
    const int p = r.ctx + (A.depth ? min(max(A.depth[at + i], 0), A.n) : i);
    unsigned long long drafted = 0, context;
    if (!A.mask) {
        context = range64(0, r.ctx + min(i + 1, r.rows), t0);
    } else {
        context = range64(0, r.ctx, t0);
        const int off = t0 - r.ctx;             // drafted row at the tile's first token
        if (off + kTile > 0) {
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
// the kernel
// ---------------------------------------------------------------------------
template <int D, int NT>
struct AttendCfg {
    static constexpr int kStageBytes = kTile * CacheBlock<D>::kTok;
    static constexpr int kCtas = 3;                         // resident CTAs an SM
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kMB = 2;                           // 16-token blocks whose scores are held at once
    static constexpr int kRows = 8 * NT;
    static constexpr int kPad = D + 4;                      // pitch of a row when warps are joined
    static constexpr int kRing = kAtWarps * kStages * kStageBytes;
    static constexpr int kJoin = kAtWarps * kRows * (kPad + 3) * 4;
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

template <int D, int NT, int P>
__global__ void __launch_bounds__(kAtThreads, AttendCfg<D, NT>::kCtas)
cache_attend_kernel(const __grid_constant__ CacheAttendArgs A, const __grid_constant__ AttendPlan L) {
    using Cfg = AttendCfg<D, NT>;
    using Blk = CacheBlock<D>;
    constexpr int kS = Cfg::kStages, kMB = Cfg::kMB, kRows = Cfg::kRows, kPad = Cfg::kPad;
    constexpr int kKW = D / 32;                 // words of a key that a lane holds
    constexpr int kVW = D / 64;                 // words of a value row that a lane holds
    constexpr int kMT = D / 16;                 // 16-row blocks of O^T
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kAtWarps][kS];
    __shared__ long long s_sum[kAtWarps];
    __shared__ long long s_found[2];
    __shared__ int s_last;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);    // uniform to the compiler too
    const int r8 = lane >> 2, c4 = lane & 3;
    const int H = A.pool.heads;
    constexpr int p_shift = P == 64 ? 6 : P == 32 ? 5 : 4;
    constexpr int ppt = kTile / P;              // page blocks a tile
    constexpr int per = 32 / ppt;               // tiles whose page ids a warp holds
    constexpr int block_bytes = Blk::bytes(P);

    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < kS; ++s) mbar_init(&full[warp][s], 1);
        fence_mbar_init();
    }

    // ---- this CTA's share: [lo, hi) of all tiles ---------------------------
    auto block_sum = [&](long long v) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_sum[warp] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < kAtWarps; ++w) v += s_sum[w];
        __syncthreads();
        return v;
    };
    auto work_of = [&](int b) {
        return b < A.B ? static_cast<long long>(H) * head_work(A, request(A, b), L.row_tiles, kRows) : 0ll;
    };
    long long mine = 0;
    for (int b = tid; b < A.B; b += kAtThreads) mine += work_of(b);
    const long long total = block_sum(mine);
    const long long units = static_cast<long long>(A.B) * H * L.row_tiles;
    long long want = total / L.min_tiles;
    if (want > units * 64) want = units * 64;   // what joins a unit must stay small beside it
    const int active = static_cast<int>(min(static_cast<long long>(gridDim.x), max(want, 1ll)));
    const int cta = blockIdx.x;
    if (cta >= active) return;
    auto start_of = [&](long long c) { return c * total / active; };
    const long long lo = start_of(cta), hi = start_of(cta + 1);
    // the request that holds tile lo, and where its tiles start
    {
        long long before = 0;
        for (int b0 = 0; b0 < A.B; b0 += kAtThreads) {
            const long long v = work_of(b0 + tid);
            long long inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            if (lane == 31) s_sum[warp] = inc;
            __syncthreads();
            long long base = before, all = 0;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) {
                if (w < warp) base += s_sum[w];
                all += s_sum[w];
            }
            const long long from = base + inc - v;
            if (v > 0 && from <= lo && lo < from + v) {
                s_found[0] = b0 + tid;
                s_found[1] = from;
            }
            __syncthreads();
            before += all;
            if (lo < before) break;
        }
    }
    int b = static_cast<int>(s_found[0]);
    long long b_from = s_found[1];
    Req rq = request(A, b);

    bool dead = false;                          // a wait gave up: nothing more is copied or waited for
    uint32_t phase[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) phase[s] = 0;
    unsigned char* ring = smem + warp * kS * Cfg::kStageBytes;
    const uint32_t ring_u32 = smem_u32(ring);
    const int tok = r8 ^ ((r8 >> 1) & 1);       // the token (of 8) that is row r8 of S^T
    const int tv0 = (2 * c4) ^ (c4 & 1);        // tokens 2c and 2c+1 of P^T's rows
    const int tv1 = (2 * c4 + 1) ^ (c4 & 1);
    // where a lane's words and scales lie from the start of a block's 16 tokens
    const uint32_t k_at = tok * Blk::kRow + c4 * (D / 8);
    const uint32_t ks_at = P * Blk::kRow + tok * Blk::kScl + (D == 128 ? c4 : c4 >> 1) * 2;
    const uint32_t v_at = Blk::v_codes(P) + r8 * (D / 16), vs_at = Blk::v_codes(P) + P * Blk::kRow + (D == 128 ? r8 >> 1 : r8 >> 2) * 2;
    const uint32_t v0_at = v_at + tv0 * Blk::kRow, v1_at = v_at + tv1 * Blk::kRow;
    const uint32_t vs0_at = vs_at + tv0 * Blk::kScl, vs1_at = vs_at + tv1 * Blk::kScl;

    for (long long pos = lo; pos < hi;) {
        // ---- the unit that holds tile pos -----------------------------------
        long long per_head = head_work(A, rq, L.row_tiles, kRows);
        while (pos >= b_from + per_head * H) {
            b_from += per_head * H;
            rq = request(A, ++b);
            per_head = head_work(A, rq, L.row_tiles, kRows);
        }
        const int h = static_cast<int>((pos - b_from) / per_head);
        const long long h_from = b_from + h * per_head;
        const int live = (rq.rows * A.G + kRows - 1) / kRows;
        const int visited = rq.visited();
        const long long in_head = pos - h_from;
        int rt, nt_unit;
        long long u_from;
        if (in_head < static_cast<long long>(live) * visited) {
            rt = static_cast<int>(in_head / visited);
            nt_unit = visited;
            u_from = h_from + static_cast<long long>(rt) * visited;
        } else {
            rt = live + static_cast<int>(in_head - static_cast<long long>(live) * visited);
            nt_unit = 1;
            u_from = pos;
        }
        const int v0 = static_cast<int>(pos - u_from);
        const int v1 = static_cast<int>(min(static_cast<long long>(nt_unit), hi - u_from));
        const int row0 = rt * kRows;
        const int live_rows = min(max(rq.rows * A.G - row0, 0), kRows);

        // ---- page ids: a lane per page block of the coming tiles ------------
        int entry = -2;
        auto load_entries = [&](int k0) {
            const int v = v0 + warp + kAtWarps * (k0 + lane / ppt);
            entry = -2;
            if (v < v1) {
                const int t = rq.real(v) * kTile + ((lane % ppt) << p_shift);
                const bool need = t < rq.len && (A.window == 0 || t < A.sinks || t + P > rq.low);
                if (need) {
                    entry = cache_page(A.tab, A.pool.num_pages, p_shift, b, t);
                    if (entry < 0 && A.status) atomicOr(A.status + b, SPEC_ST_BAD_PAGE);
                }
            }
        };
        uint32_t fifo = 0;                      // per tile in flight: which page blocks are there
        const int tiles = live_rows > 0 && v1 - v0 > warp ? (v1 - v0 - warp + kAtWarps - 1) / kAtWarps : 0;   // this warp's
        auto issue = [&](int k, int s, int depth) {
            if (k % per == 0) load_entries(k);
            const int g = (k % per) * ppt;
            const unsigned got = __ballot_sync(0xffffffffu, entry >= 0);
            const uint32_t there = (got >> g) & ((1u << ppt) - 1u);
            fifo |= there << (4 * depth);
            if (!dead) {
                if (lane == 0) mbar_expect_tx(&full[warp][s], __popc(there) * block_bytes);
                __syncwarp();
                if (lane >= g && lane < g + ppt && entry >= 0)
                    tma_load_1d(ring + s * Cfg::kStageBytes + (lane - g) * block_bytes,
                                A.pool.base + entry * A.pool.page_stride + h * A.pool.head_stride, block_bytes,
                                &full[warp][s]);
            }
        };
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (s < tiles) issue(s, s, s);

        // ---- Q, laid out like the keys' words -------------------------------
        uint32_t qf[NT][D / 16][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rho = row0 + nt * 8 + r8;
            const bool on = nt * 8 + r8 < live_rows;
            const int i = on ? rho / A.G : 0, g = on ? rho % A.G : 0;
            const uint16_t* q = A.q + b * A.q_bs + i * A.q_rs + (static_cast<long long>(h) * A.G + g) * A.q_hs +
                                c4 * (D / 4);
#pragma unroll
            for (int w = 0; w < kKW; ++w) {
                uint32_t x[4] = {0, 0, 0, 0};
                if (on) {
                    if (A.aligned) {
                        const uint4 t = *reinterpret_cast<const uint4*>(q + 8 * w);
                        x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = q[8 * w + 2 * e] | (static_cast<uint32_t>(q[8 * w + 2 * e + 1]) << 16);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    qf[nt][2 * w + u][0] = __byte_perm(x[u], x[u + 2], 0x5410);
                    qf[nt][2 * w + u][1] = __byte_perm(x[u], x[u + 2], 0x7632);
                }
            }
        }

        float o[kMT][NT][4], m[NT][2], l[NT][2], lr[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kNoMax;
            l[nt][0] = l[nt][1] = 0.0f;
            lr[nt][0] = lr[nt][1] = lr[nt][2] = lr[nt][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < kMT; ++j) o[j][nt][0] = o[j][nt][1] = o[j][nt][2] = o[j][nt][3] = 0.0f;
        }
        const float cs = A.scale * kLog2e * 16.0f;

        // ---- the tiles -------------------------------------------------------
        int s = 0;
        for (int k = 0; k < tiles; ++k) {
            const int t0 = rq.real(v0 + warp + kAtWarps * k) * kTile;
            const uint32_t there = fifo & 15u;
            fifo >>= 4;
            if (!dead) {
                uint32_t ph = 0;
#pragma unroll
                for (int q = 0; q < kS; ++q)
                    if (q == s) { ph = phase[q]; phase[q] ^= 1u; }
                if (!mbar_wait(&full[warp][s], ph)) {
                    dead = true;
                    if (lane == 0) atomicOr(&L.ctrl->error, SPEC_WS_ERR_WAIT);
                }
                dead = __any_sync(0xffffffffu, dead);
            }
            // which keys this warp's rows see; every key of most tiles
            const bool masked = t0 + kTile > rq.ctx || there != (1u << ppt) - 1u ||
                                (A.window > 0 && t0 + kTile > A.sinks && t0 < rq.low + A.n);
            unsigned long long seen = 0, any = ~0ull;
            if (masked) {
                if (lane < live_rows) seen = seen64(A, rq, b, (row0 + lane) / A.G, t0);
#pragma unroll 1
                for (int q = 0; q < ppt; ++q)
                    if (!(there >> q & 1u)) seen &= ~range64(q << p_shift, (q + 1) << p_shift, 0);
                any = seen;
                any = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any)) |
                      static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32))) << 32;
            }
            const uint32_t stage = ring_u32 + s * Cfg::kStageBytes;
            auto part = [&](auto is_masked, int g) {
                constexpr bool kMasked = decltype(is_masked)::value;
                float x[kMB][NT][4];
                // S^T = K Q^T
#pragma unroll
                for (int mb = 0; mb < kMB; ++mb) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) x[mb][nt][0] = x[mb][nt][1] = x[mb][nt][2] = x[mb][nt][3] = 0.0f;
                    const int t = (g * kMB + mb) * 16, slot = t & (P - 1);
                    const uint32_t blk = stage + (t >> p_shift) * block_bytes;
                    const uint32_t kr = blk + slot * Blk::kRow + k_at, sc = blk + slot * Blk::kScl + ks_at;
                    uint32_t wa[kKW], wb[kKW];
                    lds(wa, kr);
                    lds(wb, kr + 8 * Blk::kRow);
                    const uint32_t sa = lds16(sc) * 0x10001u, sb = lds16(sc + 8 * Blk::kScl) * 0x10001u;
                    const uint32_t ca = minus1_5(sa), cb = minus1_5(sb);
#pragma unroll
                    for (int w = 0; w < kKW; ++w) {
                        const uint32_t a0[4] = {codes2<0>(wa[w], sa, ca), codes2<0>(wb[w], sb, cb),
                                                codes2<1>(wa[w], sa, ca), codes2<1>(wb[w], sb, cb)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma(x[mb][nt], a0, qf[nt][2 * w][0], qf[nt][2 * w][1]);
                        const uint32_t a1[4] = {codes2<2>(wa[w], sa, ca), codes2<2>(wb[w], sb, cb),
                                                codes2<3>(wa[w], sa, ca), codes2<3>(wb[w], sb, cb)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma(x[mb][nt], a1, qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
                    }
                }
                if constexpr (kMasked) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = nt * 8 + 2 * c4 + e;
                            const unsigned long long v =
                                __shfl_sync(0xffffffffu, seen, row) >> (g * kMB * 16 + tok);
#pragma unroll
                            for (int mb = 0; mb < kMB; ++mb) {
                                if (!(v >> (16 * mb) & 1)) x[mb][nt][e] = -CUDART_INF_F;
                                if (!(v >> (16 * mb + 8) & 1)) x[mb][nt][2 + e] = -CUDART_INF_F;
                            }
                        }
                }
                // the running maximum, moved only when it must be
                bool move = false;
                float top[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
#pragma unroll
                        for (int mb = 1; mb < kMB; ++mb) t = fmaxf(t, fmaxf(x[mb][nt][e], x[mb][nt][2 + e]));
                        top[nt][e] = t * cs;
                        move |= top[nt][e] > m[nt][e] + kSlack;
                    }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = top[nt][e];
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                            const float mn = fmaxf(m[nt][e], t);
                            const float f = exp2_fast(m[nt][e] - mn);
                            m[nt][e] = mn;
                            l[nt][e] *= f;
                            lr[nt][e] *= f;
#pragma unroll
                            for (int j = 0; j < kMT; ++j) {
                                o[j][nt][e] *= f;
                                o[j][nt][2 + e] *= f;
                            }
                        }
                }
                // weights, as the 16 x 8 operand P^T.  They are rounded to bf16
                // for the tensor cores (2^-8 each at most, as the output's own
                // rounding); lse takes their sum before that, the output is
                // divided by the sum of the rounded ones, so that what rounding
                // they have in common cancels (one dominant key: all of it).
                // A tile with masked keys, where a row may see only a few, adds a
                // second term with what rounding took from the first.
                uint32_t pf[kMB][NT][2], pl[kMasked ? kMB : 1][NT][2];
#pragma unroll
                for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = exp2_fast(fmaf(x[mb][nt][e], cs, -m[nt][e & 1]));
                        l[nt][0] += p[0] + p[2];
                        l[nt][1] += p[1] + p[3];
                        const uint32_t lo = pack_bf16(p[0], p[1]), hi = pack_bf16(p[2], p[3]);
                        pf[mb][nt][0] = transpose8x8(lo);
                        pf[mb][nt][1] = transpose8x8(hi);
                        if constexpr (kMasked) {
                            pl[mb][nt][0] = transpose8x8(pack_bf16(p[0] - __uint_as_float(lo << 16),
                                                                   p[1] - __uint_as_float(lo & 0xffff0000u)));
                            pl[mb][nt][1] = transpose8x8(pack_bf16(p[2] - __uint_as_float(hi << 16),
                                                                   p[3] - __uint_as_float(hi & 0xffff0000u)));
                        }
                    }
                // O^T += V^T P^T, and a row of ones for the sum
                const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
                for (int mb = 0; mb < kMB; ++mb) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(lr[nt], ones, pf[mb][nt][0], pf[mb][nt][1]);
                        if constexpr (kMasked) mma(lr[nt], ones, pl[mb][nt][0], pl[mb][nt][1]);
                    }
                    const int t = (g * kMB + mb) * 16, slot = t & (P - 1);
                    const uint32_t blk = stage + (t >> p_shift) * block_bytes;
                    const uint32_t vr = blk + slot * Blk::kRow, vs = blk + slot * Blk::kScl;
                    uint32_t w0[kVW], w1[kVW], w2[kVW], w3[kVW];
                    lds(w0, vr + v0_at);
                    lds(w1, vr + v1_at);
                    lds(w2, vr + v0_at + 8 * Blk::kRow);
                    lds(w3, vr + v1_at + 8 * Blk::kRow);
                    uint32_t s0 = lds16(vs + vs0_at), s1 = lds16(vs + vs1_at);
                    uint32_t s2 = lds16(vs + vs0_at + 8 * Blk::kScl), s3 = lds16(vs + vs1_at + 8 * Blk::kScl);
                    if constexpr (kMasked) {    // what no row sees may be anything, NaN among it
                        const uint32_t a = static_cast<uint32_t>(any >> t);
                        s0 = a >> tv0 & 1 ? s0 : 0;
                        s1 = a >> tv1 & 1 ? s1 : 0;
                        s2 = a >> (tv0 + 8) & 1 ? s2 : 0;
                        s3 = a >> (tv1 + 8) & 1 ? s3 : 0;
                    }
                    const uint32_t sa = s0 | s1 << 16, sb = s2 | s3 << 16;
                    const uint32_t ca = minus1_5(sa), cb = minus1_5(sb);
#pragma unroll
                    for (int w = 0; w < kVW; ++w) {
                        // token pairs side by side: elements 0..3 and 4..7 of the word
                        const uint32_t a_lo = __byte_perm(w0[w], w1[w], 0x5410), a_hi = __byte_perm(w0[w], w1[w], 0x7632);
                        const uint32_t b_lo = __byte_perm(w2[w], w3[w], 0x5410), b_hi = __byte_perm(w2[w], w3[w], 0x7632);
#define SPEC_PV(I)                                                                                        \
    {                                                                                                     \
        const uint32_t a[4] = {codes2<I>(a_lo, sa, ca), codes2<I>(a_hi, sa, ca), codes2<I>(b_lo, sb, cb), \
                               codes2<I>(b_hi, sb, cb)};                                                  \
        _Pragma("unroll") for (int nt = 0; nt < NT; ++nt) {                                               \
            mma(o[4 * w + I][nt], a, pf[mb][nt][0], pf[mb][nt][1]);                                       \
            if constexpr (kMasked) mma(o[4 * w + I][nt], a, pl[mb][nt][0], pl[mb][nt][1]);                \
        }                                                                                                 \
    }
                        SPEC_PV(0)
                        SPEC_PV(1)
                        SPEC_PV(2)
                        SPEC_PV(3)
#undef SPEC_PV
                    }
                }
            };
            if (masked) {
#pragma unroll 1
                for (int g = 0; g < 4 / kMB; ++g) part(std::true_type{}, g);
            } else {
#pragma unroll 1
                for (int g = 0; g < 4 / kMB; ++g) part(std::false_type{}, g);
            }
            __syncwarp();
            if (k + kS < tiles) issue(k + kS, s, kS - 1);
            s = s + 1 == kS ? 0 : s + 1;
        }

        // ---- join the warps ---------------------------------------------------
        // value (row d of O^T): d = (D/8) r8 + 8 w + i (+4) lies in block j = 4w + i;
        // it is stored at place (half * kMT + j) * 8 + r8
        __syncthreads();                        // every warp is done with its ring
        float* jo = reinterpret_cast<float*>(smem);                         // [warp][row][kPad]
        float* jm = jo + kAtWarps * kRows * kPad;                           // [warp][row][3]: m, l, l of the rounded weights
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = l[nt][e];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                const int row = warp * kRows + nt * 8 + 2 * c4 + e;
                if (r8 == 0) {
                    jm[row * 3] = m[nt][e];
                    jm[row * 3 + 1] = t;
                    jm[row * 3 + 2] = lr[nt][e];
                }
#pragma unroll
                for (int j = 0; j < kMT; ++j) {
                    jo[row * kPad + j * 8 + r8] = o[j][nt][e];
                    jo[row * kPad + (kMT + j) * 8 + r8] = o[j][nt][2 + e];
                }
            }
        __syncthreads();
        const bool whole = v0 == 0 && v1 == nt_unit;
        // the CTA that holds the unit's first tile, and how many share it
        int c0 = cta, parts = 1;
        if (!whole) {
            auto cta_of = [&](long long x) {
                int c = static_cast<int>(x * active / total);
                while (start_of(c + 1) <= x) ++c;
                while (start_of(c) > x) --c;
                return c;
            };
            c0 = cta_of(u_from);
            parts = cta_of(u_from + nt_unit - 1) - c0 + 1;
        }
        const int slot = 2 * cta + (c0 == cta ? 1 : 0);
        // An item is eight neighbouring values of a row: (row, r8, w).
        constexpr int kItems = kRows * (D / 8);
        const int rows_here = min(kRows, A.n * A.G - row0);     // rows of the output in this block
        auto emit = [&](int row, int item, const float (&v)[8], float mm, float ls, float lrs) {
            const int rho = row0 + row, i = rho / A.G, g = rho % A.G;
            const long long at = (static_cast<long long>(b) * A.n + i) * A.hq + static_cast<long long>(h) * A.G + g;
            const bool on = row < live_rows && ls != 0.0f;
            const float f = on ? 16.0f / lrs : 0.0f;
            uint4 u;
            u.x = on ? pack_bf16(v[0] * f, v[1] * f) : 0;
            u.y = on ? pack_bf16(v[2] * f, v[3] * f) : 0;
            u.z = on ? pack_bf16(v[4] * f, v[5] * f) : 0;
            u.w = on ? pack_bf16(v[6] * f, v[7] * f) : 0;
            *reinterpret_cast<uint4*>(A.out + at * D + item * 8) = u;
            if (A.lse && item == 0) A.lse[at] = on ? (mm + log2f(ls)) * kLn2 : -CUDART_INF_F;
        };
#pragma unroll
        for (int x = tid; x < kItems; x += kAtThreads) {
            const int row = x / (D / 8), item = x % (D / 8);    // values 8 item .. 8 item + 7 of the row
            const int rr = item / kVW, w8 = item % kVW;
            float mm = kNoMax;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) mm = fmaxf(mm, jm[(w * kRows + row) * 3]);
            float v[8] = {}, ls = 0.0f, lrs = 0.0f;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) {
                const float* ml = jm + (w * kRows + row) * 3;
                const float f = exp2_fast(ml[0] - mm);
                ls += f * ml[1];
                lrs += f * ml[2];
                const float* src = jo + (w * kRows + row) * kPad + w8 * 32 + rr;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += f * src[(e >= 4 ? kMT * 8 : 0) + (e & 3) * 8];
            }
            if (whole) {
                if (row < rows_here) emit(row, item, v, mm, ls, lrs);
            } else {
                float4* to = reinterpret_cast<float4*>(L.part + (static_cast<long long>(slot) * kRows + row) * D + item * 8);
                __stcg(to, make_float4(v[0], v[1], v[2], v[3]));
                __stcg(to + 1, make_float4(v[4], v[5], v[6], v[7]));
                if (item == 0)
                    __stcg(reinterpret_cast<float4*>(L.ml) + slot * kRows + row, make_float4(mm, ls, lrs, 0.0f));
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const bool last = atomicAdd(&L.ctrl->arrived[c0], 1u) == static_cast<uint32_t>(parts - 1);
                if (last) L.ctrl->arrived[c0] = 0;
                s_last = last;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int x = tid; x < rows_here * (D / 8); x += kAtThreads) {
                    const int row = x / (D / 8), item = x % (D / 8);
                    auto place = [&](int c) { return (2ll * (c0 + c) + (c == 0 ? 1 : 0)) * kRows + row; };
                    float mm = kNoMax;
#pragma unroll 4
                    for (int c = 0; c < parts; ++c) mm = fmaxf(mm, __ldcg(L.ml + place(c) * 4));
                    float v[8] = {}, ls = 0.0f, lrs = 0.0f;
#pragma unroll 4
                    for (int c = 0; c < parts; ++c) {
                        const float4 ml = __ldcg(reinterpret_cast<const float4*>(L.ml) + place(c));
                        const float4* from = reinterpret_cast<const float4*>(L.part + place(c) * D + item * 8);
                        const float4 a = __ldcg(from), z = __ldcg(from + 1);
                        const float f = exp2_fast(ml.x - mm);
                        ls += f * ml.y;
                        lrs += f * ml.z;
                        v[0] += f * a.x; v[1] += f * a.y; v[2] += f * a.z; v[3] += f * a.w;
                        v[4] += f * z.x; v[5] += f * z.y; v[6] += f * z.z; v[7] += f * z.w;
                    }
                    emit(row, item, v, mm, ls, lrs);
                }
            }
        }
        // the ring is copied into again: order the joins' accesses before it
        fence_proxy_async_smem();
        __syncthreads();
        pos = u_from + v1;
    }
}

int sm_count() {
    int d = 0, v = 0;
    if (cudaGetDevice(&d) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    return v;
}

// blocks of 8 rows a warp holds at once
int row_blocks(int R) { return R <= 8 ? 1 : 2; }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
    size_t ml, part, bytes;
};
Layout layout_of(int grid, int NT, int D) {
    Layout y;
    y.ml = SPEC_CACHE_WS_CONTROL;
    y.part = y.ml + up256(static_cast<size_t>(grid) * 2 * 8 * NT * 4 * 4);
    y.bytes = y.part + static_cast<size_t>(grid) * 2 * 8 * NT * D * 4;
    return y;
}

template <int D, int NT, int P>
cudaError_t attend(const CacheAttendArgs& A, cudaStream_t st) {
    using Cfg = AttendCfg<D, NT>;
    const int grid = min(sm_count() * Cfg::kCtas, kMaxGrid);
    const Layout y = layout_of(grid, NT, D);
    AttendPlan L;
    L.grid = grid;
    L.row_tiles = (A.n * A.G + Cfg::kRows - 1) / Cfg::kRows;
    L.min_tiles = 2 * kAtWarps;
    unsigned char* ws = static_cast<unsigned char*>(A.ws);
    L.ctrl = reinterpret_cast<AttendCtrl*>(ws);
    L.ml = reinterpret_cast<float*>(ws + y.ml);
    L.part = reinterpret_cast<float*>(ws + y.part);
    const cudaError_t e = cudaFuncSetAttribute(cache_attend_kernel<D, NT, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg::kSmem);
    if (e != cudaSuccess) return e;
    cache_attend_kernel<D, NT, P><<<grid, kAtThreads, Cfg::kSmem, st>>>(A, L);
    return cudaGetLastError();
}

}  // namespace

size_t cache_attend_ws(int B, int n, int hq, int hkv, int D) {
    (void)B;
    const int NT = row_blocks(n * (hq / hkv));
    return layout_of(min(sm_count() * 3, kMaxGrid), NT, D).bytes;
}

namespace {

template <int D, int NT>
cudaError_t attend_pages(const CacheAttendArgs& A, cudaStream_t st) {
    switch (A.pool.P) {
        case 16: return attend<D, NT, 16>(A, st);
        case 32: return attend<D, NT, 32>(A, st);
        default: return attend<D, NT, 64>(A, st);
    }
}

}  // namespace

cudaError_t cache_attend_run(const CacheAttendArgs& A, cudaStream_t st) {
    const int NT = row_blocks(A.n * A.G);
    if (A.pool.D == 128) return NT == 1 ? attend_pages<128, 1>(A, st) : attend_pages<128, 2>(A, st);
    return NT == 1 ? attend_pages<64, 1>(A, st) : attend_pages<64, 2>(A, st);
}

}  // namespace spec
