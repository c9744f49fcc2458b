// spec_cache_attend_tc.cu -- attention over the paged 4-bit cache for requests
// with many rows a kv head (draft trees, long chains): tcgen05.
//
// [SD-survey] = "大模型投机解码：Medusa、MTP、EAGLE、DFlash、DDTree 与 DSpark"
// (Speculative decoding for LLMs: Medusa, MTP, EAGLE, DFlash, DDTree and
// DSpark), chzhyang.github.io, §5 "DDTree".
//
// The mathematics is that of spec_cache_attend.cu; the shape is the other way
// round: rows are the 128-row operand, S = Q K^T and O = P V, so that a thread
// owns a row of S in tensor memory and the softmax needs no exchange.
//
// One CTA an SM, in five warp groups (the fifth for one thread) that never wait
// for each other all at once:
//   warps 8-11   read the codes of a tile's 128 keys, a token a thread, while the
//                tile before waits, and write them as bf16 into shared memory
//                (128-byte swizzle); warps 12-15 the same for the values;
//   warp 16      one thread issues the tensor work: S_g = Q K^T (both in shared
//                memory) and O_g += P_g V with P_g in tensor memory where S_g was;
//   warps 0-3, 4-7  two softmax groups, g = 0 and 1, with 128 of a unit's 256 rows
//                each and their own S, P, O in tensor memory, so that one group's
//                exponentials run beside the other's products.  A unit of up to 128
//                rows is group 0's alone; its tiles take the two S in turn.
// What bounds it, a tile of 128 tokens and 256 rows at D = 128: shared memory, 64 KB
// written and 192 KB read by the tensor core at 128 bytes a cycle, and the tensor core
// itself are busy 2048 cycles each; a tile takes 5400, because a group's products and
// its exponentials follow one another (32 requests of 8192 down to 2240 tokens, trees of
// 64 down to 33 nodes, 4 heads a kv head: 212 to 221 us, 600 to 628 TFLOP/s; rows that are
// not there are multiplied too).  What shortens one of the two but adds code or
// registers lost: scores read once with a late rescale 237 us, a second tile of codes
// in flight in registers 229, or in shared memory 226.  With up to 128 rows both groups
// could take the tiles in turn: 183 us against 154 at 128 rows, for the join of
// their O and its registers.
#include <atomic>
#include <type_traits>

#include "spec_cache_attend.cuh"

namespace spec {

namespace {

constexpr int kTok = 128;                       // tokens a tile
constexpr int kWarps = 20;
constexpr int kThreads = 32 * kWarps;
constexpr int kMmaWarp = 16;
// Registers a thread: 96 at launch (640 threads), then moved from the decoders and
// the issuing group to the softmax: 256 * 56 + 128 * 72 + 256 * 144 = 60416 of the
// 61440 that the block was launched with.
constexpr int kRegsDecode = 56, kRegsIssue = 72, kRegsSoftmax = 144;
static_assert(256 * kRegsDecode + 128 * kRegsIssue + 256 * kRegsSoftmax <= 96 * kThreads, "register shares");

constexpr int kRows = 256;                      // rows a unit

template <int D>
struct TcCfg {
    static constexpr int kTileBytes = kTok * D * 2;         // a tile's keys or values in bf16
    static constexpr int kQBytes = 128 * D * 2;             // 128 rows of Q
    static constexpr int kSmem = 4 * kTileBytes + 2 * kQBytes + 1024;
};

// tensor memory, in columns: S (P) of the groups, then O
constexpr uint32_t kS(int g) { return 128 * g; }
constexpr uint32_t kO(int g) { return 256 + 128 * g; }

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tc_alloc(uint32_t* to, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(to)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_dealloc(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(at), "r"(columns));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}
// A matrix in shared memory in 64-element (128-byte) chunks of 128 rows, 128-byte
// swizzle: 8-row groups lie 1024 bytes apart, chunks 16384.  The low word of its
// descriptor holds the address (in 16 bytes) and the chunks' distance; the high
// word is constant.
__device__ __forceinline__ uint32_t tc_desc(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((16384u >> 4) << 16); }
#define TC_DESC_HIGH "0x40004040"       /* 1024 bytes, version 1, 128-byte swizzle */
// D = A B (+ D): both operands in shared memory, or A in tensor memory
template <bool kAdd>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, " TC_DESC_HIGH "};\n\tmov.b64 b, {%2, " TC_DESC_HIGH "};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
        :: "r"(d), "r"(a), "r"(b), "r"(idesc), "n"(kAdd ? 1 : 0) : "memory");
}
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, " TC_DESC_HIGH "};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
        :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_ld32(float (&x)[32], uint32_t at) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void tc_ld16(float (&x)[16], uint32_t at) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void tc_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :: "r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// kind::f16: fp32 accumulators, bf16 operands, M = 128, N columns; tb: B lies
// with its N index contiguous
constexpr uint32_t tc_idesc(int N, bool tb) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (tb ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(128 >> 4) << 24);
}
constexpr int kChunk = 16384;                   // bytes of 64 columns of 128 rows

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
// a load that stays where it stands
__device__ __forceinline__ uint32_t ld_now_u32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
// where piece j (8 elements, 16 bytes) of row r lies in such a matrix
__device__ __forceinline__ uint32_t piece_at(int r, int j) {
    return (j >> 3) * kChunk + r * 128 + (((j & 7) ^ (r & 7)) << 4);
}

template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
__device__ __forceinline__ void group_sync(int g) {
    asm volatile("bar.sync %0, 128;" :: "r"(1 + g) : "memory");
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
struct TcBars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];      // a tile's keys, values
    uint64_t s_full[2], p_full[2];              // by S
    uint64_t o_done[2], o_free[2];              // by group: a unit's last product, its O read
    uint64_t q_full, q_empty, pv_done;
    uint64_t drained;                           // all that the tensor core was given
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_attend_tc_kernel(const __grid_constant__ CacheAttendArgs A, const __grid_constant__ AttendPlan L) {
    using Cfg = TcCfg<D>;
    using Blk = CacheBlock<D>;
    constexpr int kTile = Cfg::kTileBytes;
    extern __shared__ unsigned char smem_raw[];
    __shared__ TcBars bars;
    __shared__ ShareScratch<kWarps> s_share;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_dead;
    __shared__ int s_last[2];

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int P = A.pool.P, p_shift = A.pool.p_shift;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t v_buf = base, k_buf = base + 2 * kTile, q_buf = base + 4 * kTile;

    after_earlier();
    Share<kTok, kWarps> share(A, L, s_share, kRows);
    if (share.lo() == share.hi()) return;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_full[i], 4);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 4);
            mbar_init(&bars.v_empty[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.o_done[i], 1);
            mbar_init(&bars.o_free[i], 4);
        }
        mbar_init(&bars.q_full, 8);
        mbar_init(&bars.q_empty, 1);
        mbar_init(&bars.pv_done, 1);
        mbar_init(&bars.drained, 1);
        fence_mbar_init();
        s_dead = 0;
    }
    if (warp == kMmaWarp) tc_alloc(&s_tmem, 512);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;

    // A wait that gives up ends all later ones at once: the roles run out.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (s_dead) return;
        if (!mbar_wait(bar, parity)) {
            s_dead = 1;
            atomicOr(&L.ctrl->error, SPEC_WS_ERR_WAIT);
        }
    };
    const uint32_t one2 = L.one2;

    if (warp >= 8 && warp < kMmaWarp) {
        // ---- codes to bf16 in shared memory: a token a thread ------------------
        regs_down<kRegsDecode>();
        const bool isv = warp >= 12;
        const int t = tid & 127;
        constexpr int kW = D / 8;               // words of a row's codes
        uint32_t done = 0;                      // tiles of the whole share so far
        for (long long pos = share.lo(); pos < share.hi();) {
            const Segment g = share.segment(pos);
            pos = g.u_from + g.v1;
            const Req<kTok> rq = share.rq;
            // the first position that a row's window reaches (trees: the
            // shallowest row's); what lies before may be anything
            int low = rq.low;
            if (A.window > 0 && A.depth) {
                int least = A.n;
                for (int i = lane; i < rq.rows; i += 32)
                    least = min(least, max(A.depth[static_cast<long long>(g.b) * A.n + i], 0));
                least = __reduce_min_sync(0xffffffffu, least);
                low = max(0, rq.ctx + least - A.window + 1);
            }
            const unsigned char* head = A.pool.base + g.h * A.pool.head_stride + (isv ? Blk::v_codes(P) : 0);
            // The page of tile k's token: looked up (load_page) a tile ahead and
            // judged (page_of) only when the codes are fetched, so that nothing waits
            // for the table.
            struct Page {
                int id;
                bool wanted;
            };
            auto load_page = [&](int k) {
                Page p;
                p.wanted = false;
                p.id = -1;
                if (k >= g.tiles) return p;
                const int at = rq.real(g.v0 + k) * kTok + t;
                p.wanted = rq.needs(A, at, at + 1) && !(A.window > 0 && at < low && at >= A.sinks);
                if (p.wanted && (at >> p_shift) < A.tab.width)
                    p.id = static_cast<int>(ld_now_u32(A.tab.table + g.b * A.tab.stride + (at >> p_shift)));
                return p;
            };
            auto page_of = [&](const Page& p) {
                const bool there = static_cast<unsigned>(p.id) < static_cast<unsigned>(A.pool.num_pages);
                if (p.wanted && !there && !isv && A.status) atomicOr(A.status + g.b, SPEC_ST_BAD_PAGE);
                return there ? p.id : -1;
            };
            struct Raw {
                uint32_t w[kW];
                uint32_t s[D / 64];
            };
            auto fetch = [&](Raw& r, int k, int page) {
#pragma unroll
                for (int i = 0; i < kW; ++i) r.w[i] = 0x88888888u;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) r.s[i] = 0;
                if (page < 0) return;
                const int slot = (rq.real(g.v0 + k) * kTok + t) & (P - 1);
                const unsigned char* blk = head + page * A.pool.page_stride;
                const uint4* c = reinterpret_cast<const uint4*>(blk + slot * Blk::kRow);
#pragma unroll
                for (int i = 0; i < kW / 4; ++i) {
                    const uint4 x = c[i];
                    r.w[4 * i] = x.x; r.w[4 * i + 1] = x.y; r.w[4 * i + 2] = x.z; r.w[4 * i + 3] = x.w;
                }
                const unsigned char* s = blk + P * Blk::kRow + slot * Blk::kScl;
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(s);
                    r.s[0] = x.x; r.s[1] = x.y;
                } else {
                    r.s[0] = *reinterpret_cast<const uint32_t*>(s);
                }
            };
            auto put = [&](const Raw& r) {
                const int buf = done & 1;
                wait(isv ? &bars.v_empty[buf] : &bars.k_empty[buf], ((done >> 1) & 1u) ^ 1u);
                const uint32_t to = (isv ? v_buf : k_buf) + buf * kTile;
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    const uint32_t s2 = __byte_perm(r.s[i >> 3], 0, (i >> 2) & 1 ? 0x3232 : 0x1010);
                    const uint32_t c2 = minus1_5(s2);
                    const uint32_t w = r.w[i];
                    sts128(to + piece_at(t, i), codes2<0>(w, s2, c2, one2), codes2<1>(w, s2, c2, one2),
                           codes2<2>(w, s2, c2, one2), codes2<3>(w, s2, c2, one2));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(isv ? &bars.v_full[buf] : &bars.k_full[buf]);
                ++done;
            };
            Raw a;
            Page next = load_page(0);
            fetch(a, 0, page_of(next));
            next = load_page(1);
#pragma unroll 1
            for (int k = 0; k < g.tiles; ++k) {
                put(a);
                if (k + 1 < g.tiles) fetch(a, k + 1, page_of(next));
                next = load_page(k + 2);
            }
        }
    } else if (warp >= kMmaWarp) {
        // ---- the tensor core's thread -----------------------------------------
        regs_down<kRegsIssue>();
        if (warp == kMmaWarp) {                 // (the whole warp keeps step, one thread issues)
            constexpr uint32_t kQk = tc_idesc(128, false), kPv = tc_idesc(D, true);
            uint32_t tiles_done = 0, segs = 0, p_seen[2] = {0, 0}, o_seen[2] = {0, 0};
            for (long long pos = share.lo(); pos < share.hi();) {
                const Segment g = share.segment(pos);
                pos = g.u_from + g.v1;
                if (g.tiles == 0) continue;
                const Req<kTok> rq = share.rq;
                // a job is a tile of 128 rows; it takes S i & 1, the group's with two
                // groups, else in turn
                const bool two = g.live_rows > 128;
                const int jobs = two ? 2 * g.tiles : g.tiles;
                int plain0, plain1;
                rq.plain(A, plain0, plain1);
                plain0 -= g.v0;
                plain1 -= g.v0;
                wait(&bars.q_full, segs & 1u);
                ++segs;
                // The products S = Q K^T of job i, if there is one, and of the job two
                // before it O += P V.  What they need is waited for with P last, and S
                // is committed first: the softmax waits for nothing else.
                auto step = [&](int i) {
                    const int pj = i - 2;
                    const int sb = i & 1;
                    const bool s_on = i < jobs, p_on = pj >= 0;
                    const int k_s = two ? i >> 1 : i, k_p = two ? pj >> 1 : pj, gr = two ? sb : 0;
                    const uint32_t n_s = tiles_done + k_s, n_p = tiles_done + k_p;
                    const bool first = k_p == 0, last = k_p == g.tiles - 1;
                    const bool lo = k_p < plain0 || k_p >= plain1;
                    const uint32_t q = __shfl_sync(0xffffffffu, tc_desc(q_buf + gr * Cfg::kQBytes), 0);
                    const uint32_t kb = __shfl_sync(0xffffffffu, tc_desc(k_buf + (n_s & 1) * kTile), 0);
                    const uint32_t vb = __shfl_sync(0xffffffffu, tc_desc(v_buf + (n_p & 1) * kTile), 0);
                    const uint32_t s_to = __shfl_sync(0xffffffffu, tmem + kS(sb), 0);
                    const uint32_t o_to = __shfl_sync(0xffffffffu, tmem + kO(gr), 0);
                    if (s_on && gr == 0) wait(&bars.k_full[n_s & 1], (n_s >> 1) & 1u);
                    if (p_on) {
                        if (gr == 0) wait(&bars.v_full[n_p & 1], (n_p >> 1) & 1u);
                        if (first) {            // O is written anew: the last unit's has been read
                            wait(&bars.o_free[gr], (o_seen[gr] & 1u) ^ 1u);
                            ++o_seen[gr];
                        }
                        wait(&bars.p_full[sb], p_seen[sb]++ & 1u);
                    }
                    tc_after();
                    if (elect_one()) {
                        if (p_on && !s_dead) {
#pragma unroll
                            for (int j = 0; j < kTok / 16; ++j)
                                tc_mma_ta(o_to, s_to + 16 * j, vb + j * 128, kPv, j > 0 ? 1u : !first);
                            if (lo)
#pragma unroll
                                for (int j = 0; j < kTok / 16; ++j)
                                    tc_mma_ta(o_to, s_to + 16 * j + 8, vb + j * 128, kPv, 1);
                        }
                        // (before S: whoever sees S of job i sees this of job i - 2)
                        if (p_on && !two) tc_commit(&bars.pv_done);
                        if (s_on) {
                            if (!s_dead) {
                                tc_mma<false>(s_to, q, kb, kQk);
#pragma unroll
                                for (int j = 1; j < D / 16; ++j) {
                                    const uint32_t at = ((j >> 2) * kChunk + (j & 3) * 32) >> 4;
                                    tc_mma<true>(s_to, q + at, kb + at, kQk);
                                }
                            }
#ifdef SPEC_TEST_HOOKS
                            if (!(g_test_drop && blockIdx.x == 0 && i == 0))
#endif
                            tc_commit(&bars.s_full[sb]);
                        }
                        if (p_on) {
                            if (last) tc_commit(&bars.o_done[gr]);
                            if (!two || gr == 1) tc_commit(&bars.v_empty[n_p & 1]);
                        }
                        if (s_on) {
                            if (!two || gr == 1) tc_commit(&bars.k_empty[n_s & 1]);
                            if (i == jobs - 1) tc_commit(&bars.q_empty);
                        }
                    }
                    __syncwarp();
                };
                for (int i = 0; i < jobs + 2; ++i) step(i);
                tiles_done += g.tiles;
            }
            // Products and arrivals on the barriers may still be on their way, those of
            // roles that gave up among them: tensor memory is freed, and the CTA ends,
            // only behind this last arrival.
            if (tiles_done > 0) {
                if (elect_one()) tc_commit(&bars.drained);
                __syncwarp();
                if (!mbar_wait(&bars.drained, 0)) atomicOr(&L.ctrl->error, SPEC_WS_ERR_WAIT);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax: a row a thread -------------------------------------------
        regs_up<kRegsSoftmax>();
        const int gr = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // this warp's 32 lanes, in bits 16..
        const uint32_t o_at = tmem + kO(gr) + lanes;
        const float cs = A.scale * kLog2e * 16.0f;
        uint32_t segs = 0, o_seen = 0, pv_seen = 0;
        uint32_t s_seen[2] = {0, 0};            // (both groups count both S)
        // Q's rows into shared memory: D/8 pieces of 8 a row, in the order of the
        // decoded keys (elements 0 4 1 5 2 6 3 7)
        auto load_q = [&](const Segment& g) {
            wait(&bars.q_empty, (segs & 1u) ^ 1u);
            ++segs;
            const int row = 128 * gr + r, rho = g.row0 + row;
            const bool on = row < g.live_rows;
            const int i = on ? static_cast<unsigned>(rho) / static_cast<unsigned>(A.G) : 0, gq = on ? rho - i * A.G : 0;
            const uint16_t* q = A.q + g.b * A.q_bs + i * A.q_rs + (static_cast<long long>(g.h) * A.G + gq) * A.q_hs;
            const uint32_t to = q_buf + gr * Cfg::kQBytes;
            if (on) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    uint4 x;
                    if (A.aligned) {
                        x = *reinterpret_cast<const uint4*>(q + 8 * j);
                    } else {
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = q[8 * j + 2 * e] | (static_cast<uint32_t>(q[8 * j + 2 * e + 1]) << 16);
                        x = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                    sts128(to + piece_at(r, j), __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                           __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_full);
        };
        Segment g = share.segment(share.lo());
        if (g.tiles > 0) load_q(g);
        for (;;) {
            const Req<kTok> rq = share.rq;
            const int row = 128 * gr + r, rho = g.row0 + row;
            const bool live = row < g.live_rows;
            const bool warp_live = (row & ~31) < g.live_rows, two = g.live_rows > 128;
            const int qi = static_cast<unsigned>(rho) / static_cast<unsigned>(A.G);     // the row's place among n
            float m = kNoMax;
            float2 l2 = make_float2(0.0f, 0.0f), lr2 = l2;      // two partial sums each
            const int mine = two || gr == 0 ? g.tiles : 0;      // this group's tiles
            // Whether pages are missing is asked for all of the unit's tiles at once; a
            // unit where some are looks them up again tile by tile.
            auto page_at = [&](int at) {
                if (!rq.needs(A, at, at + P)) return 0;
                return (at >> p_shift) < A.tab.width
                           ? static_cast<int>(ld_now_u32(A.tab.table + g.b * A.tab.stride + (at >> p_shift)))
                           : -1;
            };
            bool missing = false;
            {
                const int per = kTok >> p_shift, pages = mine << (7 - p_shift);
                for (int x0 = 0; x0 < pages; x0 += 128) {
                    int page[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int x = x0 + 32 * q + lane;
                        page[q] = x < pages ? page_at(rq.real(g.v0 + (x >> (7 - p_shift))) * kTok + ((x & (per - 1)) << p_shift)) : 0;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        missing |= static_cast<unsigned>(page[q]) >= static_cast<unsigned>(A.pool.num_pages);
                }
                missing = __any_sync(0xffffffffu, missing);
            }
            int plain0, plain1;
            rq.plain(A, plain0, plain1);
            plain0 -= g.v0;
            plain1 -= g.v0;
            for (int k = 0; k < mine; ++k) {
                const int sb = two ? gr : k & 1;
                const uint32_t s_at = tmem + kS(sb) + lanes;
                const bool lo = k < plain0 || k >= plain1;
                unsigned long long seen0 = ~0ull, seen1 = ~0ull;
                if (lo || missing) {
                    const int t0 = rq.real(g.v0 + k) * kTok;
                    if (live) {
                        seen0 = seen64(A, rq, g.b, qi, t0);
                        seen1 = seen64(A, rq, g.b, qi, t0 + 64);
                    }
                    if (missing) {
                        const int page = lane < kTok >> p_shift ? page_at(t0 + (lane << p_shift)) : 0;
#pragma unroll 1
                        for (uint32_t x = __ballot_sync(0xffffffffu, static_cast<unsigned>(page) >= static_cast<unsigned>(A.pool.num_pages));
                             x; x &= x - 1) {
                            const int a = (__ffs(x) - 1) << p_shift;
                            const unsigned long long off = range64(a & 63, (a & 63) + P, 0);
                            if (a < 64) seen0 &= ~off;
                            else seen1 &= ~off;
                        }
                    }
                }
                wait(&bars.s_full[sb], ((sb ? s_seen[1] : s_seen[0]) + (two ? k : k >> 1)) & 1u);
                tc_after();
                if (warp_live) {
                    auto tile = [&](auto is_masked) {
                        constexpr bool kMasked = decltype(is_masked)::value;
                        // 16 columns at a time, the next on their way
                        float x[16], y[16];
                        auto mask = [&](float (&z)[16], int c) {
                            if constexpr (kMasked) {
                                const uint32_t v = static_cast<uint32_t>((c >> 2 ? seen1 : seen0) >> (16 * (c & 3)));
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (!(v >> e & 1u)) z[e] = -CUDART_INF_F;
                            }
                        };
                        float top = -CUDART_INF_F;
                        auto look = [&](float (&z)[16], int c) {
                            mask(z, c);
#pragma unroll
                            for (int e = 0; e < 16; e += 2) top = fmaxf(top, fmaxf(z[e], z[e + 1]));
                        };
                        tc_ld16(x, s_at);
#pragma unroll 1
                        for (int c = 0; c < 8; c += 2) {
                            tc_wait_ld();
                            tc_ld16(y, s_at + 16 * (c + 1));
                            look(x, c);
                            tc_wait_ld();
                            tc_ld16(x, s_at + 16 * ((c + 2) & 7));      // (the last: the first again)
                            look(y, c + 1);
                        }
                        top *= cs;
                        // (rows that are not there multiply what lay in shared memory before:
                        // they have no say)
                        if (__any_sync(0xffffffffu, live && top > m + kSlack)) {
                            const float mn = fmaxf(m, top), f = exp2_fast(m - mn);
                            m = mn;
                            l2 = make_float2(l2.x * f, l2.y * f);
                            lr2 = make_float2(lr2.x * f, lr2.y * f);
                            if (k > 0) {
                                // the products so far must be done: with two groups S
                                // came after the group's last
                                if (!two) {
                                    wait(&bars.pv_done, (pv_seen + k - 1) & 1u);
                                    tc_after();
                                }
#pragma unroll 1
                                for (int c = 0; c < D / 16; ++c) {
                                    tc_ld16(y, o_at + 16 * c);
                                    tc_wait_ld();
                                    uint32_t u[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(y[e] * f);
                                    tc_st16(o_at + 16 * c, u);
                                }
                            }
                        }
                        // Weights, rounded to bf16 for the tensor core (2^-8 each at
                        // most); lse takes their sum before that, the output is
                        // divided by the sum of the rounded ones.  A tile where some
                        // row does not see all adds a second term with what rounding
                        // took from the first.
                        const float2 cs2 = make_float2(cs, cs), m2 = make_float2(-m, -m);
                        auto weigh = [&](float (&z)[16], int c) {
                            mask(z, c);
                            uint32_t hi[8], low[kMasked ? 8 : 1];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 a = fma2(make_float2(z[2 * e], z[2 * e + 1]), cs2, m2);
                                const float2 p = make_float2(exp2_fast(a.x), exp2_fast(a.y));
                                l2 = add2(l2, p);
                                hi[e] = pack_bf16(p.x, p.y);
                                const float2 h = make_float2(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xffff0000u));
                                if constexpr (kMasked) {
                                    low[e] = pack_bf16(p.x - h.x, p.y - h.y);
                                    lr2 = add2(lr2, lo ? p : h);
                                } else {
                                    lr2 = add2(lr2, h);
                                }
                            }
                            // P lies where its scores were: 8 columns of weights, 8 of
                            // second terms
                            tc_st8(s_at + 16 * c, hi);
                            if constexpr (kMasked) tc_st8(s_at + 16 * c + 8, low);
                        };
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            tc_wait_ld();
                            weigh(x, c);
                            tc_ld16(x, s_at + 16 * ((c + 1) & 7));
                        }
                        tc_wait_ld();
                        tc_wait_st();
                    };
                    if (lo || missing) tile(std::true_type{});
                    else tile(std::false_type{});
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[sb]);
            }
            if (two) {
                s_seen[0] += g.tiles;
                s_seen[1] += g.tiles;
            } else {
                s_seen[0] += (g.tiles + 1) >> 1;
                s_seen[1] += g.tiles >> 1;
                pv_seen += g.tiles;
            }
            const float l = l2.x + l2.y, lr = lr2.x + lr2.y;

            // ---- the next unit's Q, then this one's output ------------------------
            const Segment cur = g;
            const long long next = cur.u_from + cur.v1;
            const bool more = next < share.hi();
            if (more) {
                g = share.segment(next);
                if (g.tiles > 0) load_q(g);
            }
            if (mine > 0) {
                wait(&bars.o_done[gr], o_seen++ & 1u);
                tc_after();
            }
            const bool exists = rho < A.n * A.G;
            const long long at_row = (static_cast<long long>(cur.b) * A.n + qi) * A.hq +
                                     static_cast<long long>(cur.h) * A.G + (rho - qi * A.G);
            const bool whole = cur.whole();
            int c0 = blockIdx.x, parts = 1;
            if (!whole) share.sharers(cur, c0, parts);
            const int slot = 2 * static_cast<int>(blockIdx.x) + (c0 == static_cast<int>(blockIdx.x) ? 1 : 0);
            const long long part_row = static_cast<long long>(slot) * kRows + row;
            // 32 columns of O, in the order of the decoded values, into the output
            // or into the unit's parts
            auto emit = [&](int c, const float (&v)[32], bool on, float f) {
                uint4* to = reinterpret_cast<uint4*>(A.out + at_row * D + 32 * c);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float* y = v + 8 * w;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (on)
                        u = make_uint4(pack_bf16(y[0] * f, y[2] * f), pack_bf16(y[4] * f, y[6] * f),
                                       pack_bf16(y[1] * f, y[3] * f), pack_bf16(y[5] * f, y[7] * f));
                    to[w] = u;
                }
            };
            auto finish = [&](int c, const float (&v)[32]) {
                if (whole) {
                    const bool on = live && l != 0.0f;
                    if (exists) emit(c, v, on, on ? 16.0f / lr : 0.0f);
                } else if (live) {
                    float4* to = reinterpret_cast<float4*>(L.part + part_row * D + 32 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) __stcg(to + e, make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
                }
            };
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float v[32] = {};
                if (mine > 0 && warp_live) {
                    tc_ld32(v, o_at + 32 * c);
                    tc_wait_ld();
                }
                finish(c, v);
            }
            tc_before();
            __syncwarp();
            if (mine > 0 && lane == 0) mbar_arrive(&bars.o_free[gr]);
            {
                if (whole) {
                    if (exists && A.lse) A.lse[at_row] = live && l != 0.0f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
                } else {
                    if (live) __stcg(reinterpret_cast<float4*>(L.ml) + part_row, make_float4(m, l, lr, 0.0f));
                    __threadfence();
                    group_sync(gr);
                    if (r == 0) {
                        uint32_t* count = &L.ctrl->arrived[2 * c0 + gr];
                        const bool last = atomicAdd(count, 1u) == static_cast<uint32_t>(parts - 1);
                        if (last) *count = 0;
                        s_last[gr] = last;
                    }
                    group_sync(gr);
                    if (s_last[gr]) {
                        __threadfence();
                        auto place = [&](int c) { return (2ll * (c0 + c) + (c == 0 ? 1 : 0)) * kRows + row; };
                        float mm = kNoMax, sum = 0.0f, rsum = 0.0f;
                        if (live) {
#pragma unroll 4
                            for (int c = 0; c < parts; ++c) mm = fmaxf(mm, __ldcg(L.ml + place(c) * 4));
#pragma unroll 4
                            for (int c = 0; c < parts; ++c) {
                                const float4 ml = __ldcg(reinterpret_cast<const float4*>(L.ml) + place(c));
                                const float f = exp2_fast(ml.x - mm);
                                sum += f * ml.y;
                                rsum += f * ml.z;
                            }
                        }
                        const bool on = live && sum != 0.0f;
                        if (exists && A.lse) A.lse[at_row] = on ? (mm + log2f(sum)) * kLn2 : -CUDART_INF_F;
                        // The values, a row a warp, 16 rows in flight: a lane has D/32
                        // columns, 4 (2) of a group of 8 in the order 0 4 1 5 2 6 3 7.
                        const float scale = on ? 16.0f / rsum : 0.0f;
                        const unsigned there = __ballot_sync(0xffffffffu, exists);
                        constexpr int kRow = 16;
                        auto emit_row = [&](long long at, const float (&v)[D / 32], float f) {
                            uint16_t* to = A.out + at * D;
                            float y[D / 32];
#pragma unroll
                            for (int e = 0; e < D / 32; ++e) y[e] = f == 0.0f ? 0.0f : v[e] * f;
                            if constexpr (D == 128) {
                                to += 8 * (lane >> 1) + 2 * (lane & 1);
                                *reinterpret_cast<uint32_t*>(to) = pack_bf16(y[0], y[2]);
                                *reinterpret_cast<uint32_t*>(to + 4) = pack_bf16(y[1], y[3]);
                            } else {
                                to += 8 * (lane >> 2) + (lane & 3);
                                to[0] = __bfloat16_as_ushort(__float2bfloat16_rn(y[0]));
                                to[4] = __bfloat16_as_ushort(__float2bfloat16_rn(y[1]));
                            }
                        };
#pragma unroll 1
                        for (int q0 = 0; q0 < 32; q0 += kRow) {
                            if (!(there >> q0)) break;
                            float v[kRow][D / 32] = {};
                            for (int c = 0; c < parts; ++c) {
                                const float f_own = live ? exp2_fast(__ldcg(L.ml + place(c) * 4) - mm) : 0.0f;
                                const long long from = (2ll * (c0 + c) + (c == 0 ? 1 : 0)) * kRows + (row & ~31) + q0;
                                const float* x = L.part + from * D + lane * (D / 32);
                                // (rows that are not there: whatever lies in the parts, not used)
#pragma unroll
                                for (int q = 0; q < kRow; ++q) {
                                    const float f = __shfl_sync(0xffffffffu, f_own, q0 + q);
                                    if constexpr (D == 128) {
                                        const float4 y = __ldcg(reinterpret_cast<const float4*>(x + q * D));
                                        v[q][0] += f * y.x; v[q][1] += f * y.y; v[q][2] += f * y.z; v[q][3] += f * y.w;
                                    } else {
                                        const float2 y = __ldcg(reinterpret_cast<const float2*>(x + q * D));
                                        v[q][0] += f * y.x; v[q][1] += f * y.y;
                                    }
                                }
                            }
#pragma unroll
                            for (int q = 0; q < kRow; ++q) {
                                const float f = __shfl_sync(0xffffffffu, scale, q0 + q);
                                const long long at = __shfl_sync(0xffffffffu, at_row, q0 + q);
                                if (there >> (q0 + q) & 1u) emit_row(at, v[q], f);
                            }
                        }
                    }
                }
            }
            if (!more) break;
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, 512);
}

template <int D>
cudaError_t attend_tc(const CacheAttendArgs& A, cudaStream_t st) {
    using Cfg = TcCfg<D>;
    const int grid = min(attend_sms(), kMaxGrid / 2);
    const AttendLayout y(2 * grid, kRows, D);
    AttendPlan L;
    L.one2 = 0x3F803F80u;
    L.row_tiles = (A.n * A.G + kRows - 1) / kRows;
    L.min_tiles = 2;
    unsigned char* ws = static_cast<unsigned char*>(A.ws);
    L.ctrl = reinterpret_cast<AttendCtrl*>(ws);
    L.ml = reinterpret_cast<float*>(ws + y.ml);
    L.part = reinterpret_cast<float*>(ws + y.part);
    static std::atomic<unsigned long long> ready{0};
    const int dev = attend_device();
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(cache_attend_tc_kernel<D>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_early(cache_attend_tc_kernel<D>, grid, kThreads, Cfg::kSmem, st, A, L);
}

}  // namespace

#ifdef SPEC_TEST_HOOKS
extern "C" int spec_test_drop_commit(int on) { return static_cast<int>(cudaMemcpyToSymbol(g_test_drop, &on, sizeof(int))); }
#endif

size_t attend_tc_ws(int D) { return AttendLayout(2 * min(attend_sms(), kMaxGrid / 2), kRows, D).bytes; }

long long attend_tc_tiles(int R, int hkv, long long positions) {
    return (positions / kTok + 2) * hkv * ((R + kRows - 1) / kRows);
}

cudaError_t attend_tc_run(const CacheAttendArgs& A, cudaStream_t st) {
    return A.pool.D == 128 ? attend_tc<128>(A, st) : attend_tc<64>(A, st);
}

}  // namespace spec
