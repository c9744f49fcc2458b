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
// A tile.  Bulk copies (TMA), one per page block, bring a tile into a ring in
// shared memory.  Codes go from there straight into the registers of the tensor
// instruction (mma m16n8k16): scores are computed transposed, S^T = K Q^T and
// O^T = V^T P^T, so that the cache's side is the 16-row operand and the few
// rows of a request fill 8-column blocks instead of padding a 16-row tile.
// Four warps share a tile: each takes 16 tokens of S^T and then, P^T having
// gone through shared memory, a quarter of the D rows of O^T over all 64
// tokens.  No code is decoded twice, a warp's share of O^T is small enough for
// many CTAs an SM, and one barrier a tile is all they wait for each other.  (Tiles of
// 128 tokens halve the barriers, but their registers cost a CTA an SM: slower.)
//
// What bounds it.  No unit is at its limit: a tile is a chain (codes, S^T, exponentials,
// a barrier, O^T), and the three to six CTAs that an SM has registers for overlap
// theirs.  All with 8 heads of 128 and lengths evenly from the first down to the second:
//   4 rows a head, 4 requests of 131072 to 57344 tokens: 124 us, 434 MB, 3.5 TB/s.  68 %
//       of the issue slots; 480 instructions a tile and warp, 192 turn codes into bf16.
//   16 rows, 64 requests of 2048 to 536: 50 us.  54 % of the slots, 680 instructions a
//       tile and warp; the tensor instruction (one in 8 cycles a scheduler, 16 for every 8
//       rows of a tile and warp) 21 % of the time.  A CTA has only 14 tiles.
//   36 rows, 256 requests of 4096 to 1036: 448 us, 217 TFLOP/s.  52 % of the slots, the
//       tensor instruction 43 %; three CTAs an SM.
// One request of a few hundred tokens takes 10 us: launch, the deal of the work, one
// tile, the join.
#include <atomic>
#include <type_traits>

#include "spec_cache_attend.cuh"

namespace spec {

namespace {

constexpr int kAtWarps = 4;
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kTile = 64;                       // tokens a tile
// Rows a kv head that this kernel takes.  Its time grows with every 8 rows (past 48 it
// would need two blocks of them), the tcgen05 kernel's hardly up to 128: 64 requests of
// 2048 to 536 tokens 70 / 96 / 162 / 171 us at 32 / 48 / 64 / 96 rows against 110 / 111 /
// 112 / 116; 32 of 8192 to 2240 246 against 145 us at 64.
constexpr int kFewRows = 48;

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
// a lane's codes of a value row: D/32 of them
template <int D>
__device__ __forceinline__ uint32_t ldsv(uint32_t a) {
    if constexpr (D == 128) {
        return lds16(a);
    } else {
        uint32_t v;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
        return v;
    }
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" :: "r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t v;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(v) : "r"(x));
    return v;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
constexpr int ctas_of(int NT) { return NT == 1 ? 6 : NT <= 3 ? 5 : NT == 4 ? 4 : 3; }

template <int D, int NT>
struct AttendCfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kStageBytes = kTile * CacheBlock<D>::kTok;
    static constexpr int kP = 4 * NT * 256;                 // P^T of a tile: [16 tokens][NT][lane] of 8 bytes
    static constexpr int kQ = (D / 16) * NT * 256;          // Q: [k step][NT][lane] of 8 bytes
    static constexpr int kSmem = kStages * kStageBytes + kQ + 3 * kP;
    // resident CTAs an SM: what registers (O^T, S^T) and shared memory allow
    static constexpr int kCtas = ctas_of(NT);
    static constexpr bool kQInRegs = NT == 1;
};

template <int D, int NT>
__global__ void __launch_bounds__(kAtThreads, AttendCfg<D, NT>::kCtas)
cache_attend_kernel(const __grid_constant__ CacheAttendArgs A, const __grid_constant__ AttendPlan L) {
    using Cfg = AttendCfg<D, NT>;
    using Blk = CacheBlock<D>;
    constexpr int kS = Cfg::kStages, kRows = Cfg::kRows;
    constexpr int kKW = D / 32;                 // words of a key that a lane holds
    constexpr int kMT = D / 64;                 // 16-row blocks of O^T that a warp holds
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kS];
    __shared__ ShareScratch<kAtWarps> s_share;
    __shared__ long long s_out[kRows];          // a row's place in out and lse (-1: none)
    // which page blocks of a stage's tile are there; above them, once copies into the
    // stage were given out, kGiven and the parity that their barrier's wait takes
    constexpr uint32_t kThere = 0xfu, kGiven = 0x10u, kParity = 5;
    __shared__ uint32_t s_there[kS];
    __shared__ unsigned long long s_seen[kRows];
    __shared__ float s_max[kAtWarps][kRows];
    __shared__ float s_l[kAtWarps][kRows], s_lr[kAtWarps][kRows];
    __shared__ int s_last, s_dead;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);    // uniform to the compiler too
    const int r8 = lane >> 2, c4 = lane & 3;
    const int P = A.pool.P, p_shift = A.pool.p_shift;
    const int ppt_shift = 6 - p_shift, ppt = 1 << ppt_shift;    // page blocks a tile
    // A tile in shared memory is laid out like one block of 64 tokens, whatever
    // the pages' size.
    constexpr int kKs = kTile * Blk::kRow, kV = Blk::v_codes(kTile), kVs = kV + kTile * Blk::kRow;
    const uint32_t ring = smem_u32(smem);
    const uint32_t q_base = ring + kS * Cfg::kStageBytes, p_base = q_base + Cfg::kQ, lo_base = p_base + 2 * Cfg::kP;

    if (tid == 0) {
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            mbar_init(&full[s], 1);
            s_there[s] = 0;
        }
        fence_mbar_init();
        s_dead = 0;
    }

    after_earlier();
    Share<kTile, kAtWarps> share(A, L, s_share, kRows);
    if (share.lo() == share.hi()) return;
    const int cta = blockIdx.x;

    uint32_t phases = 0;                        // one bit a stage
    const int tok = r8 ^ ((r8 >> 1) & 1);       // the token (of 8) that is row r8 of S^T
    const int tv0 = (2 * c4) ^ (c4 & 1);        // tokens 2c and 2c+1 of P^T's rows
    const int tv1 = (2 * c4 + 1) ^ (c4 & 1);
    // where a lane's words and scales lie in a tile: its key (this warp's 16
    // tokens), and its part of the values of the first 16
    const uint32_t k_at = (warp * 16 + tok) * Blk::kRow + c4 * (D / 8);
    const uint32_t ks_at = kKs + (warp * 16 + tok) * Blk::kScl + (D == 128 ? c4 : c4 >> 1) * 2;
    const uint32_t v_at = kV + warp * (D / 8) + r8 * (D / 64);
    const uint32_t v0_at = v_at + tv0 * Blk::kRow, v1_at = v_at + tv1 * Blk::kRow;
    // A lane fetches the scale pair of tokens (2c, 2c+1) of the lane >> 2 -th 8
    // tokens for the lanes of column c.
    const uint32_t vs_at = kVs + (lane >> 2) * 8 * Blk::kScl + (D == 128 ? warp : warp >> 1) * 2;
    const uint32_t vs0_at = vs_at + tv0 * Blk::kScl, vs1_at = vs_at + tv1 * Blk::kScl;
    const float cs = A.scale * kLog2e * 16.0f;
    const uint32_t one2 = L.one2;

    // Copies: the warps take the tiles in turn, a lane per page block of the tiles that
    // a warp will copy.
    int entry = -2;
    auto issue = [&](const Segment& g, int k, int s) {
        const int in = (k >> 2) & ((32 >> ppt_shift) - 1);  // of the tiles whose page ids the lanes hold
        if (in == 0) {
            const int v = g.v0 + k + kAtWarps * (lane >> ppt_shift);
            entry = -2;
            if (v < g.v1) {
                const int t = share.rq.real(v) * kTile + ((lane & (ppt - 1)) << p_shift);
                if (share.rq.needs(A, t, t + P)) {
                    entry = cache_page(A.tab, A.pool.num_pages, p_shift, g.b, t);
                    if (entry < 0 && A.status) atomicOr(A.status + g.b, SPEC_ST_BAD_PAGE);
                }
            }
        }
        const int l0 = in << ppt_shift;
        const uint32_t there = (__ballot_sync(0xffffffffu, entry >= 0) >> l0) & ((1u << ppt) - 1u);
#ifdef SPEC_TEST_HOOKS
        if (g_test_drop && cta == 0 && k == 0) return;
#endif
        if (lane == 0) {
            s_there[s] = there | kGiven | (phases >> s & 1u) << kParity;
            mbar_expect_tx(&full[s], __popc(there) * Blk::bytes(P));
        }
        __syncwarp();
        if (lane >= l0 && lane < l0 + ppt && entry >= 0) {
            const unsigned char* from = A.pool.base + entry * A.pool.page_stride + g.h * A.pool.head_stride;
            unsigned char* to = smem + s * Cfg::kStageBytes;
            const int at = (lane - l0) << p_shift;
            if (P == kTile) {
                tma_load_1d(to, from, Blk::bytes(kTile), &full[s]);
            } else {
                tma_load_1d(to + at * Blk::kRow, from, P * Blk::kRow, &full[s]);
                tma_load_1d(to + kKs + at * Blk::kScl, from + P * Blk::kRow, P * Blk::kScl, &full[s]);
                tma_load_1d(to + kV + at * Blk::kRow, from + Blk::v_codes(P), P * Blk::kRow, &full[s]);
                tma_load_1d(to + kVs + at * Blk::kScl, from + Blk::v_codes(P) + P * Blk::kRow, P * Blk::kScl, &full[s]);
            }
        }
    };
    // The start of a segment, as far as it can run beside the end of the one
    // before it: first copies, and Q's rows into the buffer of P^T.
    auto begin = [&](const Segment& g) {
        if (!s_dead)
#pragma unroll
            for (int s = 0; s < kS; ++s)
                if (s < g.tiles && warp == (s & 3)) issue(g, s, s);
        if (A.aligned && g.tiles > 0) {
            for (int x = tid; x < kRows * (D / 8); x += kAtThreads) {
                const int row = x / (D / 8), c = x % (D / 8), rho = g.row0 + row;
                if (row < g.live_rows) {
                    const int i = static_cast<unsigned>(rho) / static_cast<unsigned>(A.G), gq = rho - i * A.G;
                    const uint16_t* q = A.q + g.b * A.q_bs + i * A.q_rs + (static_cast<long long>(g.h) * A.G + gq) * A.q_hs + c * 8;
                    cp_async16(p_base + (row * (D / 8) + (c ^ (row & 7))) * 16, q);
                }
            }
            cp_async_commit();
        }
    };

    Segment g = share.segment(share.lo());
    begin(g);
    for (;;) {
        // ---- Q, laid out like the keys' words -------------------------------
        const int row0 = g.row0, live_rows = g.live_rows, tiles = g.tiles, v0 = g.v0;
        const Req<kTile> rc = share.rq;         // the request (the cursor moves on before the segment's end)
        if (tid < kRows) {
            const int rho = row0 + tid, i = static_cast<unsigned>(rho) / static_cast<unsigned>(A.G);
            s_out[tid] = rho < A.n * A.G ? (static_cast<long long>(g.b) * A.n + i) * A.hq + static_cast<long long>(g.h) * A.G + rho - i * A.G : -1;
        }
        cp_async_wait();
        __syncthreads();
        if (tiles > 0)
            for (int x = tid; x < NT * kKW * 32; x += kAtThreads) {
                const int l = x & 31, nt = (x >> 5) % NT, w = (x >> 5) / NT;
                const int row = nt * 8 + (l >> 2), c = (l & 3) * kKW + w;
                uint32_t y[4] = {0, 0, 0, 0};
                if (row < live_rows) {
                    if (A.aligned) {
                        lds(y, p_base + (row * (D / 8) + (c ^ (row & 7))) * 16);
                    } else {
                        const int rho = row0 + row, i = static_cast<unsigned>(rho) / static_cast<unsigned>(A.G), gq = rho - i * A.G;
                        const uint16_t* q = A.q + g.b * A.q_bs + i * A.q_rs + (static_cast<long long>(g.h) * A.G + gq) * A.q_hs + c * 8;
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = q[2 * e] | (static_cast<uint32_t>(q[2 * e + 1]) << 16);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    sts64(q_base + (((2 * w + u) * NT + nt) * 32 + l) * 8, __byte_perm(y[u], y[u + 2], 0x5410),
                          __byte_perm(y[u], y[u + 2], 0x7632));
            }
        __syncthreads();
        uint32_t qf[Cfg::kQInRegs ? D / 16 : 1][NT][2];
        if constexpr (Cfg::kQInRegs) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) lds(qf[ks][nt], q_base + ((ks * NT + nt) * 32 + lane) * 8);
        }

        float o[kMT][NT][4], m[NT][2], l[NT][2], lr[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kNoMax;
            l[nt][0] = l[nt][1] = lr[nt][0] = lr[nt][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < kMT; ++j) o[j][nt][0] = o[j][nt][1] = o[j][nt][2] = o[j][nt][3] = 0.0f;
        }

        // ---- the tiles -------------------------------------------------------
        int s = 0, refill = kS - 1;             // this tile's stage, the one before it
        for (int k = 0; k < tiles; ++k) {
            const int t0 = rc.real(v0 + k) * kTile;
            if (!s_dead && !mbar_wait(&full[s], (phases >> s) & 1u)) {
                s_dead = 1;
                atomicOr(&L.ctrl->error, SPEC_WS_ERR_WAIT);
            }
            const uint32_t there = s_there[s] & kThere;
            phases ^= 1u << s;
            const uint32_t stage = ring + s * Cfg::kStageBytes;
            const uint32_t pbuf = p_base + (k & 1) * Cfg::kP;
            // every row sees every key of most tiles
            const bool masked = rc.partial(A, t0) || there != (1u << ppt) - 1u;
            auto tile = [&](auto is_masked) {
                constexpr bool kMasked = decltype(is_masked)::value;
                unsigned long long any = ~0ull;
                if constexpr (kMasked) {
                    if (tid < kRows) {
                        unsigned long long v = 0;
                        if (tid < live_rows) v = seen64(A, rc, g.b, static_cast<unsigned>(row0 + tid) / static_cast<unsigned>(A.G), t0);
#pragma unroll 1
                        for (int q = 0; q < ppt; ++q)
                            if (!(there >> q & 1u)) v &= ~range64(q << p_shift, (q + 1) << p_shift, 0);
                        s_seen[tid] = v;
                    }
                    __syncthreads();
                    any = 0;
                    for (int q = lane; q < kRows; q += 32) any |= s_seen[q];
                    any = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any)) |
                          static_cast<unsigned long long>(
                              __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32))) << 32;
                }
                // S^T = K Q^T: this warp's 16 tokens
                float x[NT][4];
                [[maybe_unused]] float y[NT][4];            // one block of rows: two chains of sums, for latency
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.0f;
                if constexpr (NT == 1) y[0][0] = y[0][1] = y[0][2] = y[0][3] = 0.0f;
                {
                    uint32_t wa[kKW], wb[kKW];
                    lds(wa, stage + k_at);
                    lds(wb, stage + k_at + 8 * Blk::kRow);
                    const uint32_t sa = lds16(stage + ks_at) * 0x10001u, sb = lds16(stage + ks_at + 8 * Blk::kScl) * 0x10001u;
                    const uint32_t ca = minus1_5(sa), cb = minus1_5(sb);
                    auto step = [&](int ks, const uint32_t (&a)[4]) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (Cfg::kQInRegs) {
                                mma(ks & 1 ? y[nt] : x[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
                            } else {
                                uint32_t q2[2];
                                lds(q2, q_base + ((ks * NT + nt) * 32 + lane) * 8);
                                mma(x[nt], a, q2[0], q2[1]);
                            }
                        }
                    };
#pragma unroll
                    for (int w = 0; w < kKW; ++w) {
                        const uint32_t a0[4] = {codes2<0>(wa[w], sa, ca, one2), codes2<0>(wb[w], sb, cb, one2),
                                                codes2<1>(wa[w], sa, ca, one2), codes2<1>(wb[w], sb, cb, one2)};
                        step(2 * w, a0);
                        const uint32_t a1[4] = {codes2<2>(wa[w], sa, ca, one2), codes2<2>(wb[w], sb, cb, one2),
                                                codes2<3>(wa[w], sa, ca, one2), codes2<3>(wb[w], sb, cb, one2)};
                        step(2 * w + 1, a1);
                    }
                    if constexpr (NT == 1) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[0][e] += y[0][e];
                    }
                }
                if constexpr (kMasked) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t v = static_cast<uint32_t>(s_seen[nt * 8 + 2 * c4 + e] >> (warp * 16 + tok));
                            if (!(v & 1u)) x[nt][e] = -CUDART_INF_F;
                            if (!(v >> 8 & 1u)) x[nt][2 + e] = -CUDART_INF_F;
                        }
                }
                // Weights under the maximum so far, as the 16 x 8 operand P^T.
                // They are rounded to bf16 for the tensor cores (2^-8 each at
                // most, as the output's own rounding); lse takes their sum
                // before that (l), the output is divided by the sum of the rounded
                // ones (lr), so that what rounding they have in common cancels
                // (one dominant key: all of it).  lr from a row of ones as another
                // row of V^T cost up to 6 % more.  A tile with masked keys, where a
                // row may see only a few, adds a second term with what rounding
                // took from the first.
                float ls[NT][2], lrs[NT][2];
                auto weights = [&]() {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = exp2_fast(fmaf(x[nt][e], cs, -m[nt][e & 1]));
                        ls[nt][0] = p[0] + p[2];
                        ls[nt][1] = p[1] + p[3];
                        const uint32_t ab = pack_bf16(p[0], p[1]), cd = pack_bf16(p[2], p[3]);
                        sts64(pbuf + ((warp * NT + nt) * 32 + lane) * 8, transpose8x8(ab), transpose8x8(cd));
                        lrs[nt][0] = __uint_as_float(ab << 16) + __uint_as_float(cd << 16);
                        lrs[nt][1] = __uint_as_float(ab & 0xffff0000u) + __uint_as_float(cd & 0xffff0000u);
                        if constexpr (kMasked) {
                            const uint32_t rab = pack_bf16(p[0] - __uint_as_float(ab << 16),
                                                           p[1] - __uint_as_float(ab & 0xffff0000u));
                            const uint32_t rcd = pack_bf16(p[2] - __uint_as_float(cd << 16),
                                                           p[3] - __uint_as_float(cd & 0xffff0000u));
                            lrs[nt][0] += __uint_as_float(rab << 16) + __uint_as_float(rcd << 16);
                            lrs[nt][1] += __uint_as_float(rab & 0xffff0000u) + __uint_as_float(rcd & 0xffff0000u);
                            sts64(lo_base + ((warp * NT + nt) * 32 + lane) * 8, transpose8x8(rab), transpose8x8(rcd));
                        }
                    }
                };
                bool move = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        move |= fmaxf(x[nt][e], x[nt][2 + e]) * cs > m[nt][e] + kSlack;
                weights();
                if (__syncthreads_or(move)) {
                    // the maximum moves: all warps agree on it, rescale, and weigh again
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = fmaxf(x[nt][e], x[nt][2 + e]) * cs;
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                            if (r8 == 0) s_max[warp][nt * 8 + 2 * c4 + e] = t;
                        }
                    __syncthreads();
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mn = m[nt][e];
#pragma unroll
                            for (int w = 0; w < kAtWarps; ++w) mn = fmaxf(mn, s_max[w][nt * 8 + 2 * c4 + e]);
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
                    weights();
                    __syncthreads();
                }
                // every warp is past the tile before this one: its stage is free
                if (warp == ((k - 1 + kS) & 3) && k > 0 && k - 1 + kS < tiles && !s_dead) issue(g, k - 1 + kS, refill);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt][0] += ls[nt][0];
                    l[nt][1] += ls[nt][1];
                    lr[nt][0] += lrs[nt][0];
                    lr[nt][1] += lrs[nt][1];
                }
                // O^T += V^T P^T: this warp's rows, all tokens
                uint32_t vscale;
                {
                    uint32_t s0 = lds16(stage + vs0_at), s1 = lds16(stage + vs1_at);
                    if constexpr (kMasked) {    // what no row sees may be anything, NaN among it
                        const uint32_t a = static_cast<uint32_t>(any >> ((lane >> 2) * 8));
                        s0 = a >> tv0 & 1 ? s0 : 0;
                        s1 = a >> tv1 & 1 ? s1 : 0;
                    }
                    vscale = s0 | s1 << 16;
                }
#pragma unroll
                for (int mb = 0; mb < 4; ++mb) {
                    const uint32_t vr = stage + mb * 16 * Blk::kRow;
                    // token pairs side by side: four (two) codes each
                    const uint32_t ab = __byte_perm(ldsv<D>(vr + v0_at), ldsv<D>(vr + v1_at), 0x5410);
                    const uint32_t cd = __byte_perm(ldsv<D>(vr + v0_at + 8 * Blk::kRow), ldsv<D>(vr + v1_at + 8 * Blk::kRow), 0x5410);
                    const uint32_t sa = __shfl_sync(0xffffffffu, vscale, mb * 8 + c4);
                    const uint32_t sb = __shfl_sync(0xffffffffu, vscale, mb * 8 + 4 + c4);
                    const uint32_t ca = minus1_5(sa), cb = minus1_5(sb);
                    uint32_t a[kMT][4];
                    a[0][0] = codes2<0>(ab, sa, ca, one2);
                    a[0][1] = codes2<1>(ab, sa, ca, one2);
                    a[0][2] = codes2<0>(cd, sb, cb, one2);
                    a[0][3] = codes2<1>(cd, sb, cb, one2);
                    if constexpr (kMT == 2) {
                        a[1][0] = codes2<2>(ab, sa, ca, one2);
                        a[1][1] = codes2<3>(ab, sa, ca, one2);
                        a[1][2] = codes2<2>(cd, sb, cb, one2);
                        a[1][3] = codes2<3>(cd, sb, cb, one2);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint32_t p2[2];
                        lds(p2, pbuf + ((mb * NT + nt) * 32 + lane) * 8);
#pragma unroll
                        for (int j = 0; j < kMT; ++j) mma(o[j][nt], a[j], p2[0], p2[1]);
                        if constexpr (kMasked) {
                            lds(p2, lo_base + ((mb * NT + nt) * 32 + lane) * 8);
#pragma unroll
                            for (int j = 0; j < kMT; ++j) mma(o[j][nt], a[j], p2[0], p2[1]);
                        }
                    }
                }
                if constexpr (kMasked) __syncthreads();     // the second terms' buffer is written again
            };
            if (masked) tile(std::true_type{});
            else tile(std::false_type{});
            refill = s;
            s = s + 1 == kS ? 0 : s + 1;
        }

        // ---- the rows' sums, and out -------------------------------------------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = l[nt][e];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                if (r8 == 0) s_l[warp][nt * 8 + 2 * c4 + e] = t;
                t = lr[nt][e];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                if (r8 == 0) s_lr[warp][nt * 8 + 2 * c4 + e] = t;
            }
        __syncthreads();
        // every warp is past its last tile: the next segment may begin
        const Segment cur = g;
        const bool more = cur.u_from + cur.v1 < share.hi();
        if (more) {
            g = share.segment(cur.u_from + cur.v1);
            begin(g);
        }
        const bool whole = cur.whole();
        // the CTA that holds the unit's first tile, and how many share it
        int c0 = cta, parts = 1;
        if (!whole) share.sharers(cur, c0, parts);
        const int slot = 2 * cta + (c0 == cta ? 1 : 0);
        const int d0 = warp * (D / 4) + r8 * (D / 32);          // this lane's D/32 values of a row
        // D/32 values from d on of a row, times f, into the output
        auto emit = [&](long long at, int d, const float (&v)[2 * kMT], float f) {
            uint16_t* to = A.out + at * D + d;
            if constexpr (kMT == 2)
                *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f));
            else
                *reinterpret_cast<uint32_t*>(to) = pack_bf16(v[0] * f, v[1] * f);
        };
        auto emit_lse = [&](long long at, bool on, float mm, float sum) {
            if (A.lse) A.lse[at] = on ? (mm + log2f(sum)) * kLn2 : -CUDART_INF_F;
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * c4 + e;
                float sum = 0.0f, v[2 * kMT];
                float rsum = 0.0f;
#pragma unroll
                for (int w = 0; w < kAtWarps; ++w) rsum += s_lr[w][row];
#pragma unroll
                for (int w = 0; w < kAtWarps; ++w) sum += s_l[w][row];
#pragma unroll
                for (int j = 0; j < kMT; ++j) {
                    v[2 * j] = o[j][nt][e];
                    v[2 * j + 1] = o[j][nt][2 + e];
                }
                if (whole) {
                    const long long at = s_out[row];
                    const bool on = row < live_rows && sum != 0.0f;
                    if (at >= 0) {
                        if (!on) {              // nothing seen: whatever O^T holds there
#pragma unroll
                            for (int j = 0; j < 2 * kMT; ++j) v[j] = 0.0f;
                        }
                        emit(at, d0, v, on ? 16.0f / rsum : 0.0f);
                        if (warp == 0 && r8 == 0) emit_lse(at, on, m[nt][e], sum);
                    }
                } else {
                    const long long at = static_cast<long long>(slot) * kRows + row;
                    if constexpr (kMT == 2)
                        __stcg(reinterpret_cast<float4*>(L.part + at * D + d0), make_float4(v[0], v[1], v[2], v[3]));
                    else
                        __stcg(reinterpret_cast<float2*>(L.part + at * D + d0), make_float2(v[0], v[1]));
                    if (warp == 0 && r8 == 0)
                        __stcg(reinterpret_cast<float4*>(L.ml) + at, make_float4(m[nt][e], sum, rsum, 0.0f));
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
                auto place = [&](int c, int row) { return (2ll * (c0 + c) + (c == 0 ? 1 : 0)) * kRows + row; };
                // first each row's maximum and sums, then the values, D/32 a thread
                if (tid < kRows) {
                    float mm = kNoMax, sum = 0.0f, rsum = 0.0f;
#pragma unroll 4
                    for (int c = 0; c < parts; ++c) mm = fmaxf(mm, __ldcg(L.ml + place(c, tid) * 4));
#pragma unroll 4
                    for (int c = 0; c < parts; ++c) {
                        const float4 ml = __ldcg(reinterpret_cast<const float4*>(L.ml) + place(c, tid));
                        const float f = exp2_fast(ml.x - mm);
                        sum += f * ml.y;
                        rsum += f * ml.z;
                    }
                    const bool on = tid < live_rows && sum != 0.0f;
                    s_max[0][tid] = mm;
                    s_max[1][tid] = on ? 16.0f / rsum : 0.0f;
                    s_max[2][tid] = on ? 1.0f : 0.0f;
                    if (s_out[tid] >= 0) emit_lse(s_out[tid], on, mm, sum);
                }
                __syncthreads();
                for (int x = tid; x < kRows * 32; x += kAtThreads) {
                    const int row = x >> 5, d = (x & 31) * (D / 32);
                    const long long at = s_out[row];
                    if (at < 0) continue;
                    const float mm = s_max[0][row];
                    float v[2 * kMT] = {};
#pragma unroll 4
                    for (int c = 0; c < parts; ++c) {
                        const long long from = place(c, row);
                        const float f = exp2_fast(__ldcg(L.ml + from * 4) - mm);
                        if constexpr (kMT == 2) {
                            const float4 z = __ldcg(reinterpret_cast<const float4*>(L.part + from * D + d));
                            v[0] += f * z.x; v[1] += f * z.y; v[2] += f * z.z; v[3] += f * z.w;
                        } else {
                            const float2 z = __ldcg(reinterpret_cast<const float2*>(L.part + from * D + d));
                            v[0] += f * z.x; v[1] += f * z.y;
                        }
                    }
                    if (s_max[2][row] == 0.0f) {
#pragma unroll
                        for (int j = 0; j < 2 * kMT; ++j) v[j] = 0.0f;
                    }
                    emit(at, d, v, s_max[1][row]);
                }
            }
        }
        if (!more) break;
        __syncthreads();                        // shared memory is written again
    }
    // After a wait that gave up: copies on their way land before the CTA ends.
    if (s_dead && tid < kS && (s_there[tid] & kGiven)) mbar_wait(&full[tid], s_there[tid] >> kParity & 1u);
}

}  // namespace

int attend_device() {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) {
        cudaGetLastError();
        return 64;                              // no device: sizes are asked for on a GB300's behalf
    }
    return d;
}

int attend_sms() {
    static std::atomic<int> known[64];
    const int d = attend_device();
    if (d >= 64) return 152;
    int v = known[d].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
            cudaGetLastError();
            return 152;
        }
        known[d].store(v, std::memory_order_relaxed);
    }
    return v;
}

namespace {

// Blocks of 8 rows that a CTA holds: all of a request's, so that a tile's codes are
// decoded once.
int row_blocks(int R) {
    static constexpr int kSizes[] = {1, 2, 3, 4, 5, 6};
    for (const int s : kSizes)
        if (8 * s >= R) return s;
    return 6;
}

template <int D, int NT>
cudaError_t attend(const CacheAttendArgs& A, cudaStream_t st) {
    using Cfg = AttendCfg<D, NT>;
    const int grid = min(attend_sms() * Cfg::kCtas, kMaxGrid);
    const AttendLayout y(2 * grid, Cfg::kRows, D);
    AttendPlan L;
    L.one2 = 0x3F803F80u;
    L.row_tiles = (A.n * A.G + Cfg::kRows - 1) / Cfg::kRows;
    L.min_tiles = 1;
    unsigned char* ws = static_cast<unsigned char*>(A.ws);
    L.ctrl = reinterpret_cast<AttendCtrl*>(ws);
    L.ml = reinterpret_cast<float*>(ws + y.ml);
    L.part = reinterpret_cast<float*>(ws + y.part);
    // the kernel's shared memory is set once a device
    static std::atomic<unsigned long long> ready{0};
    const int dev = attend_device();
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(cache_attend_kernel<D, NT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_early(cache_attend_kernel<D, NT>, grid, kAtThreads, Cfg::kSmem, st, A, L);
}

template <int D>
cudaError_t attend_rows(const CacheAttendArgs& A, cudaStream_t st) {
    switch (row_blocks(A.n * A.G)) {
        case 1: return attend<D, 1>(A, st);
        case 2: return attend<D, 2>(A, st);
        case 3: return attend<D, 3>(A, st);
        case 4: return attend<D, 4>(A, st);
        case 5: return attend<D, 5>(A, st);
        default: return attend<D, 6>(A, st);
    }
}

}  // namespace

#ifdef SPEC_TEST_HOOKS
extern "C" int spec_test_drop_copy(int on) { return static_cast<int>(cudaMemcpyToSymbol(g_test_drop, &on, sizeof(int))); }
#endif

size_t cache_attend_ws(int B, int n, int hq, int hkv, int D) {
    (void)B;
    const int R = n * (hq / hkv);
    if (R > kFewRows) return attend_tc_ws(D);
    const int NT = row_blocks(R);
    return AttendLayout(2 * min(attend_sms() * ctas_of(NT), kMaxGrid), 8 * NT, D).bytes;
}

long long cache_attend_tiles(int n, int hq, int hkv, long long positions) {
    const int R = n * (hq / hkv);
    if (R > kFewRows) return attend_tc_tiles(R, hkv, positions + n);
    const int rows = 8 * row_blocks(R);
    return ((positions + n) / kTile + 2) * hkv * ((R + rows - 1) / rows);
}

cudaError_t cache_attend_run(const CacheAttendArgs& A, cudaStream_t st) {
    if (A.n * A.G > kFewRows) return attend_tc_run(A, st);
    return A.pool.D == 128 ? attend_rows<128>(A, st) : attend_rows<64>(A, st);
}

}  // namespace spec
