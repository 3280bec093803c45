// window.cu -- paged absorbed-MLA attention over a sliding window and the first tokens, for sm_103a.
//
// Math: a token row with a context of n tokens (itself the last one) sees the tokens
//     t < min(n_sink, n)   and   max(0, n - window) <= t < n,
// and over those, with cache rows r_t (a -1 block table entry is an all-zero row),
//     s_t   = scale * (q_abs[h] . r_t)        (dot over 576)
//     p     = softmax(s),  o_lat = sum_t p_t r_t[0:512],  out = W_UV[h] o_lat.
// Decode: one token row per slot.  Chunk: several consecutive new token rows per slot.
//
// Numerics.  Scores, maxima, sums and o_lat are f32.  Three roundings go below that: the p of the second
// contraction to bf16 (the tensor core's operand type; both operands have one type and the cache is bf16),
// o_lat to a pair of bf16 (hi + lo, 2^-17: a single bf16 here would add as much error again as the output's
// own rounding does), and the output to bf16.
//
// Structure.  A unit of work is 96 heads of one slot and one split of what it sees (decode), or 32 heads of
// up to four consecutive token rows (chunk): a row in each of the 128 (96) TMEM lanes.  Clusters of two
// CTAs walk the units, cluster c taking units c, c + clusters, ...; the score CTA (rank 0) and the PV CTA
// (rank 1) of decode_core.cuh each have their roles in warps of their own, and every role runs on into the
// next unit by itself: ring slots, S buffers, P buffers and barrier phases go by running counts, never
// reset.  So the ramp of a unit (its Q, its first pages) overlaps the softmax, the second contraction and
// the write-out of the one before, which matters because a window is short: 1,024 tokens are 17 pages of
// some 0.7 us, and a unit that starts and ends alone adds about 8 us.
//   * A unit's pages are the logical pages that hold a seen token, in ascending order: those of the sinks,
//     then those of the window.  Pages in between are neither read nor looked up, so they may have been
//     freed (k3mla_pool_trim).
//   * Score CTA: three producer threads stream Q and then the page thirds through one ring of 24 KB units;
//     four warps copy Q into TMEM once the last MMA of the unit before has read the old one; three threads
//     issue the score MMAs (A = Q from TMEM, B = the page); eight softmax warps mask, keep a lazily moved
//     reference max, and pass bf16 p to the PV CTA by bulk DSMEM copies.
//   * PV CTA: four producer threads stream the pages' latents again (mostly from L2) as half pages; one
//     thread issues O[rows x 512] += P . C; four warps rescale O when a reference moved and, at a unit's
//     end, take O out of TMEM through two staged boxes while the next unit's MMAs already run; four warps
//     clear what a page holds of unseen tokens.
//   * Unseen tokens.  Their scores are replaced (never multiplied), and in the pages that hold some their
//     latents are cleared in shared memory, because p = 0 times a NaN or infinity there would still be
//     NaN.  In a chunk a token may be seen by some rows of the unit only; then just its NaNs and
//     infinities are cleared: the rows that see it already got NaN from its score.
//
// Every wait is bounded, as in decode.cu: after WAIT_NS it sets K3MLA_DEV_TIMEOUT and the roles run out.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "common.cuh"
#include "decode_core.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace k3 {

template <bool MQ> struct WCfg {
    static constexpr int RPQ = MQ ? 32 : 24;             // rows per 32-lane quarter
    static constexpr int ROWS = 4 * RPQ;                 // rows of a unit
    static constexpr int NUNIT = MQ ? 7 : 8;             // score CTA: ring of 24 KB units
    static constexpr int QPU = MQ ? 1 : 2;               // 64-column chunks of Q in one ring unit
    static constexpr int NQ = (9 + QPU - 1) / QPU;       // ring uses that a unit's Q takes
    static constexpr int QCHUNK = ROWS * 128;            // one chunk of Q, [rows][128 B]
    static constexpr int NPBUF = MQ ? 3 : 4;             // PV CTA: P buffers
    static constexpr int PSTAGE = RPQ * 128;             // score CTA: one softmax warp's P rows (x 64 tokens)
    static constexpr int PT_BYTES = ROWS * 128;          // P [rows][64 tokens] bf16, K-major, 128-byte swizzle
    static constexpr int META_ALPHA = PT_BYTES;          // f32 alpha[rows]
    static constexpr int META_FLAGS = PT_BYTES + 4 * ROWS;     // u32 flags[4]: "some row of quarter w rescaled"
    static constexpr int PCOPY = PT_BYTES + 4 * ROWS + 16;     // bytes sent per page
    static constexpr int PBUF = (PCOPY + 1023) / 1024 * 1024;  // buffer pitch
    static constexpr int BOX = ROWS * 128;               // PV CTA: one write-out box
};
constexpr int WN_S = 3;        // S buffers, one MMA issuer each
constexpr int WN_HALF = 4;     // PV CTA: half-page slots, one producer each
// rank 0: warps 0-7 softmax, 8-10 producers, 11-13 MMA issuers, 11-14 copy Q; rank 1: warps 0-3 epilogue,
// 4-7 producers, 9 MMA issuer, 10-13 clear unseen tokens.  Warp 8 allocates TMEM in both.
constexpr int W_THREADS = 480;
constexpr int WW_PROD0 = 8, WW_MMA0 = 11, WW_COPY0 = 11, WW_ALLOC = 8;
constexpr int WW_HPROD0 = 4, WW_PV = 9, WW_CLEAR0 = 10;
// named barriers (0 is __syncthreads): score CTA, the decision hand-off of a quarter's two softmax warps, their
// final combine, the four copy warps; PV CTA, the epilogue warps
constexpr uint32_t WB_HAND = 1, WB_FIN = 9, WB_COPY = 13, WB_OUT = 1;

template <bool MQ> struct __align__(1024) WSmem {
    using C = WCfg<MQ>;
    union {
        struct {
            uint8_t ring[C::NUNIT][THIRD];
            uint8_t pstage[8][C::PSTAGE];
        } c0;
        struct {
            uint8_t ring[WN_HALF][SLOT1];
            uint8_t recv[C::NPBUF][C::PBUF];
            uint8_t box[2][C::BOX];
        } c1;
    } u;
    uint64_t full[8], empty[8];          // the ring of this CTA
    uint64_t s_full[WN_S], s_empty[WN_S];
    uint64_t q_free, q_ready;            // Q of the unit before is no longer read / Q of this unit is in TMEM
    uint64_t p_full[C::NPBUF], p_empty[C::NPBUF];
    uint64_t o_done, epi_req, epi_done, clear_req, clear_done;
    uint64_t l_full[2], rl_free[2];      // 1 / l of every row, by parity of the unit
    float rl[2][C::ROWS];
    float xm[2][4][32], xa[2][4][32];    // reference max after a page and its rescale factor, by page parity
    float fin_l[2][4][32];               // the odd pages' sum of exp, by unit parity
    int32_t unit_loaded[C::NUNIT];       // uses of a ring unit whose load has been issued ...
    int32_t unit_taken[C::NUNIT];        // ... and whose consumer has taken it
    uint32_t tmem_base;
    uint32_t epi_cmd, epi_stage;         // to the epilogue warps: bit 0 rescale O, bit 1 write it out
    int32_t epi_b, epi_s, epi_hb, epi_row0, epi_rows, epi_single;
    uint32_t clear_cmd, clear_slot[2];   // to the clearing warps (0: leave): the page's two half slots, ...
    uint32_t clear_none[2], clear_some[2];  // ... its tokens that no row sees, and those that some rows see
    int32_t abort_flag;
    uint64_t wait_ns;
};

template <bool MQ> constexpr bool wsmem_fits()
{
    using C = WCfg<MQ>;
    static_assert(C::QPU * C::QCHUNK <= THIRD && C::QCHUNK % 1024 == 0 && SLOT1 % 1024 == 0 && C::PBUF % 1024 == 0 &&
                      C::BOX % 1024 == 0,
                  "operand tiles and boxes fit and start 1024-byte aligned");
    static_assert(C::NUNIT <= 8 && WN_HALF <= 8, "barrier arrays");
    static_assert(C::NPBUF * C::PBUF + 2 * C::BOX >= (C::NPBUF - 1) * C::PBUF + 128 * 128,
                  "all 128 rows of the last P buffer, read as the A operand, lie in this CTA's tile area");
    static_assert(sizeof(WSmem<MQ>) + 1024 <= 227 * 1024, "shared memory of one CTA (with alignment slack)");
    return true;
}
static_assert(wsmem_fits<false>() && wsmem_fits<true>(), "shared-memory layouts");

struct WinParams {
    const int32_t* table;
    const int32_t* ctx_len;              // decode
    const int32_t *pos0, *row_start;     // chunk
    float* ws_o;                         // [B][nsplit][96][512] f32 partials (decode, nsplit > 1)
    float2* ws_ml;                       // [B][nsplit][96]: reference max (in log2 units), sum of exp
    int32_t* dev_err;
    int B, R, max_pages, n_pages, n_layers, layer, cap;  // cap: the longest context (min of max_ctx and the table)
    int window, n_sink, split_tokens, nsplit, n_units;
    float kscale;                        // scale * log2(e) > 0
};

// A unit: which rows, which pages.
struct WUnit {
    int b, s, hb;
    int row0, rows;  // chunk: the first token row and how many; decode: 0, 1
    int n0;          // context of the first row (the next rows': one more each, all clamped to the table)
    int npg;         // pages of the unit, 0: nothing to do
    int first;       // the first of them in the list of the pages seen
    int nsp, wp0;    // entry g of that list is logical page g for g < nsp, else g - nsp + wp0
    bool single;     // the unit holds all its rows see: final o_lat
};

__host__ __device__ inline int w_clamp(int n, int cap) { return n < 0 ? 0 : (n > cap ? cap : n); }

// The pages that the rows with contexts n_lo .. n_hi see: how many, and the two numbers of WUnit.
__host__ __device__ inline int w_pages(int n_lo, int n_hi, int window, int n_sink, int& nsp, int& wp0)
{
    nsp = wp0 = 0;
    if (n_hi <= 0) return 0;
    const int lo = n_lo > window ? n_lo - window : 0;
    const int sink = n_sink < n_hi ? n_sink : n_hi;
    wp0 = lo / PAGE;
    nsp = (sink + PAGE - 1) / PAGE;
    if (nsp > wp0) nsp = wp0;
    return nsp + (n_hi + PAGE - 1) / PAGE - wp0;
}

// Unit u (a whole warp, every lane the same answer).
template <bool MQ> __device__ __forceinline__ WUnit w_unit(const WinParams& p, int u, bool report)
{
    WUnit g;
    g.npg = 0;
    g.first = 0;
    g.s = 0;
    g.hb = 0;
    g.row0 = 0;
    g.rows = 1;
    g.single = true;
    int last;
    if constexpr (MQ) {
        // group u / 3 of up to four rows, counted slot by slot: 32 slots a step
        const int gi = u / 3, lane = (int)lane_id();
        g.hb = u % 3;
        int before = 0;
        bool found = false;
        for (int b0 = 0; b0 < p.B && !found; b0 += 32) {
            const int b = b0 + lane;
            int lo = 0, nb = 0;
            if (b < p.B) {
                lo = max(0, p.row_start[b]);
                nb = max(0, min(p.R, p.row_start[b + 1]) - lo);
            }
            const int mine = (nb + 3) / 4;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, before + upto > gi);
            if (past) {
                const int src = __ffs(past) - 1;
                const int j = 4 * (gi - before - __shfl_sync(0xFFFFFFFFu, upto - mine, src));
                g.b = b0 + src;
                g.row0 = __shfl_sync(0xFFFFFFFFu, lo, src) + j;
                g.rows = min(4, __shfl_sync(0xFFFFFFFFu, nb, src) - j);
                found = true;
            }
            before += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
        if (!found) return g;
        const int64_t n0 = (int64_t)p.pos0[g.b] + (g.row0 - p.row_start[g.b]) + 1;
        const int64_t n1 = n0 + g.rows - 1;
        if (report && n1 > p.cap && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_CTX);
        g.n0 = (int)max((int64_t)-4, min(n0, (int64_t)p.cap));
        last = (int)max((int64_t)0, min(n1, (int64_t)p.cap));
    } else {
        g.b = u / p.nsplit;
        g.s = u % p.nsplit;
        const int n = p.ctx_len[g.b];
        if (report && n > p.cap && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_CTX);
        g.n0 = last = w_clamp(n, p.cap);
    }
    const int all = w_pages(max(g.n0, 0), last, p.window, p.n_sink, g.nsp, g.wp0);
    if constexpr (MQ) {
        g.npg = all;
    } else {
        const int per = slot_split(all * PAGE, p.split_tokens) / PAGE;
        g.single = all <= per;
        g.first = g.s * per;
        g.npg = min(per, max(0, all - g.first));
    }
    return g;
}

__device__ __forceinline__ int w_logical(const WUnit& g, int i)
{
    const int e = g.first + i;
    return e < g.nsp ? e : e - g.nsp + g.wp0;
}

__device__ __forceinline__ uint64_t w_low(int k) { return k >= 64 ? ~0ull : (k <= 0 ? 0ull : (1ull << k) - 1ull); }

// Which of the 64 tokens from t0 on a row with context n sees.
__device__ __forceinline__ uint64_t w_seen(const WinParams& p, int n, int t0)
{
    const uint64_t before_n = w_low(n - t0);
    return before_n & (w_low(min(p.n_sink, n) - t0) | ~w_low(max(0, n - p.window) - t0));
}

// The slab row of logical page lp of slot b, or one past the end (read as zeros).
__device__ __forceinline__ int32_t w_page_row(const WinParams& p, int b, int lp)
{
    const int32_t id = p.table[(size_t)b * p.max_pages + lp];
    if (id >= 0 && id < p.n_pages) return (id * p.n_layers + p.layer) * PAGE;
    if (id != -1 && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_BAD_PAGE);
    return p.n_pages * p.n_layers * PAGE;
}

// Producers look 32 pages of a unit up at a time, one a lane.
struct WLookup {
    int32_t row;
    __device__ __forceinline__ int32_t operator()(const WinParams& p, const WUnit& g, int i)
    {
        const int lane = (int)lane_id();
        if ((i & 31) == 0) row = i + lane < g.npg ? w_page_row(p, g.b, w_logical(g, i + lane)) : 0;
        return __shfl_sync(0xFFFFFFFFu, row, i & 31);
    }
};

template <bool MQ>
__device__ __forceinline__ void w_init(WSmem<MQ>& sm, uint32_t rank)
{
    using C = WCfg<MQ>;
    sm.wait_ns = WAIT_NS;
    sm.abort_flag = 0;
    for (int i = 0; i < 8; ++i) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < WN_S; ++i) {
        mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.s_empty[i], 4);
    }
    mbar_init(&sm.q_free, 3);
    mbar_init(&sm.q_ready, 4);
    for (int i = 0; i < C::NPBUF; ++i) {
        mbar_init(&sm.p_full[i], 1);
        mbar_init(&sm.p_empty[i], 1);
    }
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.epi_req, 1);
    mbar_init(&sm.epi_done, 4);
    mbar_init(&sm.clear_req, 1);
    mbar_init(&sm.clear_done, 4);
    for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.l_full[i], 1);
        mbar_init(&sm.rl_free[i], 1);
    }
    for (int i = 0; i < C::NUNIT; ++i) sm.unit_loaded[i] = sm.unit_taken[i] = 0;
    if (rank == 1) {  // expected before anything is sent
        for (int i = 0; i < C::NPBUF; ++i) mbar_arrive_expect_tx(&sm.p_full[i], C::PCOPY);
        for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&sm.l_full[i], 4 * C::ROWS);
    }
}

#define W_FOR_UNITS(u) for (int u = (int)blockIdx.x >> 1; u < p.n_units; u += (int)gridDim.x >> 1)

// ---- score CTA ----------------------------------------------------------------------------

// Producer t: Q uses t, t + 3, ... of a unit, then third t of each of its pages.  The uses of the ring are
// numbered on from unit to unit; use g lies in ring unit g % NUNIT.
template <bool MQ>
__device__ __forceinline__ void w_produce(WSmem<MQ>& sm, const CUtensorMap& tm_page, const CUtensorMap& tm_q,
                                          const WinParams& p, int t)
{
    using C = WCfg<MQ>;
    const bool me = lane_id() == 0;
    bool ok = true;
    int base = 0;
    auto take = [&](int g, uint32_t bytes) -> int {  // the ring unit, ready to be loaded; -1 after an abort
        const int u = g % C::NUNIT, k = g / C::NUNIT;
        if (!wait_count(&sm.unit_loaded[u], k, sm, p.dev_err) ||
            !wait_bar(&sm.empty[u], (uint32_t)(k & 1) ^ 1u, sm, p.dev_err))
            return -1;
        *reinterpret_cast<volatile int32_t*>(&sm.unit_loaded[u]) = k + 1;
        mbar_arrive_expect_tx(&sm.full[u], bytes);
        return u;
    };
    W_FOR_UNITS(un)
    {
        const WUnit g = w_unit<MQ>(p, un, false);
        if (g.npg == 0) continue;
        for (int j = t; j < C::NQ && me && ok; j += 3) {
            const int u = take(base + j, C::QPU * C::QCHUNK);
            if (u < 0) {
                ok = false;
            } else if constexpr (MQ) {
                // heads 32 hb .. of four consecutive token rows (those past the group land in lanes nobody reads)
                tma_load_4d(sm.u.c0.ring[u], &tm_q, 0, 32 * g.hb, g.row0, j, &sm.full[u]);
            } else {
                tma_load_3d(sm.u.c0.ring[u], &tm_q, 0, g.b * H, C::QPU * j, &sm.full[u]);
            }
        }
        base += C::NQ;
        WLookup rows;
        for (int i = 0; i < g.npg; ++i) {
            const int32_t y = rows(p, g, i);
            if (me && ok) {
                const int u = take(base + 3 * i + t, THIRD);
                if (u < 0) ok = false;
                else tma_load_3d(sm.u.c0.ring[u], &tm_page, 0, y, 3 * t, &sm.full[u]);
            }
        }
        base += 3 * g.npg;
    }
    if (!ok) drain_inflight();
}

// Warps WW_COPY0 .. +3: Q of the unit from the ring into TMEM, lane 32 w + l <- row RPQ w + l; then, in the
// first three of them, the score MMAs of the pages i = r (mod 3, counted on from unit to unit).
template <bool MQ>
__device__ __forceinline__ void w_copy_and_score(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase, uint32_t warp)
{
    using C = WCfg<MQ>;
    const int lane = (int)lane_id(), qd = (int)(warp & 3u), r = (int)warp - WW_MMA0;
    const int row = C::RPQ * qd + lane;
    const uint32_t taddr = tbase + ((32u * (uint32_t)qd) << 16) + Q_COL;
    bool ok = true;
    int base = 0, gp = 0, done = 0;  // ring uses, pages and units before this unit
    W_FOR_UNITS(un)
    {
        const WUnit g = w_unit<MQ>(p, un, false);
        if (g.npg == 0) continue;
        // the score MMAs of the unit before have read the old Q
        if (ok && done > 0) ok = __all_sync(0xFFFFFFFFu, wait_bar(&sm.q_free, (uint32_t)(done - 1) & 1u, sm, p.dev_err));
        tc_fence_after();
        for (int j = 0; j < C::NQ; ++j) {
            const int u = (base + j) % C::NUNIT, k = (base + j) / C::NUNIT;
            if (ok)
                ok = __all_sync(0xFFFFFFFFu, wait_count(&sm.unit_taken[u], k, sm, p.dev_err) &&
                                                 wait_bar(&sm.full[u], (uint32_t)(k & 1), sm, p.dev_err));
            if (ok)
#pragma unroll
                for (int cc = 0; cc < C::QPU; ++cc) {
                    const int c = C::QPU * j + cc;
                    if (c >= 9) break;
                    uint32_t v[32];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (lane < C::RPQ)
                            w = *reinterpret_cast<const uint4*>(sm.u.c0.ring[u] + cc * C::QCHUNK + row * 128 +
                                                                ((x ^ (row & 7)) << 4));
                        v[4 * x] = w.x, v[4 * x + 1] = w.y, v[4 * x + 2] = w.z, v[4 * x + 3] = w.w;
                    }
                    tmem_st32(taddr + 32u * (uint32_t)c, v);
                }
            tmem_wait_st();
            named_bar(WB_COPY, 128);  // all four quarters have read the ring unit
            if (warp == WW_COPY0 && lane == 0) {
                *reinterpret_cast<volatile int32_t*>(&sm.unit_taken[u]) = k + 1;
                mbar_arrive(&sm.empty[u]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready);
        base += C::NQ;
        if (r < WN_S && lane == 0 && ok) {
            ok = wait_bar(&sm.q_ready, (uint32_t)done & 1u, sm, p.dev_err);
            tc_fence_after();
            for (int i = (r + WN_S - gp % WN_S) % WN_S; i < g.npg && ok; i += WN_S) {
                const int k = (gp + i) / WN_S;
                if (!wait_bar(&sm.s_empty[r], (uint32_t)(k & 1) ^ 1u, sm, p.dev_err)) {
                    ok = false;
                    break;
                }
                for (int t = 0; t < 3 && ok; ++t) {
                    const int e = base + 3 * i + t, u = e % C::NUNIT, ku = e / C::NUNIT;
                    if (!wait_count(&sm.unit_taken[u], ku, sm, p.dev_err) ||
                        !wait_bar(&sm.full[u], (uint32_t)(ku & 1), sm, p.dev_err)) {
                        ok = false;
                        break;
                    }
                    *reinterpret_cast<volatile int32_t*>(&sm.unit_taken[u]) = ku + 1;
                    tc_fence_after();
                    issue_score_third(tbase, S_COL + 64u * (uint32_t)r, smem_u32(sm.u.c0.ring[u]), t);
                    umma_commit(&sm.empty[u]);
                }
                if (ok) umma_commit(&sm.s_full[r]);
            }
            if (ok) umma_commit(&sm.q_free);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        base += 3 * g.npg;
        gp += g.npg;
        ++done;
    }
    if (!ok) drain_inflight();
}

// Softmax warp (quarter qd, page parity par): thread l = row RPQ qd + l of the pages of its parity.  The
// reference max is a chain through a unit's pages: each warp hands its page's decision (new reference,
// rescale factor) to the other warp of the quarter.  All in log2 units.
template <bool MQ>
__device__ __forceinline__ void w_softmax(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase, uint32_t warp)
{
    using C = WCfg<MQ>;
    const int qd = (int)(warp & 3u), par = (int)(warp >> 2), l = (int)lane_id();
    const int h = C::RPQ * qd + l;
    const bool has_row = l < C::RPQ;
    const uint32_t bar_in = WB_HAND + 2u * (uint32_t)qd + (uint32_t)(par ^ 1);
    const uint32_t bar_out = WB_HAND + 2u * (uint32_t)qd + (uint32_t)par;
    const uint32_t t_lane = tbase + ((32u * (uint32_t)qd) << 16) + S_COL;
    const uint32_t recv0 = mapa(smem_u32(sm.u.c1.recv[0]), 1);
    const uint32_t pfull0 = mapa(smem_u32(&sm.p_full[0]), 1);
    const float TAU2 = TAU * 1.4426950408889634f;
    uint8_t* stage = sm.u.c0.pstage[warp];
    bool ok = true;
    int gp = 0, done = 0, singles = 0;
    W_FOR_UNITS(un)
    {
        const WUnit g = w_unit<MQ>(p, un, warp == 0 && l == 0);
        if (g.npg == 0) continue;
        const int n = MQ ? (qd < g.rows ? w_clamp(g.n0 + qd, p.cap) : 0) : g.n0;  // this quarter's context
        float m_ref = -INFINITY, lsum = 0.f;
        for (int i = (gp & 1) == par ? 0 : 1; i < g.npg; i += 2) {
            const int a = gp + i, r = a % WN_S, k = a / WN_S;
            if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bar(&sm.s_full[r], (uint32_t)(k & 1), sm, p.dev_err));
            uint32_t x[2][32];
            if (ok) {
                tc_fence_after();
                tmem_ld32(t_lane + 64u * (uint32_t)r, x[0]);
                tmem_ld32(t_lane + 64u * (uint32_t)r + 32u, x[1]);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (l == 0) mbar_arrive(&sm.s_empty[r]);
            } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) x[0][q] = x[1][q] = 0xFF800000u;
            }
            const uint64_t seen = w_seen(p, n, PAGE * w_logical(g, i));
            if (seen != ~0ull) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t bits = (uint32_t)(seen >> (32 * e));
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        if (!((bits >> q) & 1u)) x[e][q] = 0xFF800000u;  // -inf
                }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                m4[q & 3] = fmaxf(m4[q & 3], __uint_as_float(x[0][q]));
                m4[q & 3] = fmaxf(m4[q & 3], __uint_as_float(x[1][q]));
            }
            const float pmax = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.kscale;
            float m_prev = -INFINITY;
            if (i > 0) {  // the decision of the page before, from the other warp
                named_bar(bar_in, 64);
                m_prev = sm.xm[(a - 1) & 1][qd][l];
                lsum *= sm.xa[(a - 1) & 1][qd][l];
            }
            float alpha = 1.f;
            bool resc = false;
            if (i == 0) {
                m_ref = pmax;
            } else if (pmax > m_prev + TAU2) {
                alpha = ex2_approx(m_prev - pmax);
                lsum *= alpha;
                m_ref = pmax;
                resc = true;
            } else {
                m_ref = m_prev;
            }
            sm.xm[a & 1][qd][l] = m_ref;
            sm.xa[a & 1][qd][l] = alpha;
            named_bar_arrive(bar_out, 64);
            const float mb = m_ref == -INFINITY ? 0.f : m_ref;  // nothing seen yet: every p is 0
            uint32_t sp[32];
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int q = 0; q < 16; ++q) {  // p~ = bf16(2^(s - m_ref)); l sums the f32 values
                    const float e0 = ex2_approx(fmaf(__uint_as_float(x[e][2 * q]), p.kscale, -mb));
                    const float e1 = ex2_approx(fmaf(__uint_as_float(x[e][2 * q + 1]), p.kscale, -mb));
                    part[q & 3] += e0 + e1;
                    sp[16 * e + q] = pack_bf16x2(e0, e1);
                }
            lsum += (part[0] + part[1]) + (part[2] + part[3]);
            // this warp's P rows, once the bulk copy of its page before has read the staging rows
            if (l == 0) bulk_wait_read<0>();
            __syncwarp();
            if (has_row) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(stage + pt_chunk_off(h, j) - qd * C::PSTAGE) =
                        make_uint4(sp[4 * j], sp[4 * j + 1], sp[4 * j + 2], sp[4 * j + 3]);
            }
            fence_proxy_async_cta();  // the bulk copy reads the rows through the async proxy
            __syncwarp();
            const int st = a % C::NPBUF;
            bool freed = false;  // the PV CTA has finished with the buffer's page before
            if (ok) freed = wait_bar(&sm.p_empty[st], (uint32_t)((a / C::NPBUF) & 1) ^ 1u, sm, p.dev_err);
            const uint32_t dst = recv0 + (uint32_t)(st * C::PBUF);
            const uint32_t bar = pfull0 + (uint32_t)(st * sizeof(uint64_t));
            if (freed && l == 0) {
                bulk_copy_to_cluster(dst + (uint32_t)(qd * C::PSTAGE), stage, C::PSTAGE, bar);
                bulk_commit();
            }
            if (freed && has_row) st_async_b32(dst + C::META_ALPHA + 4 * h, __float_as_uint(alpha), bar);
            const uint32_t any = __ballot_sync(0xFFFFFFFFu, resc && has_row);
            if (freed && l == 0) st_async_b32(dst + C::META_FLAGS + 4 * qd, any ? 1u : 0u, bar);
        }
        const int last = gp + g.npg - 1;
        if ((last & 1) != par) {  // the last page's decision, when that page was the other warp's
            named_bar(bar_in, 64);
            m_ref = sm.xm[last & 1][qd][l];
            lsum *= sm.xa[last & 1][qd][l];
        }
        if (par == 1) sm.fin_l[done & 1][qd][l] = lsum;
        named_bar(WB_FIN + (uint32_t)qd, 64);
        if (par == 0 && ok && !aborted(sm)) {
            const float ltot = lsum + sm.fin_l[done & 1][qd][l];
            if (g.single) {  // the PV CTA lands o_lat itself
                const int sl = singles & 1;
                // (a row that sees nothing has l = 0; its o_lat is not used)
                if (wait_bar(&sm.rl_free[sl], (uint32_t)((singles >> 1) & 1) ^ 1u, sm, p.dev_err, true) && has_row)
                    st_async_b32(mapa(smem_u32(&sm.rl[sl][h]), 1), __float_as_uint(1.f / ltot),
                                 mapa(smem_u32(&sm.l_full[sl]), 1));
            } else if (has_row) {
                p.ws_ml[((size_t)g.b * p.nsplit + g.s) * H + h] = make_float2(m_ref, ltot);
            }
        }
        singles += g.single;
        gp += g.npg;
        ++done;
    }
    // this warp's bulk copies have landed, and so have the PV CTA's last releases of its P buffers
    if (l == 0) {
        bulk_wait<0>();
        for (int a = max(0, gp - C::NPBUF); a < gp && !aborted(sm); ++a)
            wait_bar(&sm.p_empty[a % C::NPBUF], (uint32_t)((a / C::NPBUF) & 1), sm, p.dev_err);
    }
}

// ---- PV CTA -------------------------------------------------------------------------------

// Producer q: the half pages u = q (mod WN_HALF), counted on from unit to unit.
template <bool MQ>
__device__ __forceinline__ void w_produce_halves(WSmem<MQ>& sm, const CUtensorMap& tm_page8, const WinParams& p, int q)
{
    const uint64_t pol = policy_evict_first();  // the last reader of the latent in this unit
    const bool me = lane_id() == 0;
    bool ok = true;
    int gp = 0;
    W_FOR_UNITS(un)
    {
        const WUnit g = w_unit<MQ>(p, un, false);
        WLookup rows;
        for (int i = 0; i < g.npg; ++i) {
            const int32_t y = rows(p, g, i);
            const int e = 2 * (gp + i) + (q & 1), k = e / WN_HALF;
            if (!me || !ok || e % WN_HALF != q) continue;
            if (!wait_bar(&sm.empty[q], (uint32_t)(k & 1) ^ 1u, sm, p.dev_err)) {
                ok = false;
                continue;
            }
            mbar_arrive_expect_tx(&sm.full[q], SLOT1);
            tma_load_3d_hint(sm.u.c1.ring[q], &tm_page8, 0, y + HALF * (q & 1), 0, &sm.full[q], pol);
        }
        gp += g.npg;
    }
    if (!ok) drain_inflight();
}

// The tokens of a page that no row of the unit sees, and those that only some of its rows see.
template <bool MQ>
__device__ __forceinline__ void w_unseen(const WinParams& p, const WUnit& g, int t0, uint64_t& none, uint64_t& some)
{
    uint64_t any = 0, all = ~0ull;
    for (int w = 0; w < (MQ ? g.rows : 1); ++w) {
        const uint64_t s = w_seen(p, MQ ? w_clamp(g.n0 + w, p.cap) : g.n0, t0);
        any |= s;
        all &= s;
    }
    none = ~any;
    some = any & ~all;
}

template <bool MQ>
__device__ __forceinline__ void w_issue_pv(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase)
{
    using C = WCfg<MQ>;
    const bool me = lane_id() == 0;
    bool ok = true, pending = false;  // pending: the epilogue has not yet taken the unit before out of TMEM
    uint32_t epi_k = 0, clear_k = 0;
    int gp = 0;
    W_FOR_UNITS(un)
    {
        const WUnit g = w_unit<MQ>(p, un, false);
        if (g.npg == 0) continue;
        for (int i = 0; i < g.npg && me && ok; ++i) {
            const int a = gp + i, st = a % C::NPBUF;
            const int q0 = (2 * a) % WN_HALF, q1 = q0 + 1;
            const uint32_t ph = (uint32_t)((2 * a / WN_HALF) & 1);
            if (!wait_bar(&sm.full[q0], ph, sm, p.dev_err) || !wait_bar(&sm.full[q1], ph, sm, p.dev_err)) {
                ok = false;
                break;
            }
            uint64_t none, some;
            w_unseen<MQ>(p, g, PAGE * w_logical(g, i), none, some);
            if (none | some || i == 0) {  // (with a unit's first page always: the clearing warps' waits stay short)
                sm.clear_cmd = 1u;
                sm.clear_slot[0] = (uint32_t)q0;
                sm.clear_slot[1] = (uint32_t)q1;
                sm.clear_none[0] = (uint32_t)none;
                sm.clear_none[1] = (uint32_t)(none >> 32);
                sm.clear_some[0] = (uint32_t)some;
                sm.clear_some[1] = (uint32_t)(some >> 32);
                mbar_arrive(&sm.clear_req);
                ok = wait_bar(&sm.clear_done, clear_k++ & 1u, sm, p.dev_err);
                if (!ok) break;
            }
            if (!wait_bar(&sm.p_full[st], (uint32_t)((a / C::NPBUF) & 1), sm, p.dev_err, true)) {
                ok = false;
                break;
            }
            fence_proxy_async_cta();  // the P tile came through DSMEM copies; the MMA reads it
            const volatile uint32_t* rf = reinterpret_cast<const volatile uint32_t*>(sm.u.c1.recv[st] + C::META_FLAGS);
            const bool resc = i > 0 && (rf[0] | rf[1] | rf[2] | rf[3]) != 0u;
            if (pending || resc) {
                if (pending) ok = wait_bar(&sm.epi_done, epi_k++ & 1u, sm, p.dev_err);
                pending = false;
                if (ok && resc) {
                    umma_commit(&sm.o_done);
                    sm.epi_cmd = 1u;
                    sm.epi_stage = (uint32_t)st;
                    mbar_arrive(&sm.epi_req);
                    ok = wait_bar(&sm.epi_done, epi_k++ & 1u, sm, p.dev_err);
                }
                if (!ok) break;
            }
            tc_fence_after();
            // each half-page slot goes back to its producer once the MMAs that read it are done
            issue_pv_half(tbase, smem_u32(sm.u.c1.ring[q0]), smem_u32(sm.u.c1.recv[st]), 0, i > 0);
            umma_commit(&sm.empty[q0]);
            issue_pv_half(tbase, smem_u32(sm.u.c1.ring[q1]), smem_u32(sm.u.c1.recv[st]), 1, i > 0);
            umma_commit(&sm.empty[q1]);
            mbar_arrive_expect_tx(&sm.p_full[st], C::PCOPY);
            umma_commit_mc(&sm.p_empty[st], (uint16_t)0x1);
        }
        if (me && ok) {  // O of the unit is complete: to be written out
            umma_commit(&sm.o_done);
            sm.epi_cmd = 2u;
            sm.epi_b = g.b;
            sm.epi_s = g.s;
            sm.epi_hb = g.hb;
            sm.epi_row0 = g.row0;
            sm.epi_rows = g.rows;
            sm.epi_single = g.single ? 1 : 0;
            mbar_arrive(&sm.epi_req);
            pending = true;
        }
        gp += g.npg;
    }
    if (!ok) {
        drain_inflight();
        *reinterpret_cast<volatile int32_t*>(&sm.abort_flag) = 1;
    } else if (me) {  // the clearing and epilogue warps leave
        if (pending) ok = wait_bar(&sm.epi_done, epi_k++ & 1u, sm, p.dev_err);
        sm.epi_cmd = 0u;
        mbar_arrive(&sm.epi_req);
        sm.clear_cmd = 0u;
        mbar_arrive(&sm.clear_req);
    }
}

// Warps WW_CLEAR0 .. +3: in the two half-page slots named, the latents of tokens that no row sees become
// zero, and the NaNs and infinities of those that some rows see.
template <bool MQ> __device__ __forceinline__ void w_clear(WSmem<MQ>& sm, const WinParams& p, uint32_t warp)
{
    const int tid = ((int)warp - WW_CLEAR0) * 32 + (int)lane_id();
    for (uint32_t k = 0;; ++k) {
        const bool got = wait_bar(&sm.clear_req, k & 1u, sm, p.dev_err);
        if (!__all_sync(0xFFFFFFFFu, got)) break;
        const volatile uint32_t *vn = sm.clear_none, *vs = sm.clear_some;
        const uint64_t none = (uint64_t)vn[1] << 32 | vn[0], some = (uint64_t)vs[1] << 32 | vs[0];
        if (!*reinterpret_cast<const volatile uint32_t*>(&sm.clear_cmd)) break;
        // 64 tokens x 64 pieces of 16 bytes: a warp takes half a token's pieces at a time
        for (int e = tid; (none | some) && e < PAGE * 64; e += 128) {
            const int t = e >> 6, piece = e & 63;
            if (!((none | some) >> t & 1ull)) continue;
            const uint32_t slot = reinterpret_cast<const volatile uint32_t*>(sm.clear_slot)[t >> 5];
            uint4* at = reinterpret_cast<uint4*>(sm.u.c1.ring[slot] + (piece >> 3) * HCHUNK + (t & 31) * 128 + (piece & 7) * 16);
            if (none >> t & 1ull) {
                *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
                uint4 v = *at;
                auto finite = [](uint32_t w) {  // bf16 with all exponent bits set: NaN or infinity
                    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
                    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
                    return w;
                };
                v.x = finite(v.x), v.y = finite(v.y), v.z = finite(v.z), v.w = finite(v.w);
                *at = v;
            }
        }
        fence_proxy_async_cta();
        __syncwarp();
        if (lane_id() == 0) mbar_arrive(&sm.clear_done);
    }
}

// O [rows x 512] f32 leaves TMEM, 64 dims at a time, through two staged boxes of 128-byte rows and bulk
// tensor stores: bf16 hi and lo of o_lat = O / l when the unit is all its rows see, else two 32-dim boxes
// of the f32 partial.  The TMEM is handed back after its last load; the stores run on behind.
template <bool MQ>
__device__ __forceinline__ void w_write_out(WSmem<MQ>& sm, const CUtensorMap& tm_out, const CUtensorMap& tm_row,
                                            const WinParams& p, uint32_t t_lane, int row, int singles)
{
    using C = WCfg<MQ>;
    const int b = sm.epi_b, s = sm.epi_s, hb = sm.epi_hb, row0 = sm.epi_row0, rows = sm.epi_rows;
    const bool single = sm.epi_single != 0, has_row = row < C::ROWS;
    float r = 1.f;
    if (single) {
        if (has_row) r = sm.rl[singles & 1][row];
        named_bar(WB_OUT, 128);
        if (threadIdx.x == 0) {  // the slot of 1 / l is free again
            mbar_arrive_expect_tx(&sm.l_full[singles & 1], 4 * C::ROWS);
            mbar_arrive_remote(mapa(smem_u32(&sm.rl_free[singles & 1]), 0));
        }
    }
    const uint32_t sw = (uint32_t)(row & 7);
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
        uint32_t v[2][32];
        tmem_ld32(t_lane + 64u * (uint32_t)k, v[0]);
        tmem_ld32(t_lane + 64u * (uint32_t)k + 32u, v[1]);
        tmem_wait_ld();
        if (k == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane_id() == 0) mbar_arrive(&sm.epi_done);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint4 q[8];
            if (single) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t* at = &v[i >> 2][8 * (i & 3) + 2 * e];
                        float f0 = __uint_as_float(at[0]), f1 = __uint_as_float(at[1]);
                        if (x == 0) {  // hi; what it leaves stays for lo
                            f0 *= r, f1 *= r;
                            w[e] = pack_bf16x2(f0, f1);
                            at[0] = __float_as_uint(f0 - bf16lo_to_f32(w[e]));
                            at[1] = __float_as_uint(f1 - bf16hi_to_f32(w[e]));
                        } else {
                            w[e] = pack_bf16x2(f0, f1);
                        }
                    }
                    q[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = make_uint4(v[x][4 * i], v[x][4 * i + 1], v[x][4 * i + 2], v[x][4 * i + 3]);
            }
            if (threadIdx.x == 0) bulk_wait_read<1>();  // the box's store before has read it
            __syncwarp();
            named_bar(WB_OUT, 128);
            uint8_t* box = sm.u.c1.box[x];
            if (has_row)
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(box + row * 128 + (((uint32_t)i ^ sw) << 4)) = q[i];
            fence_proxy_async_cta();
            __syncwarp();
            named_bar(WB_OUT, 128);
            if (threadIdx.x == 0) {
                if constexpr (MQ) {  // o_lat [2][96][R][512] as (512 dims, 96 heads, R rows, 2)
                    if (rows == 4)
                        tma_store_4d(&tm_out, box, 64 * k, 32 * hb, row0, x);
                    else
                        for (int w = 0; w < rows; ++w) tma_store_4d(&tm_row, box + 32 * w * 128, 64 * k, 32 * hb, row0 + w, x);
                } else if (single) {  // o_lat [2][96][B][512] as (512 dims, B slots, 96 heads, 2)
                    tma_store_4d(&tm_out, box, 64 * k, b, 0, x);
                } else {  // partials [B][nsplit][96][512] f32 as (512 dims, rows)
                    tma_store_2d(&tm_row, box, 64 * k + 32 * x, (b * p.nsplit + s) * H);
                }
                bulk_commit();
            }
        }
    }
}

template <bool MQ>
__device__ __forceinline__ void w_epilogue(WSmem<MQ>& sm, const CUtensorMap& tm_out, const CUtensorMap& tm_row,
                                           const WinParams& p, uint32_t tbase, uint32_t warp)
{
    using C = WCfg<MQ>;
    const int lane = (int)lane_id(), row = 32 * (int)warp + lane;
    const uint32_t t_lane = tbase + ((32u * warp) << 16);
    uint32_t od = 0;
    int singles = 0;
    for (uint32_t k = 0;; ++k) {
        // (an abort may reach one warp and not another: they agree on it, so that all or none pass the
        // write-out's barriers)
        bool got = __all_sync(0xFFFFFFFFu, wait_bar(&sm.epi_req, k & 1u, sm, p.dev_err));
        if (named_bar_any(WB_OUT, 128, !got)) break;
        const uint32_t cmd = *reinterpret_cast<volatile uint32_t*>(&sm.epi_cmd);
        if (!cmd) break;
        got = wait_bar(&sm.o_done, od++ & 1u, sm, p.dev_err);
        if ((cmd & 2u) && sm.epi_single)
            got = got && wait_bar(&sm.l_full[singles & 1], (uint32_t)(singles >> 1) & 1u, sm, p.dev_err, true);
        got = __all_sync(0xFFFFFFFFu, got);
        if (named_bar_any(WB_OUT, 128, !got)) break;
        tc_fence_after();
        if (cmd & 2u) {
            const bool single = sm.epi_single != 0;
            w_write_out<MQ>(sm, tm_out, tm_row, p, t_lane, row, singles);
            singles += single;
            continue;
        }
        const float* al = reinterpret_cast<const float*>(sm.u.c1.recv[sm.epi_stage] + C::META_ALPHA);
        const float f = row < C::ROWS ? al[row] : 1.f;
        if (__any_sync(0xFFFFFFFFu, f != 1.f)) {  // some row of this warp moved its reference
#pragma unroll 1
            for (int cb = 0; cb < LORA / 32; ++cb) {
                uint32_t v[32];
                tmem_ld32(t_lane + 32u * (uint32_t)cb, v);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * f);
                tmem_st32(t_lane + 32u * (uint32_t)cb, v);
            }
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.epi_done);
    }
    if (threadIdx.x == 0) bulk_wait<0>();
}

// ---- the kernel ---------------------------------------------------------------------------

template <bool MQ>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(128)
    k3mla_window_kernel(const __grid_constant__ CUtensorMap tm_page, const __grid_constant__ CUtensorMap tm_page8,
                        const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_out,
                        const __grid_constant__ CUtensorMap tm_row, const WinParams p)
{
    extern __shared__ uint8_t smem_raw[];
    WSmem<MQ>& sm = *reinterpret_cast<WSmem<MQ>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t rank = cluster_ctarank(), warp = threadIdx.x >> 5, lane = lane_id();
    if (threadIdx.x == 0) {
        w_init(sm, rank);
        fence_mbarrier_init_cluster();
    }
    if (warp == WW_ALLOC) {
        tmem_alloc(&sm.tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 4 && lane == 0) {
        tma_prefetch_desc(rank == 0 ? &tm_page : &tm_page8);
        tma_prefetch_desc(rank == 0 ? &tm_q : &tm_out);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    griddep_wait();
    griddep_launch_dependents();
    if (rank == 0) {
        if (warp < 8) w_softmax<MQ>(sm, p, tbase, warp);
        else if (warp < WW_MMA0) w_produce<MQ>(sm, tm_page, tm_q, p, (int)warp - WW_PROD0);
        else w_copy_and_score<MQ>(sm, p, tbase, warp);
    } else {
        if (warp < 4) w_epilogue<MQ>(sm, tm_out, tm_row, p, tbase, warp);
        else if (warp < WW_HPROD0 + WN_HALF) w_produce_halves<MQ>(sm, tm_page8, p, (int)warp - WW_HPROD0);
        else if (warp == WW_PV) w_issue_pv<MQ>(sm, p, tbase);
        else if (warp >= WW_CLEAR0 && warp < WW_CLEAR0 + 4) w_clear<MQ>(sm, p, warp);
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == WW_ALLOC) tmem_dealloc(tbase, TMEM_COLS);
}

// ---- merge of splits (decode) ---------------------------------------------------------------

constexpr int WM_THREADS = 128;

// A row (slot, head) per CTA, four dims a thread: o_lat = sum_i w_i O_i / sum_i w_i l_i with w_i = 2^(m_i - max),
// i ascending, landed as bf16 hi + lo.  The order depends on the slot's own splits only.
__global__ void __launch_bounds__(WM_THREADS) k3mla_window_merge_kernel(const WinParams p, uint16_t* olat)
{
    const int h = blockIdx.x, b = blockIdx.y, d = 4 * (int)threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    int nsp, wp0;
    const int n = w_clamp(p.ctx_len[b], p.cap);
    const int all = w_pages(n, n, p.window, p.n_sink, nsp, wp0);
    const int per = slot_split(all * PAGE, p.split_tokens) / PAGE, ns = (all + per - 1) / per;
    if (ns <= 1) return;  // landed by the split itself
    const float2* ml = p.ws_ml + (size_t)b * p.nsplit * H + h;
    const float* o = p.ws_o + ((size_t)b * p.nsplit * H + h) * LORA + d;
    float m = -INFINITY;
    for (int i = 0; i < ns; ++i) m = fmaxf(m, ml[(size_t)i * H].x);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < ns; ++i) {
        const float2 rec = ml[(size_t)i * H];
        const float4 v = *reinterpret_cast<const float4*>(o + (size_t)i * H * LORA);
        const float w = ex2_approx(rec.x - m);
        l = fmaf(w, rec.y, l);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
    }
    const float r = 1.f / l;
    acc.x *= r, acc.y *= r, acc.z *= r, acc.w *= r;
    const uint2 hi = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    const uint2 lo = make_uint2(pack_bf16x2(acc.x - bf16lo_to_f32(hi.x), acc.y - bf16hi_to_f32(hi.x)),
                                pack_bf16x2(acc.z - bf16lo_to_f32(hi.y), acc.w - bf16hi_to_f32(hi.y)));
    uint16_t* out = olat + ((size_t)h * p.B + b) * LORA + d;
    *reinterpret_cast<uint2*>(out) = hi;
    *reinterpret_cast<uint2*>(out + (size_t)H * p.B * LORA) = lo;
}

// ---- W_UV expansion ---------------------------------------------------------------------------

// OUT_h^T [128 v x 64 rows] = W_UV[h] [128 x 512] . (hi + lo)^T [512 x 64], a CTA per head taking tiles of 64
// rows in turn with W_UV[h] resident (128 KB, read before the grid wait: a weight).  o_lat streams through
// a ring of 64-dim chunks, hi and lo beside each other; two accumulators, so that a tile's outputs leave while
// the next one's MMAs run.
constexpr int WX_TILE = 64;
constexpr int WX_RING = 4;
constexpr int WX_CHUNK = WX_TILE * 128;               // one plane of a chunk
constexpr int WX_A = 8 * VH * 128;                    // W_UV[h]
constexpr int WX_OUT = WX_TILE * VH * 2;              // a tile's bf16 outputs
constexpr int WX_SMEM = WX_A + WX_RING * 2 * WX_CHUNK + WX_OUT + 1024;
constexpr int WX_EPI = 8;                             // epilogue warps 2..9
constexpr int WX_THREADS = 32 * (2 + WX_EPI);
static_assert(WX_SMEM <= 227 * 1024, "shared memory");

struct WxSmem {
    uint64_t w_full, b_full[WX_RING], b_empty[WX_RING], d_full[2], d_empty[2];
    uint32_t tmem_base;
    int32_t abort_flag;
    uint64_t wait_ns;
    int32_t valid[WX_TILE];
};

struct WxParams {
    const int32_t *ctx_len, *pos0, *row_start;  // decode: ctx_len; chunk: pos0 and row_start
    uint16_t* out;
    int32_t* dev_err;
    int B, R, cap;  // R: the rows of o_lat and out (decode: B)
};

// Whether row r sees any token.
__device__ __forceinline__ bool wx_valid(const WxParams& p, int r)
{
    if (r >= p.R) return false;
    if (p.ctx_len) return min(p.ctx_len[r], p.cap) > 0;
    int lo = 0, hi = p.B;  // the last slot with row_start[b] <= r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.row_start[mid] <= r) lo = mid;
        else hi = mid;
    }
    return r >= p.row_start[lo] && r < p.row_start[lo + 1] && (int64_t)p.pos0[lo] + (r - p.row_start[lo]) >= 0;
}

__global__ void __launch_bounds__(WX_THREADS, 1)
    k3mla_window_expand_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_o,
                               const WxParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ WxSmem sm;
    uint8_t* sa = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sb = sa + WX_A;
    uint16_t* so = reinterpret_cast<uint16_t*>(sb + WX_RING * 2 * WX_CHUNK);
    const int h = blockIdx.x, warp = threadIdx.x >> 5, lane = (int)lane_id();
    const int tiles = (p.R + WX_TILE - 1) / WX_TILE;
    if (threadIdx.x == 0) {
        sm.abort_flag = 0;
        sm.wait_ns = WAIT_NS;
        mbar_init(&sm.w_full, 1);
        for (int i = 0; i < WX_RING; ++i) {
            mbar_init(&sm.b_full[i], 1);
            mbar_init(&sm.b_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_empty[i], WX_EPI);
        }
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, 2 * WX_TILE);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&sm.w_full, WX_A);
            for (int c = 0; c < 8; ++c)
                tma_load_3d_hint(sa + c * (VH * 128), &tm_w, 0, h * WROWS_PER_HEAD + NOPE, c, &sm.w_full,
                                 policy_evict_first());
            griddep_wait();
            int g = 0;
            for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y)
                for (int c = 0; c < 8 && ok; ++c, ++g) {
                    const int s = g % WX_RING;
                    ok = wait_bar(&sm.b_empty[s], (uint32_t)((g / WX_RING) & 1) ^ 1u, sm, p.dev_err);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sm.b_full[s], 2 * WX_CHUNK);
                    for (int x = 0; x < 2; ++x)  // rows past the batch are the next head's, or zeros: not stored
                        tma_load_3d(sb + (2 * s + x) * WX_CHUNK, &tm_o, 0, (x * H + h) * p.R + t * WX_TILE, c, &sm.b_full[s]);
                }
            if (!ok) drain_inflight();
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc_bf16(128, WX_TILE, 0, 0);
            griddep_wait();  // (the bounded waits below start when o_lat is there)
            ok = wait_bar(&sm.w_full, 0, sm, p.dev_err);
            int g = 0, it = 0;
            for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y, ++it) {
                ok = wait_bar(&sm.d_empty[it & 1], (uint32_t)((it >> 1) & 1) ^ 1u, sm, p.dev_err);
                for (int c = 0; c < 8 && ok; ++c, ++g) {
                    const int s = g % WX_RING;
                    ok = wait_bar(&sm.b_full[s], (uint32_t)((g / WX_RING) & 1), sm, p.dev_err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = make_sdesc(smem_u32(sa + c * (VH * 128)), 16, 1024);
                    for (int x = 0; x < 2; ++x) {
                        const uint64_t bd = make_sdesc(smem_u32(sb + (2 * s + x) * WX_CHUNK), 16, 1024);
                        for (int ks = 0; ks < 4; ++ks)
                            umma_ss(tbase + (uint32_t)(WX_TILE * (it & 1)), ad + 2u * ks, bd + 2u * ks, idesc,
                                    (c | x | ks) != 0);
                    }
                    umma_commit(&sm.b_empty[s]);
                }
                if (ok) umma_commit(&sm.d_full[it & 1]);
            }
            if (!ok) drain_inflight();
        }
    } else {
        griddep_wait();
        griddep_launch_dependents();
        const int q = warp & 3, cg = (warp - 2) >> 2, tid = (int)threadIdx.x - 64, v = 32 * q + lane;
        int it = 0;
        for (int t = blockIdx.y; t < tiles; t += gridDim.y, ++it) {
            const int r0 = t * WX_TILE;
            if (tid < WX_TILE) sm.valid[tid] = wx_valid(p, r0 + tid);
            if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bar(&sm.d_full[it & 1], (uint32_t)(it >> 1) & 1u, sm, p.dev_err));
            if (ok) {
                tc_fence_after();
                uint32_t acc[32];
                tmem_ld32(tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)(WX_TILE * (it & 1) + 32 * cg), acc);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.d_empty[it & 1]);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    so[(32 * cg + j) * VH + v] = (uint16_t)(pack_bf16x2(__uint_as_float(acc[j]), 0.f) & 0xFFFFu);
            }
            named_bar(1, 32 * WX_EPI);
            if (ok)
                for (int e = tid; e < WX_TILE * (VH / 8); e += 32 * WX_EPI) {
                    const int r = e / (VH / 8), k = e % (VH / 8);
                    if (r0 + r < p.R) {
                        const uint4 x = reinterpret_cast<const uint4*>(so + r * VH)[k];
                        reinterpret_cast<uint4*>(p.out + ((size_t)(r0 + r) * H + h) * VH)[k] =
                            sm.valid[r] ? x : make_uint4(0u, 0u, 0u, 0u);
                    }
                }
            named_bar(1, 32 * WX_EPI);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, 2 * WX_TILE);
}

// ---- host --------------------------------------------------------------------------------------

static size_t w_up(size_t x) { return (x + 255) & ~size_t(255); }

// The most pages a slot of at most cap tokens can see, and the splits that makes.
static long long w_max_pages(int cap, int window, int n_sink)
{
    const long long all = ((long long)cap + PAGE - 1) / PAGE;
    const long long sink = ((long long)std::min(n_sink, cap) + PAGE - 1) / PAGE;
    const long long win = ((long long)std::min(window, cap) + PAGE - 2) / PAGE + 1;
    return std::min(all, sink + win);
}

static int w_nsplit(int cap, int window, int n_sink, int split_tokens)
{
    return launch_nsplit((int)std::min<long long>(w_max_pages(cap, window, n_sink) * PAGE, 0x7FFFFF00), split_tokens);
}

struct WinWs {
    size_t olat, o, ml, total;
};
static WinWs w_layout(long long rows, int nsplit)
{
    WinWs w;
    w.olat = 0;
    w.o = w_up((size_t)rows * H * LORA * 2 * 2);
    w.ml = w.o + (nsplit > 1 ? w_up((size_t)rows * nsplit * H * LORA * 4) : 0);
    w.total = w.ml + (nsplit > 1 ? w_up((size_t)rows * nsplit * H * 8) : 0);
    return w;
}

static int sm_count()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

static bool w_scale(uint16_t bits, float* kscale)
{
    uint32_t u = (uint32_t)bits << 16;
    float f;
    std::memcpy(&f, &u, 4);
    if (!(f > 0.f) || (bits & 0x7F80) == 0x7F80) return false;
    *kscale = (float)((double)f * 1.4426950408889634);
    return true;
}

template <bool MQ>
static int w_launch(const uint16_t* q_abs, const uint16_t* slab, const uint16_t* w_kv_b, uint16_t* out, uint8_t* ws,
                    const WinWs& wl, WinParams& p, cudaStream_t st)
{
    using C = WCfg<MQ>;
    uint16_t* olat = reinterpret_cast<uint16_t*>(ws + wl.olat);
    p.ws_o = p.nsplit > 1 ? reinterpret_cast<float*>(ws + wl.o) : nullptr;
    p.ws_ml = p.nsplit > 1 ? reinterpret_cast<float2*>(ws + wl.ml) : nullptr;
    CUtensorMap tm_page, tm_page8, tm_q, tm_out, tm_row, tm_w, tm_o;
    const uint64_t slab_rows = (uint64_t)p.n_pages * p.n_layers * PAGE, R = (uint64_t)p.R;
    int rc = make_tmap_slab_3d(&tm_page, slab, slab_rows, ROW, 9, PAGE, 3);
    if (!rc) rc = make_tmap_slab_3d(&tm_page8, slab, slab_rows, ROW, 9, HALF, 8);
    if (rc) return rc;
    if (MQ) {
        {   // q_abs as (64 elements, 96 heads, R rows, 9 chunks): a chunk of 32 heads of four token rows
            const uint64_t dims[4] = {64, H, R, 9}, strides[3] = {ROW * 2, (uint64_t)H * ROW * 2, 128};
            const uint32_t box[4] = {64, 32, 4, 1};
            rc = make_tmap_store(&tm_q, false, 4, q_abs, dims, strides, box, true);
        }
        const uint64_t dims[4] = {LORA, H, R, 2}, strides[3] = {R * LORA * 2, LORA * 2, (uint64_t)H * R * LORA * 2};
        const uint32_t box4[4] = {64, 32, 4, 1}, box1[4] = {64, 32, 1, 1};
        if (!rc) rc = make_tmap_store(&tm_out, false, 4, olat, dims, strides, box4, true);
        if (!rc) rc = make_tmap_store(&tm_row, false, 4, olat, dims, strides, box1, true);
    } else {
        rc = make_tmap_slab_3d(&tm_q, q_abs, R * H, ROW, 9, H, C::QPU);
        const uint64_t dims[4] = {LORA, R, H, 2}, strides[3] = {LORA * 2, R * LORA * 2, (uint64_t)H * R * LORA * 2};
        const uint32_t box[4] = {64, 1, H, 1};
        if (!rc) rc = make_tmap_store(&tm_out, false, 4, olat, dims, strides, box, true);
        tm_row = tm_out;
        if (!rc && p.nsplit > 1) {
            const uint64_t d2[2] = {LORA, R * p.nsplit * H}, s2[1] = {LORA * 4};
            const uint32_t b2[2] = {32, H};
            rc = make_tmap_store(&tm_row, true, 2, p.ws_o, d2, s2, b2, true);
        }
    }
    if (!rc) rc = make_tmap_slab_3d(&tm_w, w_kv_b, (uint64_t)H * WROWS_PER_HEAD, LORA, 8, VH, 1);
    if (!rc) rc = make_tmap_slab_3d(&tm_o, olat, 2ull * H * R, LORA, 8, WX_TILE, 1);
    if (rc) return rc;
    static bool attr_done[64] = {}, attr_expand[64] = {};
    const size_t smem = sizeof(WSmem<MQ>) + 1024;
    set_smem_attr(reinterpret_cast<const void*>(k3mla_window_kernel<MQ>), smem, attr_done);
    set_smem_attr(reinterpret_cast<const void*>(k3mla_window_expand_kernel), WX_SMEM, attr_expand);
    const int clusters = std::min(p.n_units, sm_count() / 2);
    rc = launch_pdl(k3mla_window_kernel<MQ>, dim3(2 * clusters), dim3(W_THREADS), smem, st, "k3mla_window_kernel", tm_page,
                    tm_page8, tm_q, tm_out, tm_row, p);
    if (rc) return rc;
    if (p.nsplit > 1) {
        rc = launch_pdl(k3mla_window_merge_kernel, dim3(H, p.B), dim3(WM_THREADS), 0, st, "k3mla_window_merge_kernel", p,
                        olat);
        if (rc) return rc;
    }
    WxParams x;
    x.ctx_len = p.ctx_len, x.pos0 = p.pos0, x.row_start = p.row_start, x.out = out, x.dev_err = p.dev_err;
    x.B = p.B, x.R = p.R, x.cap = p.cap;
    const int tiles = (p.R + WX_TILE - 1) / WX_TILE;
    return launch_pdl(k3mla_window_expand_kernel, dim3(H, tiles >= 6 ? 3 : 1), dim3(WX_THREADS), WX_SMEM, st,
                      "k3mla_window_expand_kernel", tm_w, tm_o, x);
}

// What both entries ask of their common arguments; fills p.
static int w_check(const char* who, const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                   const int32_t* table, int max_pages, const uint16_t* w_kv_b, uint16_t scale_bf16, const uint16_t* out,
                   const void* workspace, int max_ctx, int window, int n_sink, WinParams& p)
{
    std::memset(&p, 0, sizeof(p));
    if (n_pages <= 0 || n_layers <= 0 || layer < 0 || layer >= n_layers || max_pages <= 0 || max_ctx <= 0 || window < 1 ||
        n_sink < 0 || !w_scale(scale_bf16, &p.kscale)) {
        set_error("%s: invalid sizes, window or scale", who);
        return K3MLA_E_INVALID;
    }
    if ((long long)n_pages * n_layers * PAGE + PAGE > 0x7FFFFFFFll) {
        set_error("%s: slab rows exceed the 2^31 TMA row range", who);
        return K3MLA_E_INVALID;
    }
    if (!q_abs || !slab || !table || !w_kv_b || !out || !workspace || !aligned(q_abs, 16) || !aligned(slab, 16) ||
        !aligned(w_kv_b, 16) || !aligned(out, 16) || !aligned(workspace, 256)) {
        set_error("%s: null or misaligned pointer", who);
        return K3MLA_E_INVALID;
    }
    p.table = table;
    p.n_pages = n_pages, p.n_layers = n_layers, p.layer = layer, p.max_pages = max_pages;
    p.cap = (int)std::min<long long>(std::min(max_ctx, 0x7FFFFF00), (long long)max_pages * PAGE);
    p.window = window, p.n_sink = n_sink, p.nsplit = 1;
    return K3MLA_OK;
}

}  // namespace k3

using namespace k3;

extern "C" size_t k3mla_window_decode_workspace_bytes(int B, int max_ctx, int window, int n_sink, int split_tokens)
{
    if (B <= 0 || max_ctx <= 0 || window < 1 || n_sink < 0 || split_tokens < 0 || split_tokens % TILE != 0) return 0;
    return w_layout(B, w_nsplit(max_ctx, window, n_sink, split_tokens)).total;
}

extern "C" int k3mla_window_split_tokens(int B, int max_ctx, int window, int n_sink)
{
    if (B <= 0 || max_ctx <= 0 || window < 1 || n_sink < 0) return TILE;
    // as many splits a slot as give every pair of SMs one, none shorter than a tile
    const long long tiles = (w_max_pages(max_ctx, window, n_sink) * PAGE + TILE - 1) / TILE;
    const long long want = std::max(1, sm_count() / 2 / B);
    return (int)std::min<long long>((tiles + want - 1) / want * TILE, 0x7FFFFFFF / TILE * TILE);
}

extern "C" int k3mla_window_decode(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                                   const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                                   const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                   size_t ws_bytes, int B, int max_ctx, int window, int n_sink, int split_tokens,
                                   int32_t* dev_err, void* stream)
{
    WinParams p;
    if (B < 0 || split_tokens < 0 || split_tokens % TILE != 0) {
        set_error("k3mla_window_decode: invalid sizes, window or scale");
        return K3MLA_E_INVALID;
    }
    if (B == 0) return K3MLA_OK;
    int rc = w_check("k3mla_window_decode", q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, w_kv_b,
                     scale_bf16, out, workspace, max_ctx, window, n_sink, p);
    if (rc) return rc;
    if (!ctx_len) {
        set_error("k3mla_window_decode: null or misaligned pointer");
        return K3MLA_E_INVALID;
    }
    const size_t need = k3mla_window_decode_workspace_bytes(B, max_ctx, window, n_sink, split_tokens);
    if (ws_bytes < need) {
        set_error("k3mla_window_decode: workspace %zu < %zu bytes", ws_bytes, need);
        return K3MLA_E_WORKSPACE;
    }
    const int ns = w_nsplit(max_ctx, window, n_sink, split_tokens);
    if (B > 65535 || (long long)B * ns * H > 0x7FFFFFFFll) {  // the merge's grid; partial-row coordinates
        set_error("k3mla_window_decode: too many slots or splits");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    p.ctx_len = ctx_len;
    p.dev_err = dev_err;
    p.B = p.R = B;
    p.split_tokens = split_tokens;
    p.nsplit = ns;
    p.n_units = B * ns;
    return w_launch<false>(q_abs, slab, w_kv_b, out, reinterpret_cast<uint8_t*>(workspace), w_layout(B, ns), p,
                           reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t k3mla_window_chunk_decode_workspace_bytes(int B, int R, int max_ctx)
{
    if (B <= 0 || R <= 0 || max_ctx <= 0) return 0;
    return w_layout(R, 1).total;
}

extern "C" int k3mla_window_chunk_decode(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                                         const int32_t* block_table, int max_pages_per_slot, const int32_t* pos0,
                                         const int32_t* row_start, int B, int R, const uint16_t* w_kv_b,
                                         uint16_t scale_bf16, uint16_t* out, void* workspace, size_t ws_bytes, int max_ctx,
                                         int window, int n_sink, int32_t* dev_err, void* stream)
{
    WinParams p;
    if (B < 0 || R < 0 || (B == 0 && R > 0)) {
        set_error("k3mla_window_chunk_decode: invalid sizes, window or scale");
        return K3MLA_E_INVALID;
    }
    if (R == 0) return K3MLA_OK;
    int rc = w_check("k3mla_window_chunk_decode", q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot,
                     w_kv_b, scale_bf16, out, workspace, max_ctx, window, n_sink, p);
    if (rc) return rc;
    if (!pos0 || !row_start) {
        set_error("k3mla_window_chunk_decode: null or misaligned pointer");
        return K3MLA_E_INVALID;
    }
    const size_t need = k3mla_window_chunk_decode_workspace_bytes(B, R, max_ctx);
    if (ws_bytes < need) {
        set_error("k3mla_window_chunk_decode: workspace %zu < %zu bytes", ws_bytes, need);
        return K3MLA_E_WORKSPACE;
    }
    const long long units = 3ll * (((long long)R + 3ll * B) / 4);  // sum over slots of ceil(n_b / 4), at most
    if (units > 0x3FFFFFFFll || 2ll * R * H > 0x7FFFFFFFll) {
        set_error("k3mla_window_chunk_decode: too many rows");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    p.pos0 = pos0;
    p.row_start = row_start;
    p.dev_err = dev_err;
    p.B = B;
    p.R = R;
    p.n_units = (int)units;
    return w_launch<true>(q_abs, slab, w_kv_b, out, reinterpret_cast<uint8_t*>(workspace), w_layout(R, 1), p,
                          reinterpret_cast<cudaStream_t>(stream));
}
