// window.cu -- paged absorbed-MLA attention over a sliding window and the first tokens, for sm_103a.
//
// Math: a token row with a context of n tokens (itself the last one) sees the tokens
//     t < min(n_sink, n)   and   max(0, n - window) <= t < n,
// and over those, with cache rows r_t (a -1 block table entry is an all-zero row),
//     s_t   = scale * (q_abs[h] . r_t)        (dot over 576)
//     p     = softmax(s),  o_lat = sum_t p_t r_t[0:512],  out = W_UV[h] o_lat.
// Decode: one token row per slot.  Chunk: several consecutive new token rows per slot.
//
// Numerics.  Scores, maxima and sums are f32.  Four roundings go below that: the p of the second contraction
// to bf16 (the tensor core's operand type; both operands have one type and the cache is bf16), a split's O,
// where there are several, to f16 with a power of two per row on its way to the merge (f32 there would take
// twice the stores and loads), o_lat, the operand of the expansion, to f16 likewise (bf16 here would add as
// much error again as the output's own rounding does), and the output to bf16.  W_UV, bf16, takes part as f16
// with a power of two per row of its own: exact, but for entries below 2^-29 of their row's largest.  What each
// adds, relative to the output in the mean square, emulated at 64 to 4,600 seen tokens: the output's own 0.0017,
// p 0.0009 to 0.0014, o_lat 0.0002, 17 splits' O 0.0001 to 0.0002; together 0.0019 to 0.0022, of which the
// splits' f16 makes 0.00001.
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
//   * Score CTA: the producers stream Q and then the page thirds through one ring of 24 KB units; three
//     threads issue the score MMAs (A = Q from TMEM, B = the page); the softmax warps of each quarter take a page
//     each in turn, mask, keep a lazily moved reference max, and pass bf16 p to the PV CTA by bulk DSMEM copies
//     (and copy a unit's Q into TMEM once the last MMA of the unit before has read the old one).
//   * PV CTA: a producer streams the pages' latents again (mostly from L2) as half pages; one thread issues
//     O[rows x 512] += P . C; eight warps rescale O when a reference moved and, at a unit's end, take O out of
//     TMEM; one plans the units of both CTAs ahead.
//   * Unseen tokens.  Their scores are replaced (never multiplied).  p = 0 times a NaN or an infinity would still be
//     NaN, so where an unseen token's score shows that its row holds one, those among the page's unseen latents
//     become zero in shared memory.  In a chunk a token may be seen by some rows of the unit only: those get a NaN for
//     their p of it (its score may be -inf, whose p is 0, and 0 times the latent that was there is NaN).
//
// Measured, all kernels of a call in a graph of calls: decode of 64 slots over 4,100 seen tokens 69.1 us (324 MB, 0.69 of
// the copy rate), over 1,088 33.2 us, of one slot over 4,100 21.5 us (33 splits); chunks of 16 x 64 rows over 1,024 tokens
// 232 us (1,003 TFLOP/s, 0.52 of the measured bf16 rate), of 1,000 rows over 300 120.8 us (29 of them the expansion).
// Call after call from the host the longer ones take 1 to 4 % more (72.3, 33.4, 21.5, 236.8 and 122.5 us).  Bounds: the page
// stream for long lists of pages (decode 0.85 us a page and cluster, 64 clusters at 5.5 TB/s; chunks 0.67 us, of which
// the score MMAs take 0.57 at their full rate), else the chain through a unit and the expansion behind it (6 us).
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
    // Q in the ring: pieces of 64 columns, of all 96 rows (decode) or of two token rows' 64 (chunk)
    static constexpr int QROWS = MQ ? 64 : 96;
    static constexpr int QPIECE = QROWS * 128;           // [rows][128 B]
    static constexpr int QPU = THIRD / QPIECE;           // pieces of one ring unit: 3 or 2
    static constexpr int NPIECE = 9 * ROWS / QROWS;      // 18 or 9
    static constexpr int NQ = (NPIECE + QPU - 1) / QPU;  // ring uses that a unit's Q takes: 6 or 5
    static constexpr int NPROD = MQ ? 1 : 3;             // score CTA: producers
    static constexpr int NPBUF = MQ ? 3 : 4;             // PV CTA: P buffers
    static constexpr int NPAR = MQ ? 3 : 2;              // score CTA: softmax warps of a quarter, a page each in turn
    static constexpr int W_PROD = 4 * NPAR;              // ... behind them the producers ...
    static constexpr int W_MMA0 = W_PROD + NPROD;        // ... and three MMA issuers
    static constexpr int NISS = 3;
    static_assert(W_MMA0 + NISS <= 16, "the warps of a CTA");
    static constexpr int PSTAGE = RPQ * 128;             // score CTA: one softmax warp's P rows (x 64 tokens)
    static constexpr int PT_BYTES = ROWS * 128;          // P [rows][64 tokens] bf16, K-major, 128-byte swizzle
    static constexpr int META_ALPHA = PT_BYTES;          // f32 alpha[rows]
    static constexpr int META_FLAGS = PT_BYTES + 4 * ROWS;     // u32 flags[4], a quarter each: F_RESCALE, F_NOT_FINITE
    static constexpr int PCOPY = PT_BYTES + 4 * ROWS + 16;     // bytes sent per page
    static constexpr int PBUF = (PCOPY + 1023) / 1024 * 1024;  // buffer pitch
};
constexpr int WN_S = 3;        // S buffers, one MMA issuer each
constexpr int WN_HALF = 5;     // PV CTA: half-page slots
constexpr int W_THREADS = 512;  // 128 registers a thread
// PV CTA: the producer, the MMA issuer, eight warps of the epilogue (0-3 and 6-9: a warp reads the TMEM lanes of its own
// quarter), one that plans the units of both CTAs, one for the rows that see nothing, one that prefetches into L2 (decode)
constexpr int WW_HALVES = 4, WW_PV = 5, WW_EPI1 = 6, WW_PLAN = 10, WW_EMPTY = 11, WW_AHEAD = 12;
constexpr int W_PLANS = 8;         // planned units kept
constexpr uint32_t WB_OUT = 1;     // named barrier of the epilogue warps
constexpr int W_EPI = 8;
constexpr uint32_t F_RESCALE = 1, F_NOT_FINITE = 2;  // a row's reference moved / an unseen token's score is not finite
constexpr uint32_t E_RESCALE = 1, E_WRITE = 2, E_CLEAR = 4;  // what the epilogue warps are asked for

// A unit: which rows, which pages.
struct __align__(16) WUnit {
    int b, s, hb;
    int row0, rows;  // chunk: the first token row and how many; decode: 0, 1
    int n0;          // context of the first row (the next rows': one more each, all clamped to the table)
    int npg;         // pages of the unit, at least one; -1: there are no more units
    int first;       // the first of them in the list of the pages seen
    int nsp, wp0;    // entry g of that list is logical page g for g < nsp, else g - nsp + wp0
    int single;      // the unit holds all its rows see: final o_lat
    int n_hi;        // the last row's context
};

template <bool MQ> struct __align__(1024) WSmem {
    using C = WCfg<MQ>;
    union {
        struct {
            uint8_t ring[C::NUNIT][THIRD];
            uint8_t pstage[4 * C::NPAR][C::PSTAGE];
        } c0;
        struct {
            uint8_t ring[WN_HALF][SLOT1];
            uint8_t recv[C::NPBUF][C::PBUF];
            float rl[2][C::ROWS];          // 1 / l of every row, by parity of the unit; written by the score CTA
            float half_max[2][C::ROWS];    // the rows' largest |O| in each half of the dims
        } c1;
    } u;
    uint64_t full[8], empty[8];          // the ring of this CTA
    uint64_t s_full[WN_S], s_empty[WN_S];
    uint64_t q_free, q_ready;            // Q of the unit before is no longer read / Q of this unit is in TMEM
    uint64_t p_full[C::NPBUF], p_empty[C::NPBUF];
    uint64_t o_done, epi_req, epi_done;
    uint64_t l_full[2], rl_free[2];      // PV CTA's rl, by parity of the unit
    uint64_t hand[4][C::NPAR];           // a quarter's decision on a page, by turn
    uint64_t fin_full[2][4], fin_free[2][4];  // a quarter's sums of exp, by parity of the unit
    float xm[2][4][32];                  // reference max after a page, by parity of the page
    float fin_l[2][C::NPAR][4][32];      // a unit's sums of exp by softmax warp, by parity of the unit
    float fin_m[2][C::NPAR][4][32];      // ... and the reference each is held to
    int32_t unit_loaded[C::NUNIT];       // uses of a ring unit whose load has been issued
    int32_t unit_taken[C::NUNIT];        // uses of a ring unit that their consumer has taken
    int32_t copied[C::NUNIT];            // quarters that have copied their rows of the Q chunk in a ring unit
    WUnit plan[W_PLANS];                 // the units, in order
    uint64_t plan_full[W_PLANS];
    int32_t pv_units, pv_pages;          // PV CTA: units whose MMAs have been issued / pages whose P has arrived
    int32_t ahead_units;                 // PV CTA: units that the prefetching warp is through with
    uint32_t tmem_base;
    uint64_t epi_hidden;                 // to the epilogue warps: the tokens of page epi_page that not all rows see
    uint32_t epi_cmd;                    // ... and what to do, E_ bits
    int32_t epi_page;
    int32_t epi_t0;                      // the first token of that page
    int32_t epi_b, epi_s, epi_hb, epi_row0, epi_rows, epi_n0, epi_single;
    int32_t abort_flag;
    int32_t* dev_err;
    uint64_t wait_ns;
};

template <bool MQ> constexpr bool wsmem_fits()
{
    using C = WCfg<MQ>;
    static_assert(C::QPIECE % 1024 == 0 && SLOT1 % 1024 == 0 && C::PBUF % 1024 == 0,
                  "operand tiles fit and start 1024-byte aligned");
    static_assert(C::NUNIT <= 8 && WN_HALF <= 8, "barrier arrays");
    static_assert(WN_HALF * SLOT1 + (C::NPBUF - 1) * C::PBUF + 128 * 128 <= sizeof(WSmem<MQ>::u),
                  "all 128 rows of the last P buffer, read as the A operand, lie in this CTA's tile area");
    static_assert(sizeof(WSmem<MQ>) + 1024 <= 227 * 1024, "shared memory of one CTA (with alignment slack)");
    return true;
}
static_assert(wsmem_fits<false>() && wsmem_fits<true>(), "shared-memory layouts");

struct WinParams {
    const uint16_t* q_abs;
    const int32_t* table;
    const int32_t* ctx_len;              // decode
    const int32_t *pos0, *row_start;     // chunk
    uint16_t* olat;                      // [96][R][512] f16: o_lat times a power of two per row
    float* oscale;                       // [96][R]: what undoes it; 0 for rows that see nothing
    uint16_t* ws_o;                      // [B][nsplit][96][512] f16: a split's O (decode, nsplit > 1) ...
    float* ws_oscale;                    // [B][nsplit][96]: ... and what undoes its power of two
    float2* ws_ml;                       // [B][nsplit][96]: reference max (in log2 units), sum of exp
    int32_t* dev_err;
    int B, R, max_pages, n_pages, n_layers, layer, cap;  // cap: the longest context (min of max_ctx and the table)
    int window, n_sink, split_tokens, nsplit, n_units;
    float kscale;                        // scale * log2(e) > 0
    uint64_t wait_ns;                    // bounded-wait limit: WAIT_NS, shorter only from the diagnostic entries
    int32_t withhold;                    // diagnostic only, 0 otherwise: the PV CTA never loads the first half of a unit's page k - 1
};

template <bool MQ> __device__ __forceinline__ WSmem<MQ>& w_smem()
{
    extern __shared__ uint8_t smem_raw[];
    return *reinterpret_cast<WSmem<MQ>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

// Bounded wait for a phase of one of this CTA's barriers; false after an abort or when the time runs out.  The
// test is in line (a call where it succeeds cost a fifth of the whole kernel's time), what follows is not.
template <bool MQ> __device__ __noinline__ bool w_wait_slow(uint32_t bar, uint32_t parity)
{
    WSmem<MQ>& sm = w_smem<MQ>();
    const uint64_t t0 = globaltimer();
    for (uint32_t n = 1; !mbar_try_wait_cluster(bar, parity); ++n) {
        if (n & 127u) continue;  // (the clock is slow to read: looked at every time, 1 % of the whole call)
        if (aborted(sm)) return false;
        if (globaltimer() - t0 > sm.wait_ns) {
            *reinterpret_cast<volatile int32_t*>(&sm.abort_flag) = 1;
            if (sm.dev_err) atomicOr(sm.dev_err, (int)K3MLA_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}

template <bool MQ, bool CLUSTER = false> __device__ __forceinline__ bool w_wait(uint64_t* bar, uint32_t parity)
{
    const uint32_t a = smem_u32(bar);
    if (CLUSTER ? mbar_test_wait_cluster(a, parity) : mbar_test_wait(a, parity)) return true;
    return w_wait_slow<MQ>(a, parity);
}

template <bool MQ> __device__ __noinline__ bool w_count_slow(const int32_t* counter, int32_t target)
{
    WSmem<MQ>& sm = w_smem<MQ>();
    return wait_count(counter, target, sm, sm.dev_err);
}

// Bounded wait until a shared counter of this CTA reaches `target`.
template <bool MQ> __device__ __forceinline__ bool w_count(const int32_t* counter, int32_t target)
{
    if (*reinterpret_cast<const volatile int32_t*>(counter) >= target) return true;
    return w_count_slow<MQ>(counter, target);
}

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

// Where the search for a chunk's group stands: a cluster's units come in ascending order, so each search goes on in
// the block of 32 slots where the one before ended, and row_start is gone through once, whatever the number of slots.
struct WScan {
    int b0 = 0, before = 0;  // the block's first slot; the groups of the slots before it
};

// Unit u (a whole warp, every lane the same answer); npg is -1 where neither it nor a later one exists.
template <bool MQ>
__device__ __forceinline__ void w_unit(WUnit& g, const WinParams& p, int u, bool report, WScan& scan)
{
    g.npg = 0;
    g.first = 0;
    g.s = 0;
    g.hb = 0;
    g.row0 = 0;
    g.rows = 1;
    g.single = 1;
    int last;
    if constexpr (MQ) {
        // group u / 3 of up to four rows, counted slot by slot: 32 slots a step
        const int gi = u / 3, lane = (int)lane_id();
        g.hb = u % 3;
        bool found = false;
        while (scan.b0 < p.B) {
            const int b = scan.b0 + lane;
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
            const unsigned past = __ballot_sync(0xFFFFFFFFu, scan.before + upto > gi);
            if (past) {
                const int src = __ffs(past) - 1;
                const int j = 4 * (gi - scan.before - __shfl_sync(0xFFFFFFFFu, upto - mine, src));
                g.b = scan.b0 + src;
                g.row0 = __shfl_sync(0xFFFFFFFFu, lo, src) + j;
                g.rows = min(4, __shfl_sync(0xFFFFFFFFu, nb, src) - j);
                found = true;
                break;
            }
            scan.before += __shfl_sync(0xFFFFFFFFu, upto, 31);
            scan.b0 += 32;
        }
        if (!found) {
            g.npg = -1;
            return;
        }
        const int64_t n0 = (int64_t)p.pos0[g.b] + (g.row0 - p.row_start[g.b]) + 1;
        const int64_t n1 = n0 + g.rows - 1;
        if (report && n1 > p.cap && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_CTX);
        g.n0 = (int)max((int64_t)-4, min(n0, (int64_t)p.cap));  // (the rows' own contexts are clamped again)
        last = (int)max((int64_t)0, min(n1, (int64_t)p.cap));
    } else {
        g.b = u / p.nsplit;
        g.s = u % p.nsplit;
        const int n = p.ctx_len[g.b];
        if (report && n > p.cap && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_CTX);
        g.n0 = last = w_clamp(n, p.cap);
    }
    g.n_hi = last;
    const int all = w_pages(max(g.n0, 0), last, p.window, p.n_sink, g.nsp, g.wp0);
    if constexpr (MQ) {
        g.npg = all;
    } else {
        const int per = slot_split(all * PAGE, p.split_tokens) / PAGE;
        g.single = all <= per;
        g.first = g.s * per;
        g.npg = min(per, max(0, all - g.first));
    }
}

__device__ __forceinline__ int w_logical(const WUnit& g, int i)
{
    const int e = g.first + i;
    return e < g.nsp ? e : e - g.nsp + g.wp0;
}

__device__ __forceinline__ uint64_t w_low(int k) { return k >= 64 ? ~0ull : (k <= 0 ? 0ull : (1ull << k) - 1ull); }

// Which of the 64 tokens from t0 on lie below `end` and are sinks of it or not below `from`.
__device__ __forceinline__ uint64_t w_between(const WinParams& p, int from, int end, int t0)
{
    return w_low(end - t0) & (w_low(min(p.n_sink, end) - t0) | ~w_low(max(0, from) - t0));
}

// Whether rows with contexts n_lo .. n_hi all see the whole page at t0 (most pages: no masks to work out).
__device__ __forceinline__ bool w_whole(const WinParams& p, int n_lo, int n_hi, int t0)
{
    return t0 + PAGE <= n_lo && (t0 >= n_hi - p.window || t0 + PAGE <= p.n_sink);
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
__device__ __forceinline__ void w_init(WSmem<MQ>& sm, uint32_t rank, const WinParams& p)
{
    using C = WCfg<MQ>;
    sm.wait_ns = p.wait_ns;
    sm.dev_err = p.dev_err;
    sm.abort_flag = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < WN_S; ++i) {
        mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.s_empty[i], 4);
    }
    for (int i = 0; i < 4 * C::NPAR; ++i) mbar_init(&sm.hand[i / C::NPAR][i % C::NPAR], 1);
    mbar_init(&sm.q_free, C::NISS);
    mbar_init(&sm.q_ready, 4 * C::NPAR);
    for (int i = 0; i < C::NPBUF; ++i) {
        mbar_init(&sm.p_full[i], 1);
        mbar_init(&sm.p_empty[i], 1);
    }
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.epi_req, 1);
    mbar_init(&sm.epi_done, W_EPI);
    for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.l_full[i], 1);
        mbar_init(&sm.rl_free[i], 1);
        for (int q = 0; q < 4; ++q) {
            mbar_init(&sm.fin_full[i][q], C::NPAR - 1);
            mbar_init(&sm.fin_free[i][q], 1);
        }
    }
    for (int i = 0; i < C::NUNIT; ++i) sm.unit_loaded[i] = sm.unit_taken[i] = sm.copied[i] = 0;
    for (int i = 0; i < W_PLANS; ++i) mbar_init(&sm.plan_full[i], 1);
    sm.pv_units = sm.pv_pages = sm.ahead_units = 0;
    if (rank == 1) {  // expected before anything is sent
        for (int i = 0; i < C::NPBUF; ++i) mbar_arrive_expect_tx(&sm.p_full[i], C::PCOPY);
        for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&sm.l_full[i], 4 * C::ROWS);
    }
}

// The planner (a warp of the PV CTA) works the cluster's units out ahead of both CTAs' roles and leaves each in
// the shared memory of both.  At most three units ahead of the PV CTA's MMAs: the softmax warps are then no more
// than two further units behind (their sums of exp meet in two slots), so W_PLANS = 8 slots never run over; the
// prefetching warp, which nobody else waits for, is counted.
template <bool MQ> __device__ __forceinline__ void w_plan(WSmem<MQ>& sm, const WinParams& p)
{
    const int lane = (int)lane_id();
    bool ok = true;
    int n = 0;
    WScan scan;
    for (int u = (int)blockIdx.x >> 1; ok; u += (int)gridDim.x >> 1) {
        WUnit g;
        g.npg = -1;
        if (u < p.n_units) w_unit<MQ>(g, p, u, lane == 0, scan);
        if (g.npg == 0) continue;
        if (n >= 4 && lane == 0) ok = w_count<MQ>(&sm.pv_units, n - 3) && (MQ || w_count<MQ>(&sm.ahead_units, n - 6));
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        if (n > 0 && g.npg > 0 && lane < g.rows)  // its queries, into L2 (the first unit's are loaded at once)
            bulk_prefetch_l2(p.q_abs + ((size_t)(MQ ? g.row0 + lane : g.b) * H + 32 * g.hb) * ROW, (MQ ? 32 : H) * ROW * 2);
        const int slot = n % W_PLANS;
        if (lane < 2) {  // one lane a CTA
            const uint32_t at = mapa(smem_u32(&sm.plan[slot]), (uint32_t)lane);
            const uint4* w = reinterpret_cast<const uint4*>(&g);
#pragma unroll
            for (int i = 0; i < (int)(sizeof(WUnit) / 16); ++i) st_cluster_v4(at + 16 * i, w[i]);
            mbar_arrive_remote(mapa(smem_u32(&sm.plan_full[slot]), (uint32_t)lane));
        }
        if (g.npg < 0) return;
        ++n;
    }
}

// The n-th unit; npg is -1 behind the last one, and after an abort.
template <bool MQ> __device__ __forceinline__ WUnit w_next(WSmem<MQ>& sm, const WinParams& p, int n)
{
    WUnit g;
    if (__all_sync(0xFFFFFFFFu, w_wait<MQ, true>(&sm.plan_full[n % W_PLANS], (uint32_t)(n / W_PLANS) & 1u)))
        g = sm.plan[n % W_PLANS];
    else
        g.npg = -1;
    return g;
}

// ---- score CTA ----------------------------------------------------------------------------

// Producer t of NPROD: a unit's Q, then its pages in thirds, every NPROD-th use of the ring.  The uses are
// numbered on from unit to unit; use g lies in ring unit g % NUNIT.
template <bool MQ>
__device__ __forceinline__ void w_produce(WSmem<MQ>& sm, const CUtensorMap& tm_page, const CUtensorMap& tm_q,
                                          const WinParams& p, int t)
{
    using C = WCfg<MQ>;
    bool ok = true;  // (the elected lane's)
    int base = 0;
    auto take = [&](int use, uint32_t bytes) -> int {  // the use's ring unit, ready to be loaded
        const int u = use % C::NUNIT, k = use / C::NUNIT;
        if (C::NPROD > 1) ok = ok && w_count<MQ>(&sm.unit_loaded[u], k);
        ok = ok && w_wait<MQ>(&sm.empty[u], (uint32_t)(k & 1) ^ 1u);
        if (ok) {
            if (C::NPROD > 1) *reinterpret_cast<volatile int32_t*>(&sm.unit_loaded[u]) = k + 1;
            mbar_arrive_expect_tx(&sm.full[u], bytes);
        }
        return u;
    };
    for (int un = 0;; ++un) {
        const WUnit g = w_next<MQ>(sm, p, un);
        if (g.npg < 0) break;
        if (elect_one()) {
            for (int j = 0; j < C::NQ && ok; ++j) {
                if ((base + j) % C::NPROD != t) continue;
                const int u = take(base + j, C::QPU * C::QPIECE);
                if (!ok) break;
                if constexpr (MQ) {
                    // piece: heads 32 hb .. of two consecutive token rows (those past the group land in lanes nobody reads)
                    for (int x = 0; x < C::QPU; ++x) {
                        const int pc = C::QPU * j + x;
                        tma_load_4d(sm.u.c0.ring[u] + x * C::QPIECE, &tm_q, 0, 32 * g.hb, g.row0 + 2 * (pc & 1), pc >> 1,
                                    &sm.full[u]);
                    }
                } else {
                    tma_load_3d(sm.u.c0.ring[u], &tm_q, 0, g.b * H, C::QPU * j, &sm.full[u]);
                }
            }
        }
        __syncwarp();
        base += C::NQ;
        WLookup rows;
        for (int i = 0; i < g.npg; ++i) {
            const int32_t y = rows(p, g, i);
            if (elect_one()) {
#pragma unroll 1
                for (int x = 0; x < 3 && ok; ++x) {
                    if ((base + 3 * i + x) % C::NPROD != t) continue;
                    const int u = take(base + 3 * i + x, THIRD);
                    if (ok) tma_load_3d(sm.u.c0.ring[u], &tm_page, 0, y, 3 * x, &sm.full[u]);
                }
            }
            __syncwarp();
        }
        base += 3 * g.npg;
    }
    if (!ok) drain_inflight();
}

// Issuer r: the score MMAs of the pages a = r (mod 3), counted on from unit to unit, into S buffer r.  (One
// thread alone issues these MMAs at 50 clocks each, the tensor core retires one every 32.)
template <bool MQ> __device__ __forceinline__ void w_score(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase, int r)
{
    using C = WCfg<MQ>;
    bool ok = true;
    int base = 0, gp = 0;  // ring uses and pages before this unit
    for (int un = 0;; ++un) {
        const WUnit g = w_next<MQ>(sm, p, un);
        if (g.npg < 0) break;
        base += C::NQ;
        if (elect_one() && ok) {
            ok = w_wait<MQ>(&sm.q_ready, (uint32_t)un & 1u);
            tc_fence_after();
#pragma unroll 1
            for (int i = (r + C::NISS - gp % C::NISS) % C::NISS; i < g.npg && ok; i += C::NISS) {
                const int sb = (gp + i) % WN_S, k = (gp + i) / WN_S;
                ok = w_wait<MQ>(&sm.s_empty[sb], (uint32_t)(k & 1) ^ 1u);
#pragma unroll 1
                for (int t = 0; t < 3 && ok; ++t) {
                    const int e = base + 3 * i + t, u = e % C::NUNIT, ku = e / C::NUNIT;
                    ok = w_count<MQ>(&sm.unit_taken[u], ku) &&
                         w_wait<MQ>(&sm.full[u], (uint32_t)(ku & 1));
                    if (!ok) break;
                    *reinterpret_cast<volatile int32_t*>(&sm.unit_taken[u]) = ku + 1;
                    tc_fence_after();
                    issue_score_third(tbase, S_COL + 64u * (uint32_t)sb, smem_u32(sm.u.c0.ring[u]), t);
                    umma_commit(&sm.empty[u]);
                }
                if (ok) umma_commit(&sm.s_full[sb]);
            }
            if (ok) umma_commit(&sm.q_free);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        base += 3 * g.npg;
        gp += g.npg;
    }
    if (!ok) drain_inflight();
}

// The softmax warps copy Q from the ring into TMEM (lane 32 w + l <- row RPQ w + l), once the score MMAs of the unit
// before have read the old Q: each warp its quarter's rows, of every NPAR-th ring use, when it is through with its pages
// of the unit before.
template <bool MQ>
__device__ __forceinline__ bool w_copy_q(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase, int qd, int par, int base,
                                         int un)
{
    using C = WCfg<MQ>;
    const int lane = (int)lane_id();
    const int row = MQ ? 32 * (qd & 1) + lane : C::RPQ * qd + lane;  // of a piece
    const uint32_t taddr = tbase + ((32u * (uint32_t)qd) << 16) + Q_COL;
    if (!__all_sync(0xFFFFFFFFu, un == 0 || w_wait<MQ>(&sm.q_free, (uint32_t)(un - 1) & 1u))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int j = par; j < C::NQ; j += C::NPAR) {
        const int u = (base + j) % C::NUNIT, k = (base + j) / C::NUNIT;
        if (!__all_sync(0xFFFFFFFFu, w_count<MQ>(&sm.unit_taken[u], k) &&
                                         w_wait<MQ>(&sm.full[u], (uint32_t)(k & 1))))
            return false;
#pragma unroll 1
        for (int x = 0; x < C::QPU; ++x) {
            const int pc = C::QPU * j + x, c = MQ ? pc >> 1 : pc;
            if (pc >= C::NPIECE || (MQ && (pc & 1) != qd >> 1)) continue;
            uint32_t v[32];
            const uint8_t* src = sm.u.c0.ring[u] + x * C::QPIECE + row * 128;
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (lane < C::RPQ) w = *reinterpret_cast<const uint4*>(src + ((y ^ (row & 7)) << 4));
                v[4 * y] = w.x, v[4 * y + 1] = w.y, v[4 * y + 2] = w.z, v[4 * y + 3] = w.w;
            }
            tmem_st32(taddr + 32u * (uint32_t)c, v);
        }
        __syncwarp();
        if (lane == 0 && atomicAdd(&sm.copied[u], 1) == 3) {  // the last of the four quarters: the ring unit is read
            sm.copied[u] = 0;
            *reinterpret_cast<volatile int32_t*>(&sm.unit_taken[u]) = k + 1;
            mbar_arrive(&sm.empty[u]);
        }
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_ready);
    return true;
}

// Softmax warp (quarter qd, turn par): thread l = row RPQ qd + l of every NPAR-th page.  The reference max is a
// chain through a unit's pages: the warp of each page hands its decision on to the warp of the next one; a
// warp's sum of exp follows the reference when it comes to its own next page.  All in log2 units.  The chain of
// turns runs on through all units, so a turn's barrier is never a phase ahead of who waits on it.
// (The page's code is written to be short: the SM's instruction fetch is what these kernels run short of first.
// The scores' issue loop unrolled three times, 9 KB more, took the 16 x 64-token chunk from 328 to 358 us.)
template <bool MQ>
__device__ __forceinline__ void w_softmax(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase, uint32_t warp)
{
    using C = WCfg<MQ>;
    const int qd = (int)(warp & 3u), par = (int)(warp >> 2), l = (int)lane_id();
    const int h = C::RPQ * qd + l;
    const bool has_row = l < C::RPQ;
    const uint32_t t_lane = tbase + ((32u * (uint32_t)qd) << 16) + S_COL;
    const uint32_t recv0 = mapa(smem_u32(sm.u.c1.recv[0]), 1);
    const uint32_t pfull0 = mapa(smem_u32(&sm.p_full[0]), 1);
    const float TAU2 = TAU * 1.4426950408889634f;
    uint8_t* stage = sm.u.c0.pstage[warp];
    auto wait = [&](uint64_t* bar, int phase) { return __all_sync(0xFFFFFFFFu, w_wait<MQ>(bar, (uint32_t)phase & 1u)); };
    int base = 0, gp = 0, singles = 0;
#pragma unroll 1
    for (int un = 0;; ++un) {
        const WUnit g = w_next<MQ>(sm, p, un);
        if (g.npg < 0) break;
        if (!w_copy_q<MQ>(sm, p, tbase, qd, par, base, un)) return;
        base += C::NQ + 3 * g.npg;
        const int n = MQ ? (qd < g.rows ? w_clamp(g.n0 + qd, p.cap) : 0) : g.n0;  // this quarter's context
        float m_ref = -INFINITY, lsum = 0.f;
        const int rel = (par + C::NPAR - gp % C::NPAR) % C::NPAR;  // this warp's first page of the unit
#pragma unroll 1
        for (int i = rel; i < g.npg; i += C::NPAR) {
            const int a = gp + i, r = a % WN_S;
            if (!wait(&sm.s_full[r], a / WN_S)) return;
            tc_fence_after();
            const uint32_t t_s = t_lane + 64u * (uint32_t)r;
            const int t0 = PAGE * w_logical(g, i);
            // Unseen tokens' scores become -inf, in TMEM (a loop: short code, few pages).  Where all of them are finite, so
            // are the tokens' latents (a NaN or an infinity times anything, 0 too, stays one in the sum), and p = 0 times
            // those is 0: the PV CTA takes the page as it is.
            uint32_t flags = 0;
            if (!w_whole(p, n, n, t0)) {
                const uint64_t seen = w_between(p, n - p.window, n, t0);
                uint32_t most = 0;
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    uint32_t y[16];
                    tmem_ld16(t_s + 16u * (uint32_t)e, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (!((uint32_t)(seen >> (16 * e)) >> q & 1u)) {
                            most = max(most, y[q] & 0x7FFFFFFFu);
                            y[q] = 0xFF800000u;
                        }
                    tmem_st16(t_s + 16u * (uint32_t)e, y);
                }
                tmem_wait_st();
                if (__any_sync(0xFFFFFFFFu, has_row && most >= 0x7F800000u)) flags = F_NOT_FINITE;
            }
            uint32_t x[2][32];
            tmem_ld32(t_s, x[0]);
            tmem_ld32(t_s + 32u, x[1]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (l == 0) mbar_arrive(&sm.s_empty[r]);
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 32; ++q)
                m4[q & 3] = fmaxf(m4[q & 3], fmaxf(__uint_as_float(x[0][q]), __uint_as_float(x[1][q])));
            const float pmax = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.kscale;
            const float m_own = m_ref;
            float m_prev = pmax;  // the decision of the page before; a unit's first page sets the reference
            if (i > 0) {
                if (!wait(&sm.hand[qd][(a - 1) % C::NPAR], (a - 1) / C::NPAR)) return;
                m_prev = sm.xm[(a - 1) & 1][qd][l];
            }
            const bool resc = pmax > m_prev + TAU2;
            const float alpha = resc ? ex2_approx(m_prev - pmax) : 1.f;
            m_ref = resc ? pmax : m_prev;
            sm.xm[a & 1][qd][l] = m_ref;
            __syncwarp();
            if (l == 0) mbar_arrive(&sm.hand[qd][par]);
            lsum *= m_own == m_ref ? 1.f : ex2_approx(m_own - m_ref);  // (nothing summed yet: 0)
            const float mb = m_ref == -INFINITY ? 0.f : m_ref;  // nothing seen yet: every p is 0
            uint64_t part[2] = {0ull, 0ull};
            const uint64_t k2 = f32x2(p.kscale, p.kscale), mb2 = f32x2(-mb, -mb);
            // the bulk copy of this warp's page before has read its staging rows
            if (l == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // tokens 8 j .. 8 j + 7: p~ = bf16(2^(s - m_ref)); l sums the f32 values
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t* at = &x[j >> 2][8 * (j & 3) + 2 * q];
                    float e0, e1;
                    f32x2_parts(fma_f32x2(f32x2(__uint_as_float(at[0]), __uint_as_float(at[1])), k2, mb2), e0, e1);
                    e0 = ex2_approx(e0);
                    e1 = ex2_approx(e1);
                    part[q & 1] = add_f32x2(part[q & 1], f32x2(e0, e1));
                    w[q] = pack_bf16x2(e0, e1);
                }
                if (has_row)
                    *reinterpret_cast<uint4*>(stage + pt_chunk_off(h, j) - qd * C::PSTAGE) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            float l0, l1;
            f32x2_parts(add_f32x2(part[0], part[1]), l0, l1);
            lsum += l0 + l1;
            fence_proxy_async_cta();  // the bulk copy reads the rows through the async proxy
            __syncwarp();
            const int st = a % C::NPBUF;
            // the PV CTA has finished with the buffer's page before
            if (!wait(&sm.p_empty[st], a / C::NPBUF + 1)) return;
            const uint32_t dst = recv0 + (uint32_t)(st * C::PBUF);
            const uint32_t bar = pfull0 + (uint32_t)(st * sizeof(uint64_t));
            if (__any_sync(0xFFFFFFFFu, resc && has_row)) flags |= F_RESCALE;
            if (l == 0) {
                bulk_copy_to_cluster(dst + (uint32_t)(qd * C::PSTAGE), stage, C::PSTAGE, bar);
                bulk_commit();
                st_async_b32(dst + C::META_FLAGS + 4 * qd, flags, bar);
            }
            if (has_row) st_async_b32(dst + C::META_ALPHA + 4 * h, __float_as_uint(alpha), bar);
        }
        const int last = gp + g.npg - 1;
        // (the turn after the last page's waits for its decision all the same)
        if ((last + 1) % C::NPAR == par && !wait(&sm.hand[qd][last % C::NPAR], last / C::NPAR)) return;
        // the quarter's sums meet in the warp of turn 1; the others go on at once
        if (!wait(&sm.fin_free[un & 1][qd], (un >> 1) + 1)) return;
        sm.fin_l[un & 1][rel][qd][l] = lsum;
        sm.fin_m[un & 1][rel][qd][l] = m_ref;
        __syncwarp();
        if (par != 1) {
            if (l == 0) mbar_arrive(&sm.fin_full[un & 1][qd]);
        } else {
            if (!wait(&sm.fin_full[un & 1][qd], un >> 1)) return;
            m_ref = sm.fin_m[un & 1][(g.npg - 1) % C::NPAR][qd][l];  // the last page's warp
            float ltot = 0.f;  // by the unit's own count of pages: the order does not depend on the units before
#pragma unroll
            for (int w = 0; w < C::NPAR; ++w) {
                const float m_w = sm.fin_m[un & 1][w][qd][l], l_w = sm.fin_l[un & 1][w][qd][l];
                ltot += m_w == m_ref ? l_w : l_w * ex2_approx(m_w - m_ref);
            }
            __syncwarp();
            if (l == 0) mbar_arrive(&sm.fin_free[un & 1][qd]);
            if (g.single) {  // the PV CTA lands o_lat itself (a row that sees nothing has l = 0; its o_lat is not used)
                const int sl = singles & 1;
                if (!__all_sync(0xFFFFFFFFu, w_wait<MQ, true>(&sm.rl_free[sl], (uint32_t)((singles >> 1) + 1) & 1u))) return;
                if (has_row)
                    st_async_b32(mapa(smem_u32(&sm.u.c1.rl[sl][h]), 1), __float_as_uint(1.f / ltot),
                                 mapa(smem_u32(&sm.l_full[sl]), 1));
            } else if (!MQ && has_row) {
                p.ws_ml[((size_t)g.b * p.nsplit + g.s) * H + h] = make_float2(m_ref, ltot);
            }
        }
        singles += g.single;
        gp += g.npg;
    }
    // this warp's bulk copies have landed, and so have the PV CTA's last releases of its P buffers
    if (l == 0) {
        bulk_wait<0>();
        for (int a = max(0, gp - C::NPBUF); a < gp && !aborted(sm); ++a)
            w_wait<MQ>(&sm.p_empty[a % C::NPBUF], (uint32_t)((a / C::NPBUF) & 1));
    }
}

// ---- PV CTA -------------------------------------------------------------------------------

// Producer: the units' pages again, their latents only, as half pages.
template <bool MQ>
__device__ __forceinline__ void w_produce_halves(WSmem<MQ>& sm, const CUtensorMap& tm_page8, const WinParams& p)
{
    const uint64_t pol = policy_evict_first();  // the last reader of the latent in this unit
    bool ok = true;                             // (the elected lane's)
    int e = 0;
    for (int un = 0;; ++un) {
        const WUnit g = w_next<MQ>(sm, p, un);
        if (g.npg < 0) break;
        WLookup rows;
        for (int i = 0; i < g.npg; ++i, e += 2) {
            const int32_t y = rows(p, g, i);
            if (elect_one()) {
#pragma unroll 1
                for (int x = 0; x < 2 && ok; ++x) {
                    const int q = (e + x) % WN_HALF;
                    ok = w_wait<MQ>(&sm.empty[q], (uint32_t)(((e + x) / WN_HALF) & 1) ^ 1u);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sm.full[q], SLOT1);
                    // (diagnostic: a load never issued.  Asked here the question costs nothing that shows; in the score CTA,
                    // whose one producer sets a chunk's pace, it took 16 x 64 rows from 231.5 to 233.3 us.)
                    if (x > 0 || i + 1 != p.withhold)
                        tma_load_3d_hint(sm.u.c1.ring[q], &tm_page8, 0, y + HALF * x, 0, &sm.full[q], pol);
                }
            }
            __syncwarp();
        }
    }
    if (!ok) drain_inflight();
}

template <bool MQ>
__device__ __forceinline__ void w_issue_pv(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase)
{
    using C = WCfg<MQ>;
    // (elect_one() names the same lane every time: pending and the two counters are that lane's)
    bool ok = true, pending = false;  // pending: the epilogue has not yet taken the unit before out of TMEM
    uint32_t epi_k = 0;
    int gp = 0;
    for (int un = 0;; ++un) {
        const WUnit g = w_next<MQ>(sm, p, un);
        if (g.npg < 0) break;
        const int n_lo = w_clamp(g.n0, p.cap);
        if (elect_one() && ok) {
#pragma unroll 1
            for (int i = 0; i < g.npg && ok; ++i) {
                const int a = gp + i, st = a % C::NPBUF;
                const int q0 = (2 * a) % WN_HALF, q1 = (2 * a + 1) % WN_HALF;
                if (!w_wait<MQ>(&sm.full[q0], (uint32_t)(2 * a / WN_HALF) & 1u) ||
                    !w_wait<MQ>(&sm.full[q1], (uint32_t)((2 * a + 1) / WN_HALF) & 1u)) {
                    ok = false;
                    break;
                }
                if (!w_wait<MQ, true>(&sm.p_full[st], (uint32_t)((a / C::NPBUF) & 1))) {
                    ok = false;
                    break;
                }
                *reinterpret_cast<volatile int32_t*>(&sm.pv_pages) = a + 1;
                fence_proxy_async_cta();  // the P tile came through DSMEM copies; the MMA reads it
                const volatile uint32_t* rf = reinterpret_cast<const volatile uint32_t*>(sm.u.c1.recv[st] + C::META_FLAGS);
                const uint32_t flags = rf[0] | rf[1] | rf[2] | rf[3];
                uint32_t cmd = (flags & F_NOT_FINITE) ? E_CLEAR : 0u;
                if (i > 0 && (flags & F_RESCALE)) cmd |= E_RESCALE;
                if (pending || cmd) {
                    if (pending) ok = w_wait<MQ>(&sm.epi_done, epi_k++ & 1u);
                    pending = false;
                    if (ok && cmd) {
                        if (cmd & E_RESCALE) umma_commit(&sm.o_done);
                        sm.epi_cmd = cmd;
                        sm.epi_page = a;
                        // the rows' contexts are consecutive, n_lo .. n_hi: the tokens that not all of them see
                        sm.epi_t0 = PAGE * w_logical(g, i);
                        sm.epi_hidden = ~w_between(p, g.n_hi - p.window, n_lo, sm.epi_t0);
                        sm.epi_rows = g.rows;
                        sm.epi_n0 = g.n0;
                        mbar_arrive(&sm.epi_req);
                        ok = w_wait<MQ>(&sm.epi_done, epi_k++ & 1u);
                    }
                    if (!ok) break;
                }
                tc_fence_after();
                // each half-page slot goes back to its producer once the MMAs that read it are done
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    const int q = x ? q1 : q0;
                    issue_pv_half(tbase, smem_u32(sm.u.c1.ring[q]), smem_u32(sm.u.c1.recv[st]), x, i > 0);
                    umma_commit(&sm.empty[q]);
                }
                mbar_arrive_expect_tx(&sm.p_full[st], C::PCOPY);
                umma_commit_mc(&sm.p_empty[st], (uint16_t)0x1);
            }
            if (ok) {  // O of the unit is complete: to be written out
                umma_commit(&sm.o_done);
                sm.epi_cmd = E_WRITE;
                sm.epi_b = g.b;
                sm.epi_s = g.s;
                sm.epi_hb = g.hb;
                sm.epi_row0 = g.row0;
                sm.epi_rows = g.rows;
                sm.epi_n0 = g.n0;
                sm.epi_single = g.single;
                mbar_arrive(&sm.epi_req);
                pending = true;
                *reinterpret_cast<volatile int32_t*>(&sm.pv_units) = un + 1;
            }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        gp += g.npg;
    }
    if (!ok) {
        drain_inflight();
        *reinterpret_cast<volatile int32_t*>(&sm.abort_flag) = 1;
    } else if (elect_one()) {  // the epilogue warps leave
        if (pending) ok = w_wait<MQ>(&sm.epi_done, epi_k++ & 1u);
        sm.epi_cmd = 0u;
        mbar_arrive(&sm.epi_req);
    }
}

// The rows that see nothing, which no unit has: their o_lat counts as zero whatever the workspace holds.
template <bool MQ> __device__ __forceinline__ void w_empty_rows(const WinParams& p)
{
    const int lane = (int)lane_id(), stride = 32 * ((int)gridDim.x >> 1);
    for (int r0 = 32 * ((int)blockIdx.x >> 1); r0 < p.R; r0 += stride) {
        const int r = r0 + lane;
        bool sees = true;
        if (r < p.R) {
            if constexpr (MQ) {
                const int lo = last_slot_from(p.row_start, p.B, r);
                const int first = p.row_start[lo];
                sees = r >= first && r < p.row_start[lo + 1] && (int64_t)p.pos0[lo] + (r - first) >= 0;
            } else {
                sees = min(p.ctx_len[r], p.cap) > 0;
            }
        }
        if (!sees)
            for (int h = 0; h < H; ++h) p.oscale[(size_t)h * p.R + r] = 0.f;
    }
}

// The power of two that brings a row with largest magnitude m into f16's range (to [2^14, 2^15)), and its
// inverse; 1 for rows of zeros, infinities or NaN.
__device__ __forceinline__ float w_row_scale(float m, float& inverse)
{
    const int e = (int)(__float_as_uint(m) >> 23) & 255;  // m >= 0; (f32 subnormals count as zero)
    const bool plain = e > 0 && e < 255;
    const int up = plain ? min(max(141 - e, -126), 126) : 0;  // 2^up m in [2^14, 2^15), or as near as f32 allows
    inverse = __uint_as_float((uint32_t)(127 - up) << 23);
    return __uint_as_float((uint32_t)(127 + up) << 23);
}

// O [rows x 512] f32 leaves TMEM, half the dims a warp, as f16 with a power of two per row: o_lat = O / l when the
// unit is all its rows see, else the split's O (f32 there would take twice the stores).  Four lanes share a row: of 64
// columns lane c holds 8 n + 2 c and 8 n + 2 c + 1 for n = 0 .. 7, and stores them side by side, 32 bytes, so that a
// store instruction writes whole lines (with a row a lane, a sector each of 32 lines: 1 x 1000 rows 129 us, so 123).
// The dims of o_lat and of the splits' O thus lie in that order; the expansion puts W_UV into the same.
// Reading TMEM sets the pace (some 64 bytes a clock and SM: 2.1 us for a chunk's 256 KB), so it is read once: the
// power of two comes from the row's first 32 entries, with room for 2^8 times their largest, and the row's
// largest entry is found on the way.  A row that it shows to have left the range, or to lie far below it, has its
// warps go over their rows again with the power of two that fits.
template <bool MQ>
__device__ __forceinline__ void w_write_out(WSmem<MQ>& sm, const WinParams& p, uint32_t t_row, int quarter, int half,
                                            int singles)
{
    using C = WCfg<MQ>;
    const int b = sm.epi_b, s = sm.epi_s, hb = sm.epi_hb, row0 = sm.epi_row0, rows = sm.epi_rows;
    const bool single = MQ || sm.epi_single != 0;
    const int lane = (int)lane_id(), col = lane & 3, row = 32 * quarter + (lane >> 2);  // and row + 8, + 16, + 24
    const uint32_t t_lane = t_row + 256u * (uint32_t)half;
    // a chunk's quarter holds 32 heads of token row row0 + quarter; decode's the heads 32 quarter .. of slot b
    const bool mine = MQ ? quarter < rows && sm.epi_n0 + quarter > 0 : quarter < C::ROWS / 32;  // (and sees something)
    const int tok = MQ ? row0 + quarter : b, head = (MQ ? 32 * hb : 32 * quarter) + (lane >> 2);
    // o_lat [96][R][512], or partial O [B][nsplit][96][512]; a scale each
    const size_t at = single ? (size_t)head * p.R + tok : ((size_t)b * p.nsplit + s) * H + head;
    const size_t at8 = single ? 8 * (size_t)p.R : 8;  // eight heads on
    uint16_t* out = (single ? p.olat : p.ws_o) + at * LORA + 256 * half + 16 * col;
    float r[4], inverse[4], up[4], m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = mine && single ? sm.u.c1.rl[singles & 1][row + 8 * i] : 1.f;
        inverse[i] = up[i] = 1.f;
    }
    auto over_lanes = [](float x) {
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
        return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
    };
    if (mine) {  // the rows' first entries: their largest to [2^6, 2^7)
        uint32_t v[2][16];
        tmem_ld_rows_x4(t_row, v[0]);
        tmem_ld_rows_x4(t_row + (16u << 16), v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n)
                m[i] = fmaxf(m[i], fmaxf(fabsf(__uint_as_float(v[i >> 1][4 * n + 2 * (i & 1)])),
                                         fabsf(__uint_as_float(v[i >> 1][4 * n + 2 * (i & 1) + 1]))));
            up[i] = w_row_scale(over_lanes(m[i]) * r[i] * 256.f, inverse[i]);
        }
    }
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {  // the second only for rows whose first power of two did not fit
        if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = 0.f;
            auto leave = [&](const uint32_t (&v)[32], int k, int hi) {  // 64 columns of rows + 16 hi and + 16 hi + 8
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = 2 * hi + x;
                    const float f = r[i] * up[i];
                    uint32_t w[8];
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float a = __uint_as_float(v[4 * n + 2 * x]), c = __uint_as_float(v[4 * n + 2 * x + 1]);
                        m[i] = fmaxf(m[i], fmaxf(fabsf(a), fabsf(c)));
                        w[n] = pack_f16x2(a * f, c * f);
                    }
                    st_global_v8(out + (size_t)i * at8 * LORA + 64 * k, w);
                }
            };
            uint32_t v[32], next[32];  // one is on its way while the other is turned
            tmem_ld_rows_x8(t_lane, v);
            tmem_wait_ld();
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                tmem_ld_rows_x8(t_lane + (16u << 16) + 64u * (uint32_t)k, next);
                leave(v, k, 0);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(next[e]));  // (not read before the wait)
                tmem_ld_rows_x8(t_lane + 64u * (uint32_t)min(k + 1, 3), v);
                leave(next, k, 1);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(v[e]));
            }
        }
        if (pass) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = over_lanes(m[i]);
        if (mine && col == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sm.u.c1.half_max[half][row + 8 * i] = m[i];
        }
        named_bar(WB_OUT, 32 * W_EPI);
        if (single && threadIdx.x == 0) {  // the slot of 1 / l is free again
            mbar_arrive_expect_tx(&sm.l_full[singles & 1], 4 * C::ROWS);
            mbar_arrive_remote(mapa(smem_u32(&sm.rl_free[singles & 1]), 0));
        }
        __syncwarp();
        bool fit = true;
        if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float most = fmaxf(sm.u.c1.half_max[0][row + 8 * i], sm.u.c1.half_max[1][row + 8 * i]) * r[i];
                if (most == 0.f || (most * up[i] >= 1.f && most * up[i] < 65504.f)) continue;
                fit = false;
                up[i] = w_row_scale(most, inverse[i]);
            }
        }
        if (__all_sync(0xFFFFFFFFu, fit)) break;
    }
    if (mine && half == 0 && col == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) (single ? p.oscale : p.ws_oscale)[at + i * at8] = inverse[i];
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.epi_done);
}

// Once the P of page a has arrived, page a + W_AHEAD (of whichever unit) is prefetched into L2 for the score CTA, whose
// ring holds too few pages to cover HBM's latency under load; a warp that has fallen behind skips pages.  64 slots over
// 4,100 seen tokens 73.4 -> 69.6 us, over 1,088 33.8 -> 33.6 us (W_AHEAD 5: 73.3 and 33.9, 6: 71.4 and 33.6, 8: 69.3 and
// 34.4, 10: 70.8 and 35.8).  A chunk's pages are in L2 for most of its units:
// 235.5 and 123.6 us with it and without.
constexpr int W_AHEAD = 7;
template <bool MQ> __device__ __forceinline__ void w_prefetch(WSmem<MQ>& sm, const CUtensorMap& tm_page, const WinParams& p)
{
    int gp = 0;
    for (int un = 0;; ++un) {
        const WUnit g = w_next<MQ>(sm, p, un);
        if (g.npg < 0) break;
        WLookup rows;
        for (int i = 0; i < g.npg; ++i) {
            const int32_t y = rows(p, g, i);
            const int done = gp + i - W_AHEAD + 1;  // pages whose P has to be there
            if (done <= 0) continue;  // (a cluster's first pages are loaded at once)
            if (!__all_sync(0xFFFFFFFFu, w_count<MQ>(&sm.pv_pages, done))) return;
            if (elect_one() && y < p.n_pages * p.n_layers * PAGE &&
                *reinterpret_cast<volatile int32_t*>(&sm.pv_pages) <= done + 2)
                for (int x = 0; x < 3; ++x) tma_prefetch_3d(&tm_page, 0, y, 3 * x);
            __syncwarp();
        }
        *reinterpret_cast<volatile int32_t*>(&sm.ahead_units) = un + 1;
        gp += g.npg;
    }
}

// The NaNs and infinities among the latents of page a's tokens that not all rows of the unit see become zero: the rows
// that do not see them have p = 0 there, which only a finite latent turns into 0.  The rows of a chunk's unit that do see
// such a token get NaN, as they would from the latent itself whatever their p (0 too), by way of that p.  (Rare: the
// scores have shown that there are some.  Looking every masked page through took the chunk of 1 x 1000 rows from 137 to
// 152 us.)
template <bool MQ>
__device__ __forceinline__ void w_clear(WSmem<MQ>& sm, const WinParams& p, int a, uint64_t hidden, int w)
{
    using C = WCfg<MQ>;
    const int lane = (int)lane_id();
#pragma unroll 1
    for (int t = w; t < PAGE; t += W_EPI) {  // a warp a token: 64 pieces of 16 bytes, two a lane
        if (!(hidden >> t & 1ull)) continue;
        const int q = (2 * a + (t >= HALF ? 1 : 0)) % WN_HALF;
        uint8_t* at = sm.u.c1.ring[q] + (t & (HALF - 1)) * 128 + (lane & 7) * 16;
        bool found = false;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
            uint4* piece = reinterpret_cast<uint4*>(at + ((lane >> 3) + 4 * x) * HCHUNK);
            const uint4 v = *piece;
            auto finite = [](uint32_t b) {  // bf16 with all exponent bits set: NaN or infinity
                if ((b & 0x7F80u) == 0x7F80u) b &= 0xFFFF0000u;
                if ((b & 0x7F800000u) == 0x7F800000u) b &= 0x0000FFFFu;
                return b;
            };
            const uint4 f = make_uint4(finite(v.x), finite(v.y), finite(v.z), finite(v.w));
            found = found || f.x != v.x || f.y != v.y || f.z != v.z || f.w != v.w;
            *piece = f;
        }
        if (MQ && __any_sync(0xFFFFFFFFu, found)) {
#pragma unroll 1
            for (int qd = 0; qd < sm.epi_rows; ++qd) {
                const int n = w_clamp(sm.epi_n0 + qd, p.cap);
                if (w_between(p, n - p.window, n, sm.epi_t0) >> t & 1ull)
                    *reinterpret_cast<uint16_t*>(sm.u.c1.recv[a % C::NPBUF] + pt_chunk_off(C::RPQ * qd + lane, t >> 3) +
                                                 2 * (t & 7)) = 0x7FFFu;
            }
        }
    }
    fence_proxy_async_cta();  // the MMAs read the latents and P through the async proxy
}

// Epilogue warp: the TMEM lanes of its quarter, the dims of its half.
template <bool MQ>
__device__ __forceinline__ void w_epilogue(WSmem<MQ>& sm, const WinParams& p, uint32_t tbase, int quarter, int half)
{
    using C = WCfg<MQ>;
    const int lane = (int)lane_id(), row = 32 * quarter + lane;
    const uint32_t t_row = tbase + ((32u * (uint32_t)quarter) << 16), t_lane = t_row + 256u * (uint32_t)half;
    uint32_t od = 0;
    int singles = 0;
    for (uint32_t k = 0;; ++k) {
        // (an abort may reach one warp and not another: they agree on it, so that all or none pass the
        // write-out's barriers)
        bool got = __all_sync(0xFFFFFFFFu, w_wait<MQ>(&sm.epi_req, k & 1u));
        if (named_bar_any(WB_OUT, 32 * W_EPI, !got)) break;
        const uint32_t cmd = *reinterpret_cast<volatile uint32_t*>(&sm.epi_cmd);
        if (!cmd) break;
        const int page = sm.epi_page;
        if (cmd & (E_WRITE | E_RESCALE)) got = w_wait<MQ>(&sm.o_done, od++ & 1u);
        if ((cmd & E_WRITE) && sm.epi_single)
            got = got && w_wait<MQ, true>(&sm.l_full[singles & 1], (uint32_t)(singles >> 1) & 1u);
        got = __all_sync(0xFFFFFFFFu, got);
        if (named_bar_any(WB_OUT, 32 * W_EPI, !got)) break;
        tc_fence_after();
        if (cmd & E_WRITE) {
            const bool single = sm.epi_single != 0;
            w_write_out<MQ>(sm, p, t_row, quarter, half, singles);
            singles += single;
            continue;
        }
        if (cmd & E_CLEAR) w_clear<MQ>(sm, p, page, sm.epi_hidden, quarter + 4 * half);
        const float* al = reinterpret_cast<const float*>(sm.u.c1.recv[page % C::NPBUF] + C::META_ALPHA);
        const float f = (cmd & E_RESCALE) && row < C::ROWS ? al[row] : 1.f;
        if (__any_sync(0xFFFFFFFFu, f != 1.f)) {  // some row of this warp moved its reference
#pragma unroll 1
            for (int cb = 0; cb < LORA / 64; ++cb) {
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
}

// ---- the kernel ---------------------------------------------------------------------------

template <bool MQ>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(128)
    k3mla_window_kernel(const __grid_constant__ CUtensorMap tm_page, const __grid_constant__ CUtensorMap tm_page8,
                        const __grid_constant__ CUtensorMap tm_q, const WinParams p)
{
    using C = WCfg<MQ>;
    WSmem<MQ>& sm = w_smem<MQ>();
    const uint32_t rank = cluster_ctarank(), warp = threadIdx.x >> 5, lane = lane_id();
    if (threadIdx.x == 0) {
        w_init(sm, rank, p);
        fence_mbarrier_init_cluster();
    }
    if (warp == 4) {
        tmem_alloc(&sm.tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 5 && lane == 0) {
        tma_prefetch_desc(rank == 0 ? &tm_page : &tm_page8);
        if (rank == 0) tma_prefetch_desc(&tm_q);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    griddep_wait();
    griddep_launch_dependents();
    if (rank == 0) {
        if (warp < C::W_PROD) w_softmax<MQ>(sm, p, tbase, warp);
        else if (warp < C::W_MMA0) w_produce<MQ>(sm, tm_page, tm_q, p, (int)warp - C::W_PROD);
        else if (warp < C::W_MMA0 + C::NISS) w_score<MQ>(sm, p, tbase, (int)warp - C::W_MMA0);
    } else {
        if (warp < 4 || (warp >= WW_EPI1 && warp < WW_EPI1 + 4))
            w_epilogue<MQ>(sm, p, tbase, (int)(warp & 3u), warp >= 4 ? 1 : 0);
        else if (warp == WW_HALVES) w_produce_halves<MQ>(sm, tm_page8, p);
        else if (warp == WW_PV) w_issue_pv<MQ>(sm, p, tbase);
        else if (warp == WW_PLAN) w_plan<MQ>(sm, p);
        else if (warp == WW_EMPTY) w_empty_rows<MQ>(p);
        else if (!MQ && warp == WW_AHEAD) w_prefetch<MQ>(sm, tm_page, p);
    }
    // After an abort a role leaves wherever it stands, with copies and MMAs of its own or of others still under way: they
    // land before the CTA gives its shared memory and its TMEM back.
    if (aborted(sm)) drain_inflight();
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tbase, TMEM_COLS);
}

// ---- merge of splits (decode) ---------------------------------------------------------------

// o_lat of a row (slot, head) = sum_i w_i O_i / sum_i w_i l_i with w_i = 2^(m_i - max).  Split i belongs to group i mod 4;
// the groups' sums, each over ascending i, are added as (g0 + g1) + (g2 + g3), so that the bits depend on the slot's
// own splits only, whichever kernel adds them up: k3mla_window_merge_kernel, or the expansion when the rows are few.
constexpr int WM_GROUPS = 4;

// How many splits slot b has.  (A length is no output of the kernels of this call, and was there before the first began.)
__device__ __forceinline__ int w_splits(const WinParams& p, int b)
{
    int nsp, wp0;
    const int n = w_clamp(p.ctx_len[b], p.cap);
    const int all = w_pages(n, n, p.window, p.n_sink, nsp, wp0);
    const int per = slot_split(all * PAGE, p.split_tokens) / PAGE;
    return (all + per - 1) / per;
}

// The largest reference max of a row's ns splits (a whole warp).
__device__ __forceinline__ float w_max_ref(const WinParams& p, size_t row, int ns)
{
    float m = -INFINITY;
    for (int i = (int)lane_id(); i < ns; i += 32) m = fmaxf(m, p.ws_ml[row + (size_t)i * H].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    return m;
}

// Groups g0 .. g0 + PER - 1 of a row's sums: l, and D dims from d on (D / 2 registers of f16 pairs a split).
template <int PER, int D>
__device__ __forceinline__ void w_sum_groups(const WinParams& p, size_t row, int ns, int g0, float m, int d, float (&l)[PER],
                                             float (&part)[PER][D])
{
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        l[k] = 0.f;
#pragma unroll
        for (int e = 0; e < D; ++e) part[k][e] = 0.f;
    }
#pragma unroll(PER == 1 ? 8 : 2)
    for (int i0 = g0; i0 < ns; i0 += WM_GROUPS)
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (i0 + k >= ns) continue;
            const size_t at = row + (size_t)(i0 + k) * H;
            const float2 rec = p.ws_ml[at];
            uint32_t v[D / 2];
#pragma unroll
            for (int e = 0; e < D / 4; ++e) {
                const uint2 x = reinterpret_cast<const uint2*>(p.ws_o + at * LORA + d)[e];
                v[2 * e] = x.x, v[2 * e + 1] = x.y;
            }
            const float w = ex2_approx(rec.x - m), f = w * p.ws_oscale[at];
            l[k] = fmaf(w, rec.y, l[k]);
#pragma unroll
            for (int e = 0; e < D / 2; ++e) {
                float x0, x1;
                f16x2_parts(v[e], x0, x1);
                part[k][2 * e] = fmaf(f, x0, part[k][2 * e]);
                part[k][2 * e + 1] = fmaf(f, x1, part[k][2 * e + 1]);
            }
        }
}

// A row per CTA of 128 threads, four dims each.
__global__ void __launch_bounds__(128) k3mla_window_merge_kernel(const WinParams p)
{
    __shared__ float smax[4];
    const int h = blockIdx.x, b = blockIdx.y, d = 4 * (int)threadIdx.x;
    griddep_launch_dependents();
    const int ns = w_splits(p, b);
    griddep_wait();        // (every CTA: the expansion counts on this kernel's end for the splits' end too)
    if (ns <= 1) return;  // landed by the split itself
    const size_t row = (size_t)b * p.nsplit * H + h;
    const float m = w_max_ref(p, row, ns);
    float l[WM_GROUPS], part[WM_GROUPS][4], acc[4];
    w_sum_groups<WM_GROUPS, 4>(p, row, ns, 0, m, d, l, part);
    const float r = 1.f / ((l[0] + l[1]) + (l[2] + l[3]));
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        acc[e] = ((part[0][e] + part[1][e]) + (part[2][e] + part[3][e])) * r;
        big = fmaxf(big, fabsf(acc[e]));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, x));
    if (lane_id() == 0) smax[threadIdx.x >> 5] = big;
    __syncthreads();
    float inverse;
    const float up = w_row_scale(fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3])), inverse);
    *reinterpret_cast<uint2*>(p.olat + ((size_t)h * p.B + b) * LORA + d) =
        make_uint2(pack_f16x2(acc[0] * up, acc[1] * up), pack_f16x2(acc[2] * up, acc[3] * up));
    if (d == 0) p.oscale[(size_t)h * p.B + b] = inverse;
}

// ---- W_UV expansion ---------------------------------------------------------------------------

// OUT_h^T [128 v x 64 rows] = W_UV[h] [128 x 512] . o_lat^T [512 x 64], a CTA per head taking tiles of 64 rows in
// turn with W_UV[h] resident: read once (before the grid wait: a weight) and turned into f16 where it lies, each
// of its rows times a power of two.  o_lat streams through a ring of 64-dim chunks; two accumulators, so that
// a tile's outputs leave while the next one's MMAs run.  The powers of two come off on the way out, W_UV's by TMEM
// lane, o_lat's by column.
constexpr int WX_TILE = 64;
constexpr int WX_RING = 10;
constexpr int WX_CHUNK = WX_TILE * 128;
constexpr int WX_A = 8 * VH * 128;                    // W_UV[h]
constexpr int WX_SMEM = WX_A + WX_RING * WX_CHUNK + 1024;
constexpr int WX_EPI = 16;                            // warps 0..15 convert W_UV, then take the outputs
constexpr int WX_THREADS = 32 * (WX_EPI + 2);         // ... one loads, one issues
static_assert(WX_RING >= LORA / 64, "a whole tile's operand fits (wx_merge)");
static_assert(WX_SMEM <= 225 * 1024, "shared memory, beside a few hundred static bytes");

struct WxSmem {
    float merge_l[WX_EPI];    // a warp's sum of w_i l_i
    uint64_t w_full, w_ready, b_full[WX_RING], b_empty[WX_RING], d_full[2], d_empty[2];
    uint32_t tmem_base;
    int32_t abort_flag;
    uint64_t wait_ns;
    float wscale[VH];         // what undoes W_UV's powers of two
    float rscale[WX_EPI];     // wx_merge: ... and o_lat's; 0: the row sees nothing, its output is 0
};

struct WxParams {
    const float* oscale;
    uint16_t* out;
    int32_t* dev_err;
    int R;  // the rows of o_lat and out
};

// W_UV[h] in shared memory ([8 chunks][128 rows][128 B], 128-byte swizzle), bf16 -> f16 in place, every row times
// the power of two that brings its largest entry to [2^14, 2^15), and every chunk's 64 dims in the order of the write-out:
// 8 n + 2 j + e goes to 16 j + 2 n + e.  Four threads a row, j = 0 .. 3, the row held in registers between its maximum
// and the conversion.
__device__ __forceinline__ void wx_convert(uint8_t* sa, float* wscale)
{
    const int row = (int)threadIdx.x >> 2, j = threadIdx.x & 3;
    uint32_t v[8][8];
    uint32_t m = 0;  // the largest magnitude: bf16 bit patterns of magnitudes order like the magnitudes
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            v[c][n] = *reinterpret_cast<const uint32_t*>(sa + c * (VH * 128) + row * 128 + ((n ^ (row & 7)) << 4) + 4 * j);
            m = __vmaxu2(m, v[c][n] & 0x7FFF7FFFu);
        }
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    float inverse;
    const float up = w_row_scale(__uint_as_float(m << 16), inverse);
    auto half2 = [&](uint32_t w) { return pack_f16x2(bf16lo_to_f32(w) * up, bf16hi_to_f32(w) * up); };
    __syncwarp();  // the row has been read by all four
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x)
            *reinterpret_cast<uint4*>(sa + c * (VH * 128) + row * 128 + (((2 * j + x) ^ (row & 7)) << 4)) =
                make_uint4(half2(v[c][4 * x]), half2(v[c][4 * x + 1]), half2(v[c][4 * x + 2]), half2(v[c][4 * x + 3]));
    if (j == 0) wscale[row] = inverse;
}

// The rows' splits added up by the expansion itself, straight into the operand tile of head h (one tile: at most 16
// rows): WARPS warps a row, a group each (4) or all four (1).  Saves a kernel and o_lat's way through memory.
template <int WARPS>
__device__ __forceinline__ void wx_merge(uint8_t* sb, WxSmem& sm, const WinParams& p, int h, int ns)
{
    constexpr int PER = WM_GROUPS / WARPS;
    const int lane = (int)lane_id(), warp = (int)threadIdx.x >> 5, b = warp / WARPS, g = warp % WARPS;
    auto place = [&](int half) {  // dims 256 half + 8 lane .. + 7 of row b
        return reinterpret_cast<uint4*>(sb + (4 * half + (lane >> 3)) * WX_CHUNK + b * 128 + (((lane & 7) ^ (b & 7)) << 4));
    };
    float acc[2][8], ltot = 0.f;
    const bool several = b < p.B && ns > 1;
    if (several) {
        const size_t row = (size_t)b * p.nsplit * H + h;
        const float m = w_max_ref(p, row, ns);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float l[PER], part[PER][8];
            w_sum_groups<PER, 8>(p, row, ns, g, m, 256 * half + 8 * lane, l, part);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[half][e] = PER == 1 ? part[0][e]
                                        : (part[0][e] + part[1 % PER][e]) + (part[2 % PER][e] + part[3 % PER][e]);
            ltot = PER == 1 ? l[0] : (l[0] + l[1 % PER]) + (l[2 % PER] + l[3 % PER]);
        }
    } else if (b < p.B && g == 0) {  // landed by the split itself, or nothing seen
        const size_t at = (size_t)h * p.B + b;
#pragma unroll
        for (int half = 0; half < 2; ++half)
            *place(half) = *reinterpret_cast<const uint4*>(p.olat + at * LORA + 256 * half + 8 * lane);
        if (lane == 0) sm.rscale[b] = p.oscale[at];
    }
    if constexpr (WARPS > 1) {  // the groups meet in the row's first warp, by way of the tile's unused rows 8 .. 63
        auto meet = [&](int w, int k) {
            return reinterpret_cast<float4*>(sb + (w >> 1) * WX_CHUNK + 1024 + (w & 1) * 2048) + 32 * k + lane;
        };
        if (several && g > 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float* a = &acc[k >> 1][4 * (k & 1)];
                *meet(warp, k) = make_float4(a[0], a[1], a[2], a[3]);
            }
            if (lane == 0) sm.merge_l[warp] = ltot;
        }
        named_bar(1, 32 * WX_EPI);
        if (several && g == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float* a = &acc[k >> 1][4 * (k & 1)];
                const float4 s1 = *meet(warp + 1, k), s2 = *meet(warp + 2, k), s3 = *meet(warp + 3, k);
                a[0] = (a[0] + s1.x) + (s2.x + s3.x);
                a[1] = (a[1] + s1.y) + (s2.y + s3.y);
                a[2] = (a[2] + s1.z) + (s2.z + s3.z);
                a[3] = (a[3] + s1.w) + (s2.w + s3.w);
            }
            ltot = (ltot + sm.merge_l[warp + 1]) + (sm.merge_l[warp + 2] + sm.merge_l[warp + 3]);
        }
    }
    if (several && g == 0) {
        const float r = 1.f / ltot;
        float big = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[half][e] *= r;
                big = fmaxf(big, fabsf(acc[half][e]));
            }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, x));
        float inverse;
        const float up = w_row_scale(big, inverse);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float* a = acc[half];
            *place(half) = make_uint4(pack_f16x2(a[0] * up, a[1] * up), pack_f16x2(a[2] * up, a[3] * up),
                                      pack_f16x2(a[4] * up, a[5] * up), pack_f16x2(a[6] * up, a[7] * up));
        }
        if (lane == 0) sm.rscale[b] = inverse;
    }
    fence_proxy_async_cta();  // the MMAs read the tile through the async proxy
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.b_full[0]);
}

// MERGE: o_lat's rows come from memory (0), or from their splits, 1 or 4 warps a row.
template <int MERGE>
__global__ void __launch_bounds__(WX_THREADS, 1)
    k3mla_window_expand_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_o,
                               const WxParams p, const WinParams win)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ WxSmem sm;
    uint8_t* sa = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sb = sa + WX_A;
    const int h = blockIdx.x, warp = threadIdx.x >> 5, lane = (int)lane_id();
    const int tiles = (p.R + WX_TILE - 1) / WX_TILE;
    if (threadIdx.x == 32 * WX_EPI) {
        sm.abort_flag = 0;
        sm.wait_ns = WAIT_NS;
        mbar_init(&sm.w_full, 1);
        mbar_init(&sm.w_ready, WX_EPI);
        for (int i = 0; i < WX_RING; ++i) {
            mbar_init(&sm.b_full[i], MERGE ? WX_EPI : 1);
            mbar_init(&sm.b_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_empty[i], WX_EPI);
        }
        fence_mbarrier_init_cluster();
        mbar_arrive_expect_tx(&sm.w_full, WX_A);
        for (int c = 0; c < 8; ++c)
            tma_load_3d_hint(sa + c * (VH * 128), &tm_w, 0, h * WROWS_PER_HEAD + NOPE, c, &sm.w_full, policy_evict_first());
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, 2 * WX_TILE);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    bool ok = true;
    if (warp == WX_EPI) {
        if (!MERGE && elect_one()) {
            griddep_wait();
            int g = 0;
            for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y)
                for (int c = 0; c < 8 && ok; ++c, ++g) {
                    const int s = g % WX_RING;
                    ok = wait_bar(&sm.b_empty[s], (uint32_t)((g / WX_RING) & 1) ^ 1u, sm, p.dev_err);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sm.b_full[s], WX_CHUNK);
                    // (rows past the batch are the next head's, or zeros: not stored)
                    tma_load_3d(sb + s * WX_CHUNK, &tm_o, 0, h * p.R + t * WX_TILE, c, &sm.b_full[s]);
                }
            if (!ok) drain_inflight();
        }
    } else if (warp == WX_EPI + 1) {
        if (elect_one()) {
            const uint32_t idesc = make_idesc_f16(128, WX_TILE);
            griddep_wait();  // (the bounded waits below start when o_lat is there)
            ok = wait_bar(&sm.w_ready, 0, sm, p.dev_err);
            int g = 0, it = 0;
            for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y, ++it) {
                ok = wait_bar(&sm.d_empty[it & 1], (uint32_t)((it >> 1) & 1) ^ 1u, sm, p.dev_err);
                for (int c = 0; c < 8 && ok; ++c, ++g) {
                    const int s = g % WX_RING;
                    if (!MERGE || c == 0) ok = wait_bar(&sm.b_full[s], (uint32_t)((g / WX_RING) & 1), sm, p.dev_err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = make_sdesc(smem_u32(sa + c * (VH * 128)), 16, 1024);
                    const uint64_t bd = make_sdesc(smem_u32(sb + s * WX_CHUNK), 16, 1024);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma_ss(tbase + (uint32_t)(WX_TILE * (it & 1)), ad + 2u * ks, bd + 2u * ks, idesc, (c | ks) != 0);
                    umma_commit(&sm.b_empty[s]);
                }
                if (ok) umma_commit(&sm.d_full[it & 1]);
            }
            if (!ok) drain_inflight();
        }
    } else {
        ok = __all_sync(0xFFFFFFFFu, wait_bar(&sm.w_full, 0, sm, p.dev_err));
        if (ok) wx_convert(sa, sm.wscale);
        fence_proxy_async_cta();  // the MMAs read it through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.w_ready);
        int ns = 0;
        if (MERGE && warp / max(MERGE, 1) < win.B) ns = w_splits(win, warp / max(MERGE, 1));
        griddep_wait();
        griddep_launch_dependents();
        if constexpr (MERGE != 0) wx_merge<MERGE>(sb, sm, win, h, ns);
        const int q = warp & 3, cg = warp >> 2, v = 32 * q + lane;
        named_bar(1, 32 * WX_EPI);  // wscale is complete
        const float ws = sm.wscale[v];
        auto scale_of = [&](int t) {  // undoes o_lat's power of two: lane j has row 16 cg + j of tile t
            const int row = 16 * cg + (lane & 15), r = t * WX_TILE + row;
            if (MERGE) return row < WX_EPI ? sm.rscale[row] : 0.f;
            return r < p.R ? p.oscale[(size_t)h * p.R + r] : 0.f;
        };
        int it = 0;
        float next = scale_of(blockIdx.y);
        for (int t = blockIdx.y; t < tiles; t += gridDim.y, ++it) {
            const float rs = next;
            next = scale_of(t + gridDim.y);  // (a tile ahead: its latency stays off the path)
            if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bar(&sm.d_full[it & 1], (uint32_t)(it >> 1) & 1u, sm, p.dev_err));
            if (!ok) break;
            tc_fence_after();
            uint32_t acc[16];
            tmem_ld16(tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)(WX_TILE * (it & 1) + 16 * cg), acc);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.d_empty[it & 1]);
            uint16_t* out = p.out + ((size_t)(t * WX_TILE + 16 * cg) * H + h) * VH + v;
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // 64 bytes of a row a warp
                const float s = __shfl_sync(0xFFFFFFFFu, rs, j);
                const float x = s == 0.f ? 0.f : __uint_as_float(acc[j]) * ws * s;
                if (t * WX_TILE + 16 * cg + j < p.R) out[(size_t)j * H * VH] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xFFFFu);
            }
        }
    }
    if (aborted(sm)) drain_inflight();  // (as in the attention kernel)
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tbase, 2 * WX_TILE);
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
    size_t olat, scale, o, oscale, ml, total;
};
static WinWs w_layout(long long rows, int nsplit)
{
    WinWs w;
    w.olat = 0;
    w.scale = w_up((size_t)rows * H * LORA * 2);
    w.o = w.scale + w_up((size_t)rows * H * 4);
    const size_t records = nsplit > 1 ? (size_t)rows * nsplit * H : 0;
    w.oscale = w.o + w_up(records * LORA * 2);
    w.ml = w.oscale + w_up(records * 4);
    w.total = w.ml + w_up(records * 8);
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
    const double k = (double)f * 1.4426950408889634;
    *kscale = (float)k;
    return k <= 3.4028234663852886e38;  // (an infinite factor would make NaN of every score of 0)
}

template <bool MQ>
static int w_launch(const uint16_t* q_abs, const uint16_t* slab, const uint16_t* w_kv_b, uint16_t* out, uint8_t* ws,
                    const WinWs& wl, WinParams& p, cudaStream_t st)
{
    using C = WCfg<MQ>;
    p.olat = reinterpret_cast<uint16_t*>(ws + wl.olat);
    p.oscale = reinterpret_cast<float*>(ws + wl.scale);
    p.ws_o = p.nsplit > 1 ? reinterpret_cast<uint16_t*>(ws + wl.o) : nullptr;
    p.ws_oscale = p.nsplit > 1 ? reinterpret_cast<float*>(ws + wl.oscale) : nullptr;
    p.ws_ml = p.nsplit > 1 ? reinterpret_cast<float2*>(ws + wl.ml) : nullptr;
    CUtensorMap tm_page, tm_page8, tm_q, tm_w, tm_o;
    const uint64_t slab_rows = (uint64_t)p.n_pages * p.n_layers * PAGE, R = (uint64_t)p.R;
    int rc = make_tmap_slab_3d(&tm_page, slab, slab_rows, ROW, 9, PAGE, 3);
    if (!rc) rc = make_tmap_slab_3d(&tm_page8, slab, slab_rows, ROW, 9, HALF, 8);
    if (rc) return rc;
    if (MQ) {
        // q_abs as (64 elements, 96 heads, R rows, 9 chunks): 64 columns of 32 heads of two token rows
        const uint64_t dims[4] = {64, H, R, 9}, strides[3] = {ROW * 2, (uint64_t)H * ROW * 2, 128};
        const uint32_t box[4] = {64, 32, 2, 1};
        rc = make_tmap_store(&tm_q, false, 4, q_abs, dims, strides, box, true);
    } else {
        rc = make_tmap_slab_3d(&tm_q, q_abs, R * H, ROW, 9, H, C::QPU);
    }
    if (!rc) rc = make_tmap_slab_3d(&tm_w, w_kv_b, (uint64_t)H * WROWS_PER_HEAD, LORA, 8, VH, 1);
    if (!rc) rc = make_tmap_slab_3d(&tm_o, p.olat, (uint64_t)H * R, LORA, 8, WX_TILE, 1);
    if (rc) return rc;
    static bool attr_done[64] = {}, attr_expand[3][64] = {};
    const size_t smem = sizeof(WSmem<MQ>) + 1024;
    set_smem_attr(reinterpret_cast<const void*>(k3mla_window_kernel<MQ>), smem, attr_done);
    const int clusters = std::min(p.n_units, sm_count() / 2);
    rc = launch_pdl(k3mla_window_kernel<MQ>, dim3(2 * clusters), dim3(W_THREADS), smem, st, "k3mla_window_kernel", tm_page,
                    tm_page8, tm_q, p);
    if (rc) return rc;
    // Few rows: the expansion adds the splits up itself, four warps a row (a slot of 3 splits 20.5 -> 16.9 us, of 33 27.5 ->
    // 21.2 us, four slots of 17 26.2 -> 25.5 us) or one (16 slots of 3 26.5 -> 25.0 us, 16 of 4 38.2 -> 36.1 us; but ten of
    // 6 26.8 -> 27.3 us, five of 11 25.8 -> 30.0 us: a warp then goes through its list in several rounds).
    const int merge = MQ || p.nsplit == 1 ? 0 : (p.B <= WX_EPI / 4 ? 4 : (p.B <= WX_EPI && p.nsplit <= WM_GROUPS ? 1 : 0));
    if (p.nsplit > 1 && !merge) {
        rc = launch_pdl(k3mla_window_merge_kernel, dim3(H, p.B), dim3(128), 0, st, "k3mla_window_merge_kernel", p);
        if (rc) return rc;
    }
    WxParams x;
    x.oscale = p.oscale, x.out = out, x.dev_err = p.dev_err, x.R = p.R;
    const int tiles = (p.R + WX_TILE - 1) / WX_TILE;
    const auto expand = MQ || merge == 0 ? k3mla_window_expand_kernel<0>
                                         : (merge == 4 ? k3mla_window_expand_kernel<4> : k3mla_window_expand_kernel<1>);
    set_smem_attr(reinterpret_cast<const void*>(expand), WX_SMEM, attr_expand[merge == 4 ? 2 : merge]);
    // Three CTAs a head fill two rounds of the SMs where one leaves a third of them idle, but load and convert W_UV three
    // times: 4,000 rows (63 tiles) 458 -> 446 us, 2,000 235 -> 231, 1,000 122.7 -> 122.2, but 600 75.0 -> 78.3, 250 37.8 -> 41.6.
    return launch_pdl(expand, dim3(H, tiles >= 16 ? 3 : 1), dim3(WX_THREADS), WX_SMEM, st, "k3mla_window_expand_kernel", tm_w,
                      tm_o, x, p);
}

// A unit's pages take up to 0.85 us each, and its write-out waits for all of them within WAIT_NS: half of that is allowed.
constexpr long long W_UNIT_PAGES = 1 << 19;

static bool w_unit_fits(const char* who, long long pages)
{
    if (pages <= W_UNIT_PAGES) return true;
    set_error("%s: %lld pages in one unit of work, more than %lld", who, pages, W_UNIT_PAGES);
    return false;
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
    p.q_abs = q_abs, p.table = table;
    p.n_pages = n_pages, p.n_layers = n_layers, p.layer = layer, p.max_pages = max_pages;
    p.cap = (int)std::min<long long>(std::min(max_ctx, 0x7FFFFF00), (long long)max_pages * PAGE);
    p.window = window, p.n_sink = n_sink, p.nsplit = 1;
    p.wait_ns = WAIT_NS;
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
    // As many splits a slot as give every pair of SMs one, none shorter than a tile.  Two to four slots leave the
    // expansion's CTAs, one a head, an SM each, where they ready W_UV meanwhile, unless that makes the splits longer by
    // more than six pages, which is what the 3 us of W_UV and the fewer partials are worth.  Full plan against that one,
    // longer by 2 pages: two slots over 3,000 tokens 23.9 -> 20.7 us, four over 1,000 21.3 -> 20.0; by 4: two over 7,000
    // 26.1 -> 24.4, three over 4,096 24.8 -> 23.4; by 6: four over 4,096 25.4 -> 24.4, two over 10,000 27.7 -> 27.0 (but over
    // 8,192 24.4 -> 25.2); by 8: three over 7,000 26.6 -> 27.4, four over 6,000 26.5 -> 27.7; by 24: three over 32,768 41.7 -> 58.6.
    // One slot over 4,096 21.5 -> 21.1, but over 16,384 (6 more) 25.7 -> 27.0; five over 2,000 (4 more) 24.9 -> 26.4: their
    // splits meet in a kernel of its own.
    const long long tiles = (w_max_pages(max_ctx, window, n_sink) * PAGE + TILE - 1) / TILE;
    const int sms = sm_count();
    auto per = [&](int n) {  // tiles of a split when n SMs share the lists
        const long long want = std::max(1, n / 2 / B);
        return (tiles + want - 1) / want;
    };
    long long split = per(sms);
    if (B > 1 && B <= 4 && sms > H && (per(sms - H) - split) * (TILE / PAGE) <= 6) split = per(sms - H);
    return (int)std::min<long long>(split * TILE, 0x7FFFFFFF / TILE * TILE);
}

static int window_decode(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                         const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                         const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace, size_t ws_bytes, int B,
                         int max_ctx, int window, int n_sink, int split_tokens, int32_t* dev_err, void* stream,
                         uint64_t wait_ns, int withhold)
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
    const long long longest = w_max_pages(p.cap, window, n_sink), split = (split_tokens ? split_tokens : SPLIT_MAX) / PAGE;
    if (!w_unit_fits("k3mla_window_decode", std::min(longest, split))) return K3MLA_E_INVALID;
    if (B > 65535 || (long long)B * ns * H > 0x7FFFFFFFll) {  // the merge's grid; partial-row coordinates
        set_error("k3mla_window_decode: too many slots or splits");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    p.ctx_len = ctx_len;
    p.dev_err = dev_err;
    p.wait_ns = wait_ns;
    p.withhold = withhold;
    p.B = p.R = B;
    p.split_tokens = split_tokens;
    p.nsplit = ns;
    p.n_units = B * ns;
    return w_launch<false>(q_abs, slab, w_kv_b, out, reinterpret_cast<uint8_t*>(workspace), w_layout(B, ns), p,
                           reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int k3mla_window_decode(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                                   const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                                   const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                   size_t ws_bytes, int B, int max_ctx, int window, int n_sink, int split_tokens,
                                   int32_t* dev_err, void* stream)
{
    return window_decode(q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, ctx_len, w_kv_b, scale_bf16, out,
                         workspace, ws_bytes, B, max_ctx, window, n_sink, split_tokens, dev_err, stream, WAIT_NS, 0);
}

static bool w_diag_check(const char* who, int withhold_page, uint32_t wait_us)
{
    if (withhold_page >= 1 && withhold_page < 1 << 30 && wait_us >= 100 && wait_us <= 100000) return true;
    set_error("%s: 1 <= withhold_page < 2^30 and 100 <= wait_us <= 100000", who);
    return false;
}

extern "C" int k3mla_diag_window_timeout(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                                         const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                                         const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                         size_t ws_bytes, int B, int max_ctx, int window, int n_sink, int split_tokens,
                                         int withhold_page, uint32_t wait_us, int32_t* dev_err, void* stream)
{
    if (!w_diag_check("k3mla_diag_window_timeout", withhold_page, wait_us)) return K3MLA_E_INVALID;
    return window_decode(q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, ctx_len, w_kv_b, scale_bf16, out,
                         workspace, ws_bytes, B, max_ctx, window, n_sink, split_tokens, dev_err, stream,
                         (uint64_t)wait_us * 1000ull, withhold_page + 1);
}

extern "C" size_t k3mla_window_chunk_decode_workspace_bytes(int B, int R, int max_ctx)
{
    if (B <= 0 || R <= 0 || max_ctx <= 0) return 0;
    return w_layout(R, 1).total;
}

static int window_chunk_decode(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                               const int32_t* block_table, int max_pages_per_slot, const int32_t* pos0,
                               const int32_t* row_start, int B, int R, const uint16_t* w_kv_b, uint16_t scale_bf16,
                               uint16_t* out, void* workspace, size_t ws_bytes, int max_ctx, int window, int n_sink,
                               int32_t* dev_err, void* stream, uint64_t wait_ns, int withhold)
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
    // (four rows' windows reach three tokens further than one's)
    if (!w_unit_fits("k3mla_window_chunk_decode", w_max_pages(p.cap, std::min(window, 0x7FFFFF00) + 3, n_sink)))
        return K3MLA_E_INVALID;
    // (the planner's one pass over 2^20 slots takes some 30 ms, far inside the bounded waits for its first unit)
    if (units > 0x3FFFFFFFll || (long long)R * H > 0x7FFFFFFFll || B > 1 << 20) {
        set_error("k3mla_window_chunk_decode: too many rows or slots");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    p.pos0 = pos0;
    p.row_start = row_start;
    p.dev_err = dev_err;
    p.wait_ns = wait_ns;
    p.withhold = withhold;
    p.B = B;
    p.R = R;
    p.n_units = (int)units;
    return w_launch<true>(q_abs, slab, w_kv_b, out, reinterpret_cast<uint8_t*>(workspace), w_layout(R, 1), p,
                          reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int k3mla_window_chunk_decode(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers, int layer,
                                         const int32_t* block_table, int max_pages_per_slot, const int32_t* pos0,
                                         const int32_t* row_start, int B, int R, const uint16_t* w_kv_b,
                                         uint16_t scale_bf16, uint16_t* out, void* workspace, size_t ws_bytes, int max_ctx,
                                         int window, int n_sink, int32_t* dev_err, void* stream)
{
    return window_chunk_decode(q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, pos0, row_start, B, R, w_kv_b,
                               scale_bf16, out, workspace, ws_bytes, max_ctx, window, n_sink, dev_err, stream, WAIT_NS, 0);
}

extern "C" int k3mla_diag_window_chunk_timeout(const uint16_t* q_abs, const uint16_t* slab, int n_pages, int n_layers,
                                               int layer, const int32_t* block_table, int max_pages_per_slot,
                                               const int32_t* pos0, const int32_t* row_start, int B, int R,
                                               const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                               size_t ws_bytes, int max_ctx, int window, int n_sink, int withhold_page,
                                               uint32_t wait_us, int32_t* dev_err, void* stream)
{
    if (!w_diag_check("k3mla_diag_window_chunk_timeout", withhold_page, wait_us)) return K3MLA_E_INVALID;
    return window_chunk_decode(q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, pos0, row_start, B, R, w_kv_b,
                               scale_bf16, out, workspace, ws_bytes, max_ctx, window, n_sink, dev_err, stream,
                               (uint64_t)wait_us * 1000ull, withhold_page + 1);
}
