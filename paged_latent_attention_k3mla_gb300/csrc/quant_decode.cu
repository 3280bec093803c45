// quant_decode.cu -- absorbed-MLA decode over the 8-bit latent cache (quant.cuh), over the whole context or a window and the
// first tokens, for sm_103a.
//
// Math: as window.cu's decode, with row_t the values that the cache stands for: code 2^n_t and rope 2^n_t.  With raw_t the
// product of q_abs with the row in the row's own units,
//     s_t = scale 2^n_t raw_t,   p = softmax(s),   o_lat = sum_t (p_t 2^n_t) code_t,   out = W_UV o_lat.
// Slots are cut into splits as in window.cu, and what a split leaves behind -- o_lat, or O and its reference and sum -- is what
// window.cu's merge and expansion take.
//
// The codes are never converted: both contractions are 8-bit MMAs with the codes as they lie in shared memory as the
// operand of M, and what multiplies them is written as a sum of two e4m3 numbers, the second in units of 1 / 32, in columns of
// their own:
//     S^T[128 tokens x 96] = codes . (q1 | q2)^T  (+ the rope part in bf16, onto q1's columns),   raw = S1 + S2 / 32
//     O^T[512 dims x 96]  += codes^T . (P1 | P2) 2^e,                                             O = O1 + O2 / 32
// The second is a block-scaled MMA (kind::mxf8f6f4): e is an exponent of every head and 32 tokens, K of one MMA, that brings
// the largest P there to [2^7, 2^8).  Without it the numbers' 2^22 between their largest and their smallest step have to hold
// all that a row weighs, and where a few tokens take most of its mass the thousands that it answers with are lost
// together (the first of 4,096 tokens takes 0.87: the output off by 0.087 of itself, of 16,384 by 0.36; with it by 0.0017).  It
// costs 37 shuffles a tile and warp, and saves the moves of a reference that holds all in range: 64 slots of 4,096 tokens 65.3 ->
// 66.7 us, with four times as large scores 73.5 -> 66.8.
// A pair has 8 bits, as a bf16 does, and two such MMAs cost what one in bf16 does (e4m3 runs at twice the rate), without the
// 65,536 conversions a tile that a bf16 form would begin with.  96 columns are 48 heads: two CTAs a split, each with all of its
// tokens.  Tokens on M and not heads, because 48 heads would leave half of M's 128 rows empty, and because O then fits: TMEM
// holds O in 4 x 96 columns and S in 96, and the exponents in 8, 488 of 512.
//
// Numerics.  Scores, maxima and sums are f32.  Below that: q as a pair (times a power of two for the CTA's 48 heads; exact for
// entries down to 2^-14 of their largest, within 1.25 * 2^-22 of it below), p times its row's power of two as a pair (by way of
// an f16: 2^-8 of it, as a bf16 is; within 1.25 * 2^-22 of the largest of its block below that), then as in window.cu o_lat and a
// split's O as f16 with a power of two a row, and the output as bf16.  As the exponents carry P's size, a reference only keeps
// the f32 sums in range: a head's is the largest score at first and moves when one passes it by 2^60, as does the unit that O is
// held in, the largest row's power of two.  Two, because rows may be as far apart as bf16's range: p alone goes into the sum of
// exp, p times the row's size into O.  (Held to one reference, of their product, rows of 2^-20 before rows of 2^110 lost their
// weight.)  What is lost is p below 2^-126 of the reference, and rows 2^126 times smaller than another of their block.  Against
// 64 bits the outputs are off by 0.0017 to 0.0019 (relative, mean square), of which 0.0017 are their own rounding.
//
// Structure of a CTA: eight softmax warps (a quarter of the tile's tokens x 24 heads each: a lane has a token, so a row's scale,
// mask and sums of exp are the thread's own; a block's largest P is found by 13 shuffles of a warp, and what meets every tile is
// one vote of four warps whether a reference has to move), and one warp each that loads, issues S and issues PV.  A tile is two
// pages; its five chunks of 128 tokens x 128 B (the rope part and four times 128 latents) go through a ring of nine.
//
// Measured: 64 slots of 4,096 tokens 66.7 us (190 MB: 2.8 TB/s, 0.42 of the copy rate; 834 TFLOP/s), 64 of 15,000 to
// 16,384 208 us (3.2 TB/s, 1,005 TFLOP/s, 0.53 of the measured bf16 rate), one of 32,768 29.2 us, 128 of up to 256 29.3 us;
// k3mla_window_decode over the bf16 cache takes 68.2 us for 64 of 4,100.  What bounds it: a tile's MMAs take 1,990 clocks -- 56 each
// for 128 x 96 x 32, as both operands come from shared memory at 128 B a clock -- and a tile some 3,100.  With S and the queries'
// pairs there is room for 1.8 tiles, so the second contraction (1,700 beside S of the next tile), the loads over what it
// frees (1,000), the last scores (600) and the softmax (1,700, and the search for the blocks' largest) of every second tile stand in
// one chain; the tensor pipe is 44% busy.  Small calls: 3.9 us until the queries' pairs are there, 2.2 for the write-out, and the
// expansion's 9.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "decode_core.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "window.cuh"

namespace k3 {

struct QdParams {
    const uint16_t* q_abs;
    const uint8_t* slab;
    const int32_t *table, *ctx_len;
    uint16_t* olat;
    float* oscale;
    uint16_t* ws_o;
    float* ws_oscale;
    float2* ws_ml;
    int32_t* dev_err;
    int B, max_pages, n_pages, n_layers, layer, cap;
    int window, n_sink, split_tokens, nsplit;
    float kscale;  // scale * log2(e) > 0
    uint64_t wait_ns;   // bounded-wait limit: WAIT_NS, shorter only from the diagnostic entry
    int32_t withhold;   // diagnostic only, 0 otherwise: of a unit's tile k - 1 the first latent chunk is never loaded
};

// A unit of work: split s of slot b, npg pages from entry `first` of the list of the pages that the slot sees (none: 0).
struct QdUnit {
    int n, npg, first, nsp, wp0;
    bool single;
};

__device__ __forceinline__ QdUnit qd_unit(const QdParams& p, int b, int s, bool report)
{
    QdUnit g;
    const int n = p.ctx_len[b];
    if (report && n > p.cap && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_CTX);
    g.n = w_clamp(n, p.cap);
    const int all = w_pages(g.n, g.n, p.window, p.n_sink, g.nsp, g.wp0);
    const int per = slot_split(all * PAGE, p.split_tokens) / PAGE;
    g.single = all <= per;
    g.first = s * per;
    g.npg = min(per, max(0, all - g.first));
    return g;
}

__device__ __forceinline__ int qd_logical(const QdUnit& g, int i)
{
    const int e = g.first + i;
    return e < g.nsp ? e : e - g.nsp + g.wp0;
}

// The page block of logical page lp of slot b, or -1 (zero rows).
__device__ __forceinline__ int32_t qd_block(const QdParams& p, int b, int lp, bool report)
{
    const int32_t id = p.table[(size_t)b * p.max_pages + lp];
    if (id >= 0 && id < p.n_pages) return id * p.n_layers + p.layer;
    if (report && id != -1 && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_BAD_PAGE);
    return -1;
}

__device__ __forceinline__ bool qd_seen(const QdParams& p, int n, int t) { return t < n && (t < p.n_sink || t >= n - p.window); }

// ---- shared memory, barriers ----------------------------------------------------------------

constexpr int QD_HEADS = 48;                    // heads of a CTA
constexpr int QD_MINE = 24;                     // ... of a softmax warp
constexpr int QD_TILE = 128;                    // tokens of a tile: two pages of the unit's list
constexpr int QD_PAIRS = 2 * QD_HEADS;          // columns: every head twice, a first and a second e4m3 number
constexpr int QD_CHUNK = QD_TILE * 128;         // a tile's chunk: [128 tokens][128 B]; a tile is the rope chunk, then 4 of latents
constexpr int QD_CHUNKS = 5;
constexpr int QD_RING = 9;                      // (what fits; a tenth chunk would wait for the same second contraction)
constexpr int QD_QCHUNK = QD_PAIRS * 128;       // 128 dims of the queries' pairs
constexpr int QD_SOFTMAX = 8;                   // warps 0 .. 7: quarter of the tile's tokens w & 3, group of the heads w >> 2
constexpr int QW_LOAD = 8, QW_SCORE = 9, QW_PV = 10;
constexpr int QD_THREADS = 352;
constexpr uint32_t QD_S_COL = 4 * QD_PAIRS;     // TMEM: O by blocks of 128 dims at 96 d, then S
constexpr uint32_t QD_ONE_COL = 5 * QD_PAIRS, QD_SF_COL = QD_ONE_COL + 4;  // ... scale factors: the latents', 1; P's
// A tile's pages, one each of the two CTAs, are fetched into L2 this many tiles before its scores.  64 slots x 4,096 tokens, when the
// loads' and the scores' loops were not written out yet, by a warp of its own: 1 74.3 us, 2 69.3, 3 69.7, 4 70.5, 6 71.6, without
// 73.9; by softmax warp 0, this many: 69.3.
constexpr int QD_AHEAD = 3;
constexpr uint32_t QB_GROUP = 1, QB_ALL = 3;    // named barriers: a group's four softmax warps (1, 2); all of them
constexpr float QD_TAU = 60.f;                  // a reference, or O's unit, moves when something passes it by more than 2^TAU
constexpr float QD_BIG = 1048576.f;             // scores this large are rounded by so much that s less the reference has to be taken
                                                // from the rounded s that it is one of, or none may come near it
constexpr float QD_NONE = 1e30f;                // makes any score that is not -inf pass a reference that is not there yet
constexpr float QD_LOW = 32.f;                  // the second number's units are 1 / 32: half a step of the first at 256 is 8
constexpr uint32_t QD_IDESC_S = make_idesc_e4m3(128, QD_PAIRS, 0, 0);
constexpr uint32_t QD_IDESC_ROPE = make_idesc_bf16(128, QD_HEADS, 0, 0);
constexpr uint32_t QD_IDESC_PV = make_idesc_mx_e4m3(128, QD_PAIRS, 1, 1, 0);
constexpr uint32_t QD_IDESC_NEXT = 1u << 4;     // the next 32 tokens' factors

struct __align__(1024) QdSmem {
    uint8_t q[4][QD_QCHUNK];          // K-major B of the scores: rows h (first numbers) and 48 + h (second)
    uint8_t q_rope[QD_HEADS * 128];
    uint8_t ring[QD_RING][QD_CHUNK];
    uint8_t p[QD_TILE * 128];         // MN-major B of the second contraction: [token][group: 24 first, 24 second numbers]
    // P's exponents as tmem_copy_scales takes them: column n's for quarter q at 16 (n % 32) + 4 (n / 32) + q
    alignas(128) uint8_t sf[512];
    uint64_t full[QD_RING], empty[QD_RING];
    uint64_t q_ready, s_full, s_empty, p_full, pv_done;
    alignas(16) float m_neg[QD_HEADS];  // the references in log2 units, negated; QD_NONE before there is one
    float m_ref[QD_HEADS];            // ... as they are
    float alpha[QD_HEADS], turn[QD_HEADS];  // what a moved reference turns the sums by, and O, whose unit may have moved too
    float part[4][QD_HEADS];          // a quarter's maxima or sums
    alignas(16) int32_t unit[2][4];   // a group's largest row exponents, by quarter
    int32_t od[2];                    // ... and the exponent of O's unit
    uint32_t most[QD_SOFTMAX][2];     // the prologue's maxima by warp: latents, rope
    uint32_t tmem_base;
    int32_t abort_flag;
    uint64_t wait_ns;
};
static_assert(QD_QCHUNK % 1024 == 0 && (QD_HEADS * 128) % 1024 == 0, "operand tiles start 1024-byte aligned");
static_assert(sizeof(QdSmem) + 1024 <= 227 * 1024, "shared memory of one CTA (with alignment slack)");
static_assert(QD_SF_COL + 4 <= 512, "TMEM columns");

__device__ __forceinline__ bool qd_wait(QdSmem& sm, const QdParams& p, uint64_t* bar, int phase)
{
    return wait_bar(bar, (uint32_t)phase & 1u, sm, p.dev_err);
}

__device__ __forceinline__ void qd_init(QdSmem& sm, const QdParams& p)
{
    sm.wait_ns = p.wait_ns;
    sm.abort_flag = 0;
#pragma unroll 1
    for (int i = 0; i < QD_RING; ++i) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_ready, QD_SOFTMAX);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_empty, QD_SOFTMAX);
    mbar_init(&sm.p_full, QD_SOFTMAX);
    mbar_init(&sm.pv_done, 1);
}

// A unit's page blocks, 32 looked up at a time, one a lane; -1: zero rows.
struct QdLookup {
    int32_t block;
    __device__ __forceinline__ int32_t operator()(const QdParams& p, const QdUnit& g, int b, int i, bool report)
    {
        const int lane = (int)lane_id();
        if ((i & 31) == 0) block = i + lane < g.npg ? qd_block(p, b, qd_logical(g, i + lane), report) : -1;
        return __shfl_sync(0xFFFFFFFFu, block, i & 31);
    }
};

// ---- roles --------------------------------------------------------------------------------

// The producer: every chunk of a tile from its two pages.  (This loop and the scores' are written out: what one thread does for
// a chunk stands in the chain of a tile.  64 x 4,096 tokens 67.2 -> 65.4 us, one slot of 32,768 26.6 -> 26.9.)
__device__ __forceinline__ void qd_produce(QdSmem& sm, const CUtensorMap& tm_page, const QdParams& p, const QdUnit& g, int b,
                                           int tiles)
{
    bool ok = true;  // (the elected lane's)
    QdLookup look;
    const int none = p.n_pages * p.n_layers;  // past the end: read as zeros
    for (int i = 0; i < tiles; ++i) {
        look(p, g, b, 2 * i, true);
        int32_t at[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) at[x] = __shfl_sync(0xFFFFFFFFu, look.block, (2 * i + x) & 31);
        if (elect_one()) {
            const int32_t at0 = at[0] < 0 ? none : at[0], at1 = at[1] < 0 ? none : at[1];
            int u = QD_CHUNKS * i % QD_RING, phase = QD_CHUNKS * i / QD_RING ^ 1;
#pragma unroll
            for (int c = 0; c < QD_CHUNKS && ok; ++c) {
                ok = qd_wait(sm, p, &sm.empty[u], phase);
                if (!ok) break;
                mbar_arrive_expect_tx(&sm.full[u], QD_CHUNK);
                // (diagnostic: a load never issued)
                if (c != 1 || i + 1 != p.withhold) {
                    const int z = c ? c - 1 : 4;
                    tma_load_4d(sm.ring[u], &tm_page, 0, 0, z, at0, &sm.full[u]);
                    tma_load_4d(sm.ring[u] + PAGE * 128, &tm_page, 0, 0, z, at1, &sm.full[u]);
                }
                if (++u == QD_RING) u = 0, phase ^= 1;
            }
        }
        __syncwarp();
    }
    if (!ok) drain_inflight();
}

// S[128 tokens x 96] = tile . queries: four chunks of 128 e4m3 latents, the rope chunk in bf16 onto the first numbers' columns.
// Issued as soon as a chunk is there, beside PV of the tile before.  (One issuer in a fixed order, PV(i) then S(i + 2), had S in
// the softmax's shadow but the loads behind PV: 64 x 4,096 tokens 75.0 us.)
__device__ __forceinline__ void qd_score(QdSmem& sm, const QdParams& p, uint32_t tbase, int tiles)
{
    if (elect_one()) {
        bool ok = qd_wait(sm, p, &sm.q_ready, 0);
        const uint64_t q0 = make_sdesc(smem_u32(sm.q[0]), 16, 1024), qr = make_sdesc(smem_u32(sm.q_rope), 16, 1024);
        const uint64_t r0 = make_sdesc(smem_u32(sm.ring[0]), 16, 1024);
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
            ok = qd_wait(sm, p, &sm.s_empty, i ^ 1);
            const int use = QD_CHUNKS * i, ur = use % QD_RING;
#pragma unroll
            for (int c = 0; c < 4 && ok; ++c) {
                const int u = (use + 1 + c) % QD_RING;
                ok = qd_wait(sm, p, &sm.full[u], (use + 1 + c) / QD_RING);
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = r0 + (uint64_t)(u * (QD_CHUNK >> 4)), q = q0 + (uint64_t)(c * (QD_QCHUNK >> 4));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_ss_8bit(tbase + QD_S_COL, a + 2u * k, q + 2u * k, QD_IDESC_S, (c | k) != 0);
                if (c == 0) {
                    ok = qd_wait(sm, p, &sm.full[ur], use / QD_RING);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t r = r0 + (uint64_t)(ur * (QD_CHUNK >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_ss(tbase + QD_S_COL, r + 2u * k, qr + 2u * k, QD_IDESC_ROPE, 1u);
                    umma_commit(&sm.empty[ur]);
                }
            }
            if (ok) umma_commit(&sm.s_full);
        }
        if (!ok) drain_inflight();
    }
    __syncwarp();
}

// O^T[512 dims x 96] += latents^T . P: a block of 128 dims a chunk.
__device__ __forceinline__ void qd_pv(QdSmem& sm, const QdParams& p, uint32_t tbase, int tiles)
{
    if (elect_one()) {
        bool ok = true;
        const uint64_t pd = make_sdesc(smem_u32(sm.p), QD_CHUNK, 1024), r0 = make_sdesc(smem_u32(sm.ring[0]), QD_CHUNK, 1024);
        const uint32_t one = tbase + QD_ONE_COL, sf = tbase + QD_SF_COL, sf_at = smem_u32(sm.sf);
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
            ok = qd_wait(sm, p, &sm.p_full, i);  // (whose scores have waited for the chunks: 64 x 4,096 tokens 68.7 -> 67.4 us)
            if (!ok) break;
            tc_fence_after();
            tmem_copy_scales(sf, sf_at);
#pragma unroll 1
            for (int c = 0; c < 4 && ok; ++c) {
                const int u = (QD_CHUNKS * i + 1 + c) % QD_RING;
                const uint64_t a = r0 + (uint64_t)(u * (QD_CHUNK >> 4));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_ss_mx(tbase + (uint32_t)(QD_PAIRS * c), a + 256u * k, pd + 256u * k, QD_IDESC_PV + QD_IDESC_NEXT * k, one, sf,
                               (i | k) != 0);
                umma_commit(&sm.empty[u]);
            }
            if (ok) umma_commit(&sm.pv_done);
        }
        if (!ok) drain_inflight();
    }
    __syncwarp();
}

// The queries of this CTA's heads, by the softmax warps: all of them times one power of two 2^a that brings the largest finite
// latent entry to [2^7, 2^8) (less where the rope entries would leave bf16's range), as a sum of two e4m3 numbers, the second
// in units of 1 / 32.  A bf16 has 8 bits, the two numbers 4 each and a sign: exact down to 2^-14 of the largest, and within
// 2^-15 below, half of the second number's smallest step (and 2^-17, half an f16's on the way).
struct QdQueries {
    static constexpr int STEP = 32 * QD_SOFTMAX / 64, ITEMS = QD_HEADS / STEP, ROPES = 32 * QD_SOFTMAX / 8;
    static_assert(STEP * ITEMS == QD_HEADS && ITEMS % 4 == 0 && 2 * ROPES >= QD_HEADS, "whole pieces");
    const uint16_t* src;
    int j, h_first, hr, jr;  // pieces j (8 entries) of heads h_first, + STEP, ..., pieces jr of the rope entries of hr, + ROPES
    uint4 v[ITEMS], v_rope[2];
    uint32_t most, most_rope;  // maxima of magnitudes, two at a time

    __device__ __forceinline__ uint4 piece(int i) const
    {
        return *reinterpret_cast<const uint4*>(src + (size_t)(h_first + STEP * i) * ROW + 8 * j);
    }
    __device__ __forceinline__ uint4 rope(int h) const { return *reinterpret_cast<const uint4*>(src + (size_t)h * ROW + LORA + 8 * jr); }
    static __device__ __forceinline__ uint32_t of8(uint32_t m, const uint4& w)
    {
        constexpr uint32_t A = 0x7FFF7FFFu;
        return max_u16x2(max_u16x2(max_u16x2(max_u16x2(m, w.x & A), w.y & A), w.z & A), w.w & A);
    }
    static __device__ __forceinline__ uint32_t of_warp(uint32_t m) { return __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16)); }
    // the largest in n pieces, step entries apart, NaN and infinities aside
    static __device__ __noinline__ uint32_t finite(const uint16_t* piece, int n, int step)
    {
        uint32_t m = 0;
#pragma unroll 1
        for (int i = 0; i < 8 * n; ++i) {
            const uint32_t x = piece[(size_t)(i >> 3) * step + (i & 7)] & 0x7FFFu;
            if (x < 0x7F80u) m = max(m, x);
        }
        return __reduce_max_sync(0xFFFFFFFFu, m);
    }

    // Reads them once (before the unit's length is known: neither waits for the other).
    __device__ __forceinline__ void read(const QdParams& p, int b, int rank)
    {
        const int tid = (int)threadIdx.x;
        src = p.q_abs + ((size_t)b * H + rank * QD_HEADS) * ROW;
        j = tid & 63, h_first = tid >> 6, hr = tid >> 3, jr = tid & 7;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) v[i] = piece(i);
        v_rope[0] = rope(hr), v_rope[1] = hr + ROPES < QD_HEADS ? rope(hr + ROPES) : make_uint4(0u, 0u, 0u, 0u);
        most_rope = of8(of8(0u, v_rope[0]), v_rope[1]);
        most = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) most = of8(most, v[i]);
    }

    // Leaves them in shared memory; returns 2^-a.
    __device__ __forceinline__ float store(QdSmem& sm)
    {
        const int tid = (int)threadIdx.x, lane = tid & 31;
        most = of_warp(most);
        most_rope = of_warp(most_rope);
        const bool odd = most >= 0x7F80u;
        if (odd) most = finite(src + (size_t)h_first * ROW + 8 * j, ITEMS, STEP * ROW);
        if (most_rope >= 0x7F80u) most_rope = finite(src + (size_t)hr * ROW + LORA + 8 * jr, hr + ROPES < QD_HEADS ? 2 : 1, ROPES * ROW);
        if (lane == 0) sm.most[tid >> 5][0] = most, sm.most[tid >> 5][1] = most_rope;
        if (tid < QD_HEADS) sm.m_ref[tid] = -INFINITY, sm.m_neg[tid] = QD_NONE;
        named_bar(QB_ALL, 32 * QD_SOFTMAX);
        most = __reduce_max_sync(0xFFFFFFFFu, sm.most[lane % QD_SOFTMAX][0]);
        most_rope = __reduce_max_sync(0xFFFFFFFFu, sm.most[lane % QD_SOFTMAX][1]);
        // (exponent fields: a value in [2^(e - 127), 2^(e - 126)))
        int a = most ? 134 - (int)(most >> 7) : 0;
        a = max(min(min(a, 246 - (int)(most_rope >> 7)), 100), -120);
        const float up = __uint_as_float((uint32_t)(127 + a) << 23);
        const float to_f16 = up * (1.f / 256.f);  // (2^-128 at least: exact as a subnormal)
        // A bf16 pair -> first numbers in bytes 0 and 2, second numbers in the lower half.  As with the probabilities: v, the
        // scaled entry times 2^-8, as an f16 has e4m3's bits 7 higher, subnormals included.
        auto two = [&](uint32_t w, uint32_t& first, uint32_t& second) {
            float x, y;
            f32x2_parts(mul_f32x2(f32x2(bf16lo_to_f32(w), bf16hi_to_f32(w)), f32x2(to_f16, to_f16)), x, y);
            const uint32_t v = pack_f16x2(x, y), f = (v + 0x00400040u) & 0xFF80FF80u;
            first = ((f >> 7) & 0x007F007Fu) | ((f >> 8) & ~0x007F007Fu);
            second = pack_e4m3x2_f16(rest_f16x2(v, f));
        };
        auto place = [&](int h) { return sm.q[j >> 4] + h * 128 + ((((j >> 1) & 7) ^ (h & 7)) << 4) + 8 * (j & 1); };
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            uint32_t f[4], s[4];
            two(v[i].x, f[0], s[0]), two(v[i].y, f[1], s[1]), two(v[i].z, f[2], s[2]), two(v[i].w, f[3], s[3]);
            uint8_t* at = place(h_first + STEP * i);
            *reinterpret_cast<uint2*>(at) = make_uint2(__byte_perm(f[0], f[1], 0x6420), __byte_perm(f[2], f[3], 0x6420));
            *reinterpret_cast<uint2*>(at + QD_HEADS * 128) = make_uint2(s[0] | s[1] << 16, s[2] | s[3] << 16);
        }
        if (odd) {  // NaN and infinities become NaN
#pragma unroll 1
            for (int i = 0; i < ITEMS; ++i) {
                const uint16_t* w = src + (size_t)(h_first + STEP * i) * ROW + 8 * j;
                uint8_t* at = place(h_first + STEP * i);
#pragma unroll 1
                for (int e = 0; e < 8; ++e)
                    if ((w[e] & 0x7F80u) == 0x7F80u) at[e] = at[QD_HEADS * 128 + e] = 0x7Fu;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = hr + ROPES * i;
            float x[8];
            unpack8(v_rope[i], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= up;
            if (h < QD_HEADS) *reinterpret_cast<uint4*>(sm.q_rope + h * 128 + ((jr ^ (h & 7)) << 4)) = pack8(x);
        }
        fence_proxy_async_cta();  // the MMAs read them through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready);
        return __uint_as_float((uint32_t)(127 - a) << 23);
    }
};

// A float as an integer that orders like it; NaN below everything.
__device__ __forceinline__ int32_t qd_order(float x)
{
    const int32_t i = (int32_t)__float_as_uint(x);
    return x != x ? (int32_t)0x80000000 : i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float qd_unorder(int32_t i)
{
    return i == (int32_t)0x80000000 ? -INFINITY : __uint_as_float((uint32_t)(i ^ ((i >> 31) & 0x7FFFFFFF)));
}

// Registers that a TMEM load fills are not read before the wait for it.
template <int N> __device__ __forceinline__ void qd_pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The 48 columns of a block of O that hold this group's pairs: first numbers, then second ones.
__device__ __forceinline__ void qd_load_pairs(uint32_t at, uint32_t (&v)[2 * QD_MINE])
{
    tmem_ld32(at, reinterpret_cast<uint32_t(&)[32]>(v));
    tmem_ld16(at + 32u, reinterpret_cast<uint32_t(&)[16]>(v[32]));
}

// x 2^n, x a power of two; 0 and 2^127 beyond what f32 has.
__device__ __forceinline__ float qd_times_power(float x, int n)
{
    const int field = (int)(__float_as_uint(x) >> 23) + n;
    return __uint_as_float(field <= 0 ? 0u : (uint32_t)min(field, 254) << 23);
}

// The references of this group's heads move to the largest score of the tile, rounded up to a whole number, and O's unit 2^od to
// the largest row's, where those are larger; sums and O follow.  All four warps of the group come here together.  u: the raw
// scores; c: what makes log2 units of them; largest: the exponent of the warp's largest row.
__device__ __forceinline__ bool qd_move(QdSmem& sm, const QdParams& p, const float (&u)[QD_MINE], float (&l)[QD_MINE], float c,
                                        int largest, int& od, bool seen, uint32_t tbase, int quarter, int group, int i)
{
    const int lane = (int)lane_id(), h0 = QD_MINE * group;
    int32_t mine = (int32_t)0x80000000;
#pragma unroll
    for (int h = 0; h < QD_MINE; ++h) {
        const int32_t m = __reduce_max_sync(0xFFFFFFFFu, seen ? qd_order(__fmul_rn(u[h], c)) : (int32_t)0x80000000);
        if (lane == h) mine = m;
    }
    if (lane < QD_MINE) sm.part[quarter][h0 + lane] = qd_unorder(mine);
    if (lane == 0) sm.unit[group][quarter] = largest;
    named_bar(QB_GROUP + group, 128);
    if (quarter == 0 && lane < QD_MINE) {
        const float old = sm.m_ref[h0 + lane];
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, sm.part[w][h0 + lane]);
        m = fmaxf(old, ceilf(m));
        sm.m_ref[h0 + lane] = m;
        sm.m_neg[h0 + lane] = m == -INFINITY ? QD_NONE : -m;
        const int4 r = *reinterpret_cast<const int4*>(sm.unit[group]);
        const int now = max(max(od, max(r.x, r.y)), max(r.z, r.w));
        const float f = m == old ? 1.f : ex2_approx(old - m);
        sm.alpha[h0 + lane] = f;
        sm.turn[h0 + lane] = f * ex2_approx((float)(od - now));
        if (lane == 0) sm.od[group] = now;
    }
    named_bar(QB_GROUP + group, 128);
    od = sm.od[group];
    if (i == 0) return true;
    float f[QD_MINE];
#pragma unroll
    for (int h = 0; h < QD_MINE; ++h) {
        l[h] *= sm.alpha[h0 + h];
        f[h] = sm.turn[h0 + h];
    }
    if (!__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.pv_done, i - 1))) return false;
    tc_fence_after();
    const uint32_t t0 = tbase + ((32u * (uint32_t)quarter) << 16) + 2u * (uint32_t)h0;
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
        uint32_t v[2 * QD_MINE];
        qd_load_pairs(t0 + (uint32_t)(QD_PAIRS * x), v);
        tmem_wait_ld();
        qd_pin(v);
#pragma unroll
        for (int e = 0; e < 2 * QD_MINE; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f[e % QD_MINE]);
        tmem_st32(t0 + (uint32_t)(QD_PAIRS * x), reinterpret_cast<uint32_t(&)[32]>(v));
        tmem_st16(t0 + (uint32_t)(QD_PAIRS * x) + 32u, reinterpret_cast<uint32_t(&)[16]>(v[32]));
    }
    tmem_wait_st();
    tc_fence_before();
    return true;
}

// An unseen token whose scores are not finite: its latents become zero, as p = 0 times a NaN would be one.
__device__ __noinline__ void qd_clear(QdSmem& sm, int i, int token)
{
    for (int c = 0; c < 4; ++c) {
        uint4* row = reinterpret_cast<uint4*>(sm.ring[(QD_CHUNKS * i + 1 + c) % QD_RING] + token * 128);
        for (int x = 0; x < 8; ++x) row[x] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Softmax warp: the tokens of its quarter, a lane each, and the heads of its group.  A token's factor is its thread's, and the
// sums of exp stay in the thread until the end; what meets in every tile is the largest P of a head, within the warp, and one
// vote of the group's four warps, whether a row has passed its reference.
__device__ __forceinline__ void qd_softmax(QdSmem& sm, const QdParams& p, QdQueries& queries, const QdUnit& g, int b, int s,
                                           int rank, uint32_t tbase, int tiles)
{
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id(), quarter = warp & 3, group = warp >> 2, h0 = QD_MINE * group;
    const int token = 32 * quarter + lane, line = token & (PAGE - 1), page = quarter >> 1;
    QdLookup look, later;
    if (warp == 0) later(p, g, b, 0, false);
    // Of this thread's token in tile i; the smallest for tokens that are not there, zero rows that are to leave the others their
    // exponent.
    auto row_scale = [&](int i) {
        look(p, g, b, 2 * i, false);
        const int32_t at = __shfl_sync(0xFFFFFFFFu, look.block, (2 * i + page) & 31);
        return at < 0 ? (uint16_t)0x0F80u : *reinterpret_cast<const uint16_t*>(p.slab + (size_t)at * QPAGE + QSCALES + 2 * line);
    };
    const float kq = queries.store(sm) * p.kscale;
    uint16_t next = row_scale(0);
    const uint32_t t_lane = tbase + ((32u * (uint32_t)quarter) << 16);
    if (group == 0) {  // (seen by the second contraction as P is)
        tmem_fill4(t_lane + QD_ONE_COL, 0x7F7F7F7Fu);
        tmem_wait_st();
    }
    // The head of this warp's whose largest weight this lane finds (two lanes of eight: another's again), the lane that finds
    // head h's, and where this one's factors lie.
    const int mine = 12 * (lane >> 4) + 6 * (lane >> 3 & 1) + 2 * (lane & 4 ? 2 : lane >> 1 & 1) + (lane & 1);
    const auto lane_of = [](int h) { return 16 * (h / 12) + 8 * (h / 6 & 1) + h % 6; };
    const auto sf_place = [&](int n) { return 16 * (n & 31) + 4 * (n >> 5) + quarter; };
    const int sf_at = sf_place(2 * h0 + mine) | sf_place(2 * h0 + QD_MINE + mine) << 16;
    float l[QD_MINE];
#pragma unroll
    for (int h = 0; h < QD_MINE; ++h) l[h] = 0.f;
    int od = -127;      // O's unit is 2^od: the largest row's so far, or within 2^TAU of it
    bool big = false;   // a reference of this group's heads is QD_BIG or more
    bool dead = false;  // a wait ran out: this warp only goes on to where the four can leave together
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
        const int e = 2 * i + page, t = PAGE * qd_logical(g, e) + line;
        const bool seen = e < g.npg && qd_seen(p, g.n, t);
        const float scale = __uint_as_float(seen ? (uint32_t)next << 16 : 0x0F800000u);
        const int field = (int)(__float_as_uint(scale) >> 23), largest = __reduce_max_sync(0xFFFFFFFFu, field);
        const float c = kq * scale, up = scale * __uint_as_float((uint32_t)max(254 - largest, 1) << 23);
        const float room = QD_TAU - (float)max(field - 127 - od, 0);  // for a score above its reference
        const bool whole = __all_sync(0xFFFFFFFFu, seen);
        if (i + 1 < tiles) next = row_scale(i + 1);
        dead = dead || !__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.s_full, i));
        float u[QD_MINE];
        {
            uint32_t a[QD_MINE], z[QD_MINE];
            tc_fence_after();
            tmem_ld16(t_lane + QD_S_COL + (uint32_t)h0, reinterpret_cast<uint32_t(&)[16]>(a));
            tmem_ld8(t_lane + QD_S_COL + (uint32_t)h0 + 16u, a + 16);
            tmem_ld16(t_lane + QD_S_COL + (uint32_t)(QD_HEADS + h0), reinterpret_cast<uint32_t(&)[16]>(z));
            tmem_ld8(t_lane + QD_S_COL + (uint32_t)(QD_HEADS + h0) + 16u, z + 16);
            tmem_wait_ld();
            qd_pin(a);
            qd_pin(z);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_empty);
#pragma unroll
            for (int h = 0; h < QD_MINE; h += 2)
                f32x2_parts(fma_f32x2(f32x2(__uint_as_float(z[h]), __uint_as_float(z[h + 1])), f32x2(1.f / QD_LOW, 1.f / QD_LOW),
                                      f32x2(__uint_as_float(a[h]), __uint_as_float(a[h + 1]))),
                            u[h], u[h + 1]);
        }
        float x[QD_MINE];
        auto arguments = [&]() {
#pragma unroll
            for (int h = 0; h < QD_MINE; h += 4) {
                const float4 m = *reinterpret_cast<const float4*>(&sm.m_neg[h0 + h]);
                f32x2_parts(fma_f32x2(f32x2(u[h], u[h + 1]), f32x2(c, c), f32x2(m.x, m.y)), x[h], x[h + 1]);
                f32x2_parts(fma_f32x2(f32x2(u[h + 2], u[h + 3]), f32x2(c, c), f32x2(m.z, m.w)), x[h + 2], x[h + 3]);
            }
            if (big) {
#pragma unroll
                for (int h = 0; h < QD_MINE; ++h) {
                    const float m = sm.m_neg[h0 + h];
                    if (fabsf(m) >= QD_BIG) x[h] = __fmul_rn(u[h], c) + m;
                }
            }
        };
        arguments();
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int h = 4; h < QD_MINE; ++h) m4[h & 3] = fmaxf(m4[h & 3], x[h]);
        const float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // (the first tile sets the references and the unit, without a vote: 64 x 4,096 tokens 67.0 -> 66.8 us)
        if (i == 0 || named_bar_any(QB_GROUP + group, 128, dead || (seen && !(most <= room)))) {
            if (named_bar_any(QB_GROUP + group, 128, dead)) return;
            dead = !qd_move(sm, p, u, l, c, largest - 127, od, seen, tbase, quarter, group, i);
            big = __any_sync(0xFFFFFFFFu, lane < QD_MINE && fabsf(sm.m_neg[h0 + min(lane, QD_MINE - 1)]) >= QD_BIG);
            arguments();
        }
        if (!whole) {
            bool odd = false;
#pragma unroll
            for (int h = 0; h < QD_MINE; ++h) {
                odd = odd || (__float_as_uint(u[h]) & 0x7F800000u) == 0x7F800000u;
                if (!seen) x[h] = -INFINITY;
            }
            if (!seen && odd) qd_clear(sm, i, token);
        }
        // Weights times their rows' powers of two, in units of the largest of those.
#pragma unroll
        for (int h = 0; h < QD_MINE; h += 2) {
            const uint64_t e2 = f32x2(ex2_approx(x[h]), ex2_approx(x[h + 1]));
            f32x2_parts(add_f32x2(f32x2(l[h], l[h + 1]), e2), l[h], l[h + 1]);
            f32x2_parts(mul_f32x2(e2, f32x2(up, up)), x[h], x[h + 1]);
        }
        // The largest of each head over the warp's 32 tokens, a block of the second contraction: two heads a register by the
        // upper halves of their bits (which order like them), half of the heads to the other half of the lanes twice.
        uint32_t sf, unit;
        {
            uint32_t m[QD_MINE / 2];
#pragma unroll
            for (int h = 0; h < QD_MINE; h += 2) m[h / 2] = __byte_perm(__float_as_uint(x[h]), __float_as_uint(x[h + 1]), 0x7632);
            auto halve = [&](auto half, int o) {
                constexpr int n = decltype(half)::value;
                const bool high = lane & o;
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const uint32_t keep = high ? m[j + n] : m[j], give = high ? m[j] : m[j + n];
                    m[j] = max_u16x2(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
                }
            };
            halve(std::integral_constant<int, 6>(), 16);
            halve(std::integral_constant<int, 3>(), 8);
            static_assert(QD_MINE == 24, "three registers a lane");
            // (three: two stay with one half of the lanes, one with the other)
            const uint32_t give = __shfl_xor_sync(0xFFFFFFFFu, lane & 4 ? m[0] : m[2], 4);
            m[1] = max_u16x2(m[1], __shfl_xor_sync(0xFFFFFFFFu, m[1], 4));
            m[0] = max_u16x2(lane & 4 ? m[2] : m[0], give);
            const bool second = (lane & 6) == 2;
            uint32_t pair = __shfl_xor_sync(0xFFFFFFFFu, (lane & 6) == 0 ? m[1] : m[0], 2);
            pair = max_u16x2(second ? m[1] : m[0], pair);
            pair = max_u16x2(pair, __shfl_xor_sync(0xFFFFFFFFu, pair, 1));
            const int top = (int)((lane & 1 ? pair >> 16 : pair & 0xFFFFu) >> 7);  // the largest: in [2^(top - 127), 2^(top - 126))
            // to [1 / 2, 1): P is 2^8 times that
            unit = (uint32_t)(253 - min(top, 252)) << 23;
            sf = (uint32_t)min(max(top + largest - (7 + 127) - od, 0), 254);
        }
        uint32_t w[QD_MINE / 2];  // 24 first numbers, 24 second ones
#pragma unroll
        for (int y = 0; y < QD_MINE / 4; ++y) {
            // (a shuffle each: 64 x 4,096 tokens 67.0 us, by way of shared memory 68.2)
            auto up2 = [&](int h, float& p0, float& p1) {
                const uint32_t f0 = __shfl_sync(0xFFFFFFFFu, unit, lane_of(h)), f1 = __shfl_sync(0xFFFFFFFFu, unit, lane_of(h + 1));
                f32x2_parts(mul_f32x2(f32x2(x[h], x[h + 1]), f32x2(__uint_as_float(f0), __uint_as_float(f1))), p0, p1);
            };
            float a[4];
            up2(4 * y, a[0], a[2]);
            up2(4 * y + 2, a[1], a[3]);
            // Heads 0 and 2 of the four in one register, 1 and 3 in the other.  v = p 2^-8 as an f16 has e4m3's bits, 7 higher,
            // subnormals included: the first number is v rounded there, and no conversion (a quarter of the arithmetic's
            // rate) is needed for it or for what is left.  (Masked so that a NaN stays within its head, whose sum is one too.)
            const uint32_t va = pack_f16x2(a[0], a[1]), vb = pack_f16x2(a[2], a[3]);
            const uint32_t fa = (va + 0x00400040u) & 0x7F807F80u, fb = (vb + 0x00400040u) & 0x7F807F80u;
            w[y] = (fa >> 7) + (fb << 1);
            const uint32_t sa = pack_e4m3x2_f16(rest_f16x2(va, fa)), sb = pack_e4m3x2_f16(rest_f16x2(vb, fb));
            w[QD_MINE / 4 + y] = __byte_perm(sa, sb, 0x5140);
        }
        if (i > 0) dead = dead || !__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.pv_done, i - 1));
#pragma unroll
        for (int y = 0; y < 3; ++y)
            *reinterpret_cast<uint4*>(sm.p + token * 128 + (((3 * group + y) ^ (token & 7)) << 4)) =
                make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
        sm.sf[sf_at & 0xFFFF] = sm.sf[sf_at >> 16] = (uint8_t)sf;
        fence_proxy_async_cta();  // the MMAs read P, and what was cleared, through the async proxy
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
        if (warp == 0 && i + QD_AHEAD < tiles) {  // (a warp that waits for the next scores now)
            const int e2 = 2 * (i + QD_AHEAD);
            later(p, g, b, e2, false);
            const int32_t at = __shfl_sync(0xFFFFFFFFu, later.block, (e2 + rank) & 31);
            if (at >= 0 && lane == 0) bulk_prefetch_l2(p.slab + (size_t)at * QPAGE, QPAGE);
        }
    }
    // The sums of exp: over the lanes -- half of the heads go to the other half of the lanes three times, so that three heads a
    // lane are left to add up over four -- then over the quarters.
    {
        int first = 0;
        auto halve = [&](auto half, int o) {
            constexpr int n = decltype(half)::value;
            const bool high = lane & o;
#pragma unroll
            for (int h = 0; h < n; ++h) {
                const uint32_t lo = __float_as_uint(l[h]), hi = __float_as_uint(l[h + n]), x = high ? lo ^ hi : 0u;
                l[h] = __uint_as_float(lo ^ x) + __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, hi ^ x, o));
            }
            if (high) first += n;
        };
        halve(std::integral_constant<int, 12>(), 16);
        halve(std::integral_constant<int, 6>(), 8);
        halve(std::integral_constant<int, 3>(), 4);
        static_assert(QD_MINE == 24, "three heads a lane");
        auto four = [](float x) {
            x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
            return x + __shfl_xor_sync(0xFFFFFFFFu, x, 1);
        };
        const float l0 = four(l[0]), l1 = four(l[1]), l2 = four(l[2]);
        const int k = lane & 3;
        if (k < 3) sm.part[quarter][h0 + first + k] = k == 0 ? l0 : k == 1 ? l1 : l2;
    }
    dead = dead || !__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.pv_done, tiles - 1));
    if (named_bar_any(QB_GROUP + group, 128, dead)) return;
    tc_fence_after();
    // lane h has head h0 + h of this CTA's
    float total = 1.f;
    if (lane < QD_MINE)
        total = (sm.part[0][h0 + lane] + sm.part[1][h0 + lane]) + (sm.part[2][h0 + lane] + sm.part[3][h0 + lane]);
    float r = g.single ? 1.f / total : 1.f;
    // thread = dim 128 d + 32 quarter + lane of every block d; first the heads' largest entries (two blocks stay in registers)
    auto load = [&](int d, float (&o)[QD_MINE]) {
        uint32_t v[2 * QD_MINE];
        qd_load_pairs(t_lane + (uint32_t)(QD_PAIRS * d + 2 * h0), v);
        tmem_wait_ld();
        qd_pin(v);
#pragma unroll
        for (int h = 0; h < QD_MINE; ++h)
            o[h] = fmaf(__uint_as_float(v[QD_MINE + h]), 1.f / QD_LOW, __uint_as_float(v[h]));
    };
    float o[2][QD_MINE], top[QD_MINE];
#pragma unroll
    for (int d = 3; d >= 0; --d) {
        load(d, o[d & 1]);
#pragma unroll
        for (int h = 0; h < QD_MINE; ++h) top[h] = d == 3 ? fabsf(o[1][h]) : fmaxf(top[h], fabsf(o[d & 1][h]));
    }
    uint32_t most = 0;
#pragma unroll
    for (int h = 0; h < QD_MINE; ++h) {
        const uint32_t v = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top[h]));
        if (lane == h) most = v;
    }
    named_bar(QB_GROUP + group, 128);  // the sums have been read
    if (lane < QD_MINE) sm.part[quarter][h0 + lane] = __uint_as_float(most);
    named_bar(QB_GROUP + group, 128);
    auto place = [&](int h) { return g.single ? (size_t)h * p.B + b : ((size_t)b * p.nsplit + s) * H + h; };
    if (lane < QD_MINE) {
        const int h = h0 + lane;
        float inverse;
        r *= w_row_scale(fmaxf(fmaxf(sm.part[0][h], sm.part[1][h]), fmaxf(sm.part[2][h], sm.part[3][h])) * r, inverse);
        if (quarter == 0) {
            const size_t at = place(rank * QD_HEADS + h);
            // A record's sum comes to [2^-16, 2^-15), its reference takes the power of two (exactly, below 2^22): O is then at most
            // that much of the rows' largest, and f32 holds what undoes its power of two, and the merge's sums.
            const float m = sm.m_ref[h];
            const bool turns = !g.single && fabsf(m) < 4194304.f && total > 0.f && total < INFINITY;
            const int e = turns ? (int)(__float_as_uint(total) >> 23) - 111 : 0;
            (g.single ? p.oscale : p.ws_oscale)[at] = qd_times_power(inverse, od - e);
            if (!g.single) p.ws_ml[at] = make_float2(m + (float)e, total * qd_times_power(1.f, -e));
        }
    }
    // two lanes trade, so that each has a pair of neighbouring dims of every second block
    const bool upper = lane & 1;
    uint16_t* out = (g.single ? p.olat : p.ws_o) + place(rank * QD_HEADS + h0) * LORA;
    const size_t step = (g.single ? (size_t)p.B : 1) * LORA;
#pragma unroll
    for (int d = 0; d < 4; d += 2) {
        if (d > 0) load(d, o[0]), load(d + 1, o[1]);
        uint16_t* to = out + w_dim_place(128 * (upper ? d + 1 : d) + 32 * quarter + (lane & ~1));
#pragma unroll
        for (int h = 0; h < QD_MINE; ++h) {
            const float f = __shfl_sync(0xFFFFFFFFu, r, h), mine0 = o[0][h] * f, mine1 = o[1][h] * f;
            const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? mine0 : mine1, 1);
            *reinterpret_cast<uint32_t*>(to + h * step) = upper ? pack_f16x2(other, mine1) : pack_f16x2(mine0, other);
        }
    }
}

// ---- the kernel ---------------------------------------------------------------------------

// Two CTAs a unit, split s of slot b: 48 heads each.
__global__ void __launch_bounds__(QD_THREADS, 1)
    k3mla_quant_decode_kernel(const __grid_constant__ CUtensorMap tm_page, const QdParams p)
{
    extern __shared__ uint8_t smem_raw[];
    QdSmem& sm = *reinterpret_cast<QdSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int rank = (int)(blockIdx.x & 1u), warp = (int)(threadIdx.x >> 5), unit = (int)(blockIdx.x >> 1);
    const int b = unit % p.B, s = unit / p.B;  // (first splits first: where lists are cut unevenly, the short rests come last)
    if (threadIdx.x == 32 * QW_LOAD) {
        qd_init(sm, p);
        fence_mbarrier_init_cluster();
        tma_prefetch_desc(&tm_page);
    }
    if (warp == QW_PV) {
        tmem_alloc(&sm.tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    griddep_wait();
    griddep_launch_dependents();
    QdQueries queries;
    if (warp < QD_SOFTMAX) queries.read(p, b, rank);
    const QdUnit g = qd_unit(p, b, s, s == 0 && rank == 0 && threadIdx.x == 0);
    if (s == 0 && g.n == 0 && threadIdx.x < QD_HEADS) p.oscale[(size_t)(rank * QD_HEADS + (int)threadIdx.x) * p.B + b] = 0.f;
    const int tiles = (g.npg + 1) / 2;
    if (tiles > 0) {
        if (warp < QD_SOFTMAX) qd_softmax(sm, p, queries, g, b, s, rank, tbase, tiles);
        else if (warp == QW_LOAD) qd_produce(sm, tm_page, p, g, b, tiles);
        else if (warp == QW_SCORE) qd_score(sm, p, tbase, tiles);
        else if (warp == QW_PV) qd_pv(sm, p, tbase, tiles);
    }
    // After an abort a role leaves wherever it stands, with copies and MMAs under way: they land before the CTA gives its
    // shared memory and its TMEM back.
    if (aborted(sm)) drain_inflight();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == QW_PV) tmem_dealloc(tbase, TMEM_COLS);
}

}  // namespace k3

using namespace k3;

extern "C" size_t k3mla_quant_decode_workspace_bytes(int B, int max_ctx, int window, int n_sink, int split_tokens)
{
    if (B <= 0 || max_ctx <= 0 || window < 1 || n_sink < 0 || split_tokens < 0 || split_tokens % TILE != 0) return 0;
    return w_layout(B, w_nsplit(max_ctx, window, n_sink, split_tokens)).total;
}

extern "C" int k3mla_quant_split_tokens(int B, int max_ctx, int window, int n_sink)
{
    // Up to four slots: the expansion adds the splits up, and window.cu's rule is within 3% of the best of up to 22 lengths.
    if (B <= 4 || max_ctx <= 0 || window < 1 || n_sink < 0) return k3mla_window_split_tokens(B, max_ctx, window, n_sink);
    // More: the length with which the last CTA ends first, two a split, the rests of the lists behind their full splits, at 7.6
    // us a unit and 1.6 a tile, and 3.3 us and what the records cost for the merge.  Over 120 pairs of 6 to 220 slots and 300 to
    // 30,000 tokens that is within 0.1% of the best of up to 40 lengths on average.  Window.cu's rule, which fills one round,
    // against it: 10 slots over 500 tokens 21.2 -> 18.6 us, 26 over 10,000 86 -> 76, 40 over 10,000 145 -> 109 and over 30,000
    // 401 -> 261, 64 over 4,096 the same and over 30,000 403 -> 367, 90 over 30,000 797 -> 520.
    const long long sms = sm_count(), tiles = (w_max_pages(max_ctx, window, n_sink) * PAGE + TILE - 1) / TILE;
    double least = 1e300;
    long long split = tiles;
    auto look = [&](long long part) {
        const long long parts = (tiles + part - 1) / part, rest = tiles - (parts - 1) * part;
        if (parts > 4 * sms) return;
        const double us = units_span(2ll * B * (parts - 1), 7.6 + 1.6 * (double)part, 2ll * B, 7.6 + 1.6 * (double)rest, sms) +
                          (parts > 1 ? 3.3 + (0.21 + 0.025 * B) * (double)parts : 0.);
        if (us < least) least = us, split = part;
    };
    for (long long n = 1; n <= std::min(tiles, 4 * sms); ++n) look((tiles + n - 1) / n);
    for (long long part = 1, step = 1 + tiles / 1024; part < tiles; part += step) look(part);
    return (int)std::min<long long>(split * TILE, W_UNIT_PAGES * PAGE);  // (a unit takes no more)
}

static int quant_decode(const uint16_t* q_abs, const uint8_t* slab, int n_pages, int n_layers, int layer,
                        const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len, const uint16_t* w_kv_b,
                        uint16_t scale_bf16, uint16_t* out, void* workspace, size_t ws_bytes, int B, int max_ctx, int window,
                        int n_sink, int split_tokens, int32_t* dev_err, void* stream, uint64_t wait_ns, int withhold)
{
    QdParams p;
    std::memset(&p, 0, sizeof(p));
    if (B < 0 || split_tokens < 0 || split_tokens % TILE != 0) {
        set_error("k3mla_quant_decode: invalid sizes, window or scale");
        return K3MLA_E_INVALID;
    }
    if (B == 0) return K3MLA_OK;
    if (n_pages <= 0 || n_layers <= 0 || layer < 0 || layer >= n_layers || max_pages_per_slot <= 0 || max_ctx <= 0 ||
        window < 1 || n_sink < 0 || !w_scale(scale_bf16, &p.kscale)) {
        set_error("k3mla_quant_decode: invalid sizes, window or scale");
        return K3MLA_E_INVALID;
    }
    if ((long long)n_pages * n_layers + 1 > 0x7FFFFFFFll) {
        set_error("k3mla_quant_decode: more than 2^31 page blocks");
        return K3MLA_E_INVALID;
    }
    if (!q_abs || !slab || !block_table || !ctx_len || !w_kv_b || !out || !workspace || !aligned(q_abs, 16) ||
        !aligned(slab, 128) || !aligned(w_kv_b, 16) || !aligned(out, 16) || !aligned(workspace, 256)) {
        set_error("k3mla_quant_decode: null or misaligned pointer");
        return K3MLA_E_INVALID;
    }
    const size_t need = k3mla_quant_decode_workspace_bytes(B, max_ctx, window, n_sink, split_tokens);
    if (ws_bytes < need) {
        set_error("k3mla_quant_decode: workspace %zu < %zu bytes", ws_bytes, need);
        return K3MLA_E_WORKSPACE;
    }
    p.cap = (int)std::min<long long>(std::min(max_ctx, 0x7FFFFF00), (long long)max_pages_per_slot * PAGE);
    const int ns = w_nsplit(max_ctx, window, n_sink, split_tokens);
    const long long longest = w_max_pages(p.cap, window, n_sink), split = (split_tokens ? split_tokens : SPLIT_MAX) / PAGE;
    if (!w_unit_fits("k3mla_quant_decode", std::min(longest, split))) return K3MLA_E_INVALID;
    if (B > 65535 || (long long)B * ns * H > 0x7FFFFFFFll) {
        set_error("k3mla_quant_decode: too many slots or splits");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    const WinWs wl = w_layout(B, ns);
    uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
    p.q_abs = q_abs, p.slab = slab, p.table = block_table, p.ctx_len = ctx_len;
    p.olat = reinterpret_cast<uint16_t*>(ws + wl.olat);
    p.oscale = reinterpret_cast<float*>(ws + wl.scale);
    p.ws_o = ns > 1 ? reinterpret_cast<uint16_t*>(ws + wl.o) : nullptr;
    p.ws_oscale = ns > 1 ? reinterpret_cast<float*>(ws + wl.oscale) : nullptr;
    p.ws_ml = ns > 1 ? reinterpret_cast<float2*>(ws + wl.ml) : nullptr;
    p.dev_err = dev_err;
    p.B = B, p.max_pages = max_pages_per_slot, p.n_pages = n_pages, p.n_layers = n_layers, p.layer = layer;
    p.window = window, p.n_sink = n_sink, p.split_tokens = split_tokens, p.nsplit = ns;
    p.wait_ns = wait_ns, p.withhold = withhold;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    CUtensorMap tm_page;
    const uint64_t dims[4] = {128, PAGE, QD_CHUNKS, (uint64_t)n_pages * n_layers}, strides[3] = {QROW, 128, QPAGE};
    const uint32_t box[4] = {128, PAGE, 1, 1};
    int rc = make_tmap_bytes(&tm_page, 4, slab, dims, strides, box);
    if (rc) return rc;
    static bool attr_done[64] = {};
    const size_t smem = sizeof(QdSmem) + 1024;
    set_smem_attr(reinterpret_cast<const void*>(k3mla_quant_decode_kernel), smem, attr_done);
    rc = launch_pdl(k3mla_quant_decode_kernel, dim3((unsigned)(2 * B * ns)), dim3(QD_THREADS), smem, st,
                    "k3mla_quant_decode_kernel", tm_page, p);
    if (rc) return rc;
    TailArgs t;
    t.ctx_len = ctx_len, t.olat = p.olat, t.oscale = p.oscale, t.ws_o = p.ws_o, t.ws_oscale = p.ws_oscale, t.ws_ml = p.ws_ml;
    t.w_kv_b = w_kv_b, t.out = out, t.dev_err = dev_err, t.B = B, t.cap = p.cap, t.window = window, t.n_sink = n_sink;
    t.split_tokens = split_tokens, t.nsplit = ns;
    return launch_window_tail(t, st);
}

extern "C" int k3mla_quant_decode(const uint16_t* q_abs, const uint8_t* slab, int n_pages, int n_layers, int layer,
                                  const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                                  const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                  size_t ws_bytes, int B, int max_ctx, int window, int n_sink, int split_tokens,
                                  int32_t* dev_err, void* stream)
{
    return quant_decode(q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, ctx_len, w_kv_b, scale_bf16, out,
                        workspace, ws_bytes, B, max_ctx, window, n_sink, split_tokens, dev_err, stream, WAIT_NS, 0);
}

extern "C" int k3mla_diag_quant_timeout(const uint16_t* q_abs, const uint8_t* slab, int n_pages, int n_layers, int layer,
                                        const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                                        const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                        size_t ws_bytes, int B, int max_ctx, int window, int n_sink, int split_tokens,
                                        int withhold_tile, uint32_t wait_us, int32_t* dev_err, void* stream)
{
    if (withhold_tile < 0 || withhold_tile >= 1 << 30 || wait_us < 100 || wait_us > 100000) {
        set_error("k3mla_diag_quant_timeout: 0 <= withhold_tile < 2^30 and 100 <= wait_us <= 100000");
        return K3MLA_E_INVALID;
    }
    return quant_decode(q_abs, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot, ctx_len, w_kv_b, scale_bf16, out,
                        workspace, ws_bytes, B, max_ctx, window, n_sink, split_tokens, dev_err, stream,
                        (uint64_t)wait_us * 1000ull, withhold_tile + 1);
}
