// quant_decode.cu -- absorbed-MLA decode over the 8-bit latent cache (quant.cuh), over the whole context or a window and the
// first tokens, for sm_103a.
//
// Math: as window.cu's decode, with row_t the values that the cache stands for: code 2^n_t and rope 2^n_t.  With raw_t the
// product of q_abs with the row in the row's own units,
//     s_t = scale 2^n_t raw_t,   p = softmax(s),   o_lat = sum_t (p_t 2^n_t) code_t,   out = W_UV o_lat.
// Slots are cut into splits by window.cu's rule, and what a split leaves behind -- o_lat, or O and its reference and sum -- is
// what window.cu's merge and expansion take.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

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
constexpr int QD_HALF = 24;                     // ... of a softmax warp
constexpr int QD_TILE = 128;                    // tokens of a tile: two pages of the unit's list
constexpr int QD_PAIRS = 2 * QD_HEADS;          // columns: every head twice, a first and a second e4m3 number
constexpr int QD_CHUNK = QD_TILE * 128;         // a tile's chunk: [128 tokens][128 B]; a tile is the rope chunk, then 4 of latents
constexpr int QD_CHUNKS = 5;
constexpr int QD_RING = 9;
constexpr int QD_QCHUNK = QD_PAIRS * 128;       // 128 dims of the queries' pairs
constexpr int QD_SOFTMAX = 8;                   // warps 0 .. 7: quarter of the tile's tokens w & 3, half of the heads w >> 2
constexpr int QW_LOAD = 8, QW_SCORE = 9, QW_PV = 10, QW_AHEAD = 11;
constexpr int QD_THREADS = 384;
constexpr uint32_t QD_S_COL = 4 * QD_PAIRS;     // TMEM: O by blocks of 128 dims at 96 d, then S
constexpr uint32_t QB_HALF = 1, QB_ALL = 3;     // named barriers: a half's four softmax warps (1, 2); all eight
constexpr float QD_TAU = 1.f;                   // a reference moves when a row passes it by more than 2^TAU
constexpr float QD_UP = 64.f;                   // p times its row's power of two is at most QD_UP 2^TAU times a scale's mantissa: 256
constexpr float QD_LOW = 16.f;                  // the second number's units: 1 / 16
constexpr uint32_t QD_IDESC_S = make_idesc_e4m3(128, QD_PAIRS, 0, 0);
constexpr uint32_t QD_IDESC_ROPE = make_idesc_bf16(128, QD_HEADS, 0, 0);
constexpr uint32_t QD_IDESC_PV = make_idesc_e4m3(128, QD_PAIRS, 1, 1);

struct __align__(1024) QdSmem {
    uint8_t q[4][QD_QCHUNK];          // K-major B of the scores: rows h (first numbers) and 48 + h (second)
    uint8_t q_rope[QD_HEADS * 128];
    uint8_t ring[QD_RING][QD_CHUNK];
    uint8_t p[QD_TILE * 128];         // MN-major B of the second contraction: [token][half: 24 first, 24 second numbers]
    uint64_t full[QD_RING], empty[QD_RING];
    uint64_t q_ready, s_full, s_empty, p_full, pv_done;
    float m_ref[QD_HEADS];            // the references, in log2 units
    float alpha[QD_HEADS];            // what a moved reference turns the sums by
    float part[4][QD_HEADS];          // a quarter's maxima or sums
    float up[QD_HEADS];               // the write-out's powers of two
    uint32_t most[QD_SOFTMAX][2];     // the prologue's maxima by warp: latents, rope
    uint32_t tmem_base;
    int32_t tiles_done;               // tiles whose second contraction has been issued
    int32_t abort_flag;
    uint64_t wait_ns;
};
static_assert(QD_QCHUNK % 1024 == 0 && (QD_HEADS * 128) % 1024 == 0, "operand tiles start 1024-byte aligned");
static_assert(sizeof(QdSmem) + 1024 <= 227 * 1024, "shared memory of one CTA (with alignment slack)");
static_assert(4 * QD_PAIRS + QD_PAIRS <= 512, "TMEM columns");

__device__ __forceinline__ bool qd_wait(QdSmem& sm, const QdParams& p, uint64_t* bar, int phase)
{
    return wait_bar(bar, (uint32_t)phase & 1u, sm, p.dev_err, true);
}

__device__ __forceinline__ void qd_init(QdSmem& sm, const QdParams& p)
{
    sm.wait_ns = p.wait_ns;
    sm.abort_flag = 0;
    sm.tiles_done = 0;
#pragma unroll 1
    for (int i = 0; i < QD_RING; ++i) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], 2);  // both CTAs have read theirs: a load writes to both
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

// The producer: of every chunk this CTA's page (entry 2 i + rank of the list), into both CTAs.
__device__ __forceinline__ void qd_produce(QdSmem& sm, const CUtensorMap& tm_page, const QdParams& p, const QdUnit& g, int b,
                                           int rank, int tiles)
{
    bool ok = true;  // (the elected lane's)
    QdLookup look;
    const int none = p.n_pages * p.n_layers;  // past the end: read as zeros
    for (int i = 0; i < tiles; ++i) {
        look(p, g, b, 2 * i, true);
        const int32_t at = __shfl_sync(0xFFFFFFFFu, look.block, (2 * i + rank) & 31);
        if (elect_one()) {
#pragma unroll 1
            for (int c = 0; c < QD_CHUNKS && ok; ++c) {
                const int use = QD_CHUNKS * i + c, u = use % QD_RING;
                ok = qd_wait(sm, p, &sm.empty[u], (use / QD_RING) ^ 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&sm.full[u], QD_CHUNK);
                // (diagnostic: a load never issued)
                if (c != 1 || i + 1 != p.withhold)
                    tma_load_4d_mc(sm.ring[u] + rank * (PAGE * 128), &tm_page, 0, 0, c ? c - 1 : 4, at < 0 ? none : at,
                                   &sm.full[u], 3);
            }
        }
        __syncwarp();
    }
    if (!ok) drain_inflight();
}

// S[128 tokens x 96] = tile . queries: four chunks of 128 e4m3 latents, the rope chunk in bf16 onto the first numbers' columns.
__device__ __forceinline__ void qd_score(QdSmem& sm, const QdParams& p, uint32_t tbase, int tiles)
{
    if (elect_one()) {
        bool ok = qd_wait(sm, p, &sm.q_ready, 0);
        const uint64_t q0 = make_sdesc(smem_u32(sm.q[0]), 16, 1024), qr = make_sdesc(smem_u32(sm.q_rope), 16, 1024);
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
            ok = qd_wait(sm, p, &sm.s_empty, i ^ 1);
            const int use = QD_CHUNKS * i, ur = use % QD_RING;
#pragma unroll 1
            for (int c = 0; c < 4 && ok; ++c) {
                const int u = (use + 1 + c) % QD_RING;
                ok = qd_wait(sm, p, &sm.full[u], (use + 1 + c) / QD_RING);
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = make_sdesc(smem_u32(sm.ring[u]), 16, 1024), q = q0 + (uint64_t)(c * (QD_QCHUNK >> 4));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_ss_8bit(tbase + QD_S_COL, a + 2u * k, q + 2u * k, QD_IDESC_S, (c | k) != 0);
                if (c == 0) {
                    ok = qd_wait(sm, p, &sm.full[ur], use / QD_RING);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t r = make_sdesc(smem_u32(sm.ring[ur]), 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_ss(tbase + QD_S_COL, r + 2u * k, qr + 2u * k, QD_IDESC_ROPE, 1u);
                    umma_commit_mc(&sm.empty[ur], 3);
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
        const uint64_t pd = make_sdesc(smem_u32(sm.p), QD_CHUNK, 1024);
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
            ok = qd_wait(sm, p, &sm.p_full, i);
#pragma unroll 1
            for (int c = 0; c < 4 && ok; ++c) {
                const int use = QD_CHUNKS * i + 1 + c, u = use % QD_RING;
                ok = qd_wait(sm, p, &sm.full[u], use / QD_RING);
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = make_sdesc(smem_u32(sm.ring[u]), QD_CHUNK, 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_ss_8bit(tbase + (uint32_t)(QD_PAIRS * c), a + 256u * k, pd + 256u * k, QD_IDESC_PV, (i | k) != 0);
                umma_commit_mc(&sm.empty[u], 3);
            }
            if (ok) umma_commit(&sm.pv_done);
            *reinterpret_cast<volatile int32_t*>(&sm.tiles_done) = i + 1;
        }
        if (!ok) drain_inflight();
    }
    __syncwarp();
}

// Page blocks into L2, QD_AHEAD tiles before their second contraction.
constexpr int QD_AHEAD = 4;
__device__ __forceinline__ void qd_prefetch(QdSmem& sm, const QdParams& p, const QdUnit& g, int b, int rank, int tiles)
{
    QdLookup look;
    for (int i = 0; i < tiles; ++i) {
        look(p, g, b, 2 * i, false);
        const int32_t at = __shfl_sync(0xFFFFFFFFu, look.block, (2 * i + rank) & 31);
        if (i < 2) continue;  // (the first tiles are loaded at once)
        if (!__all_sync(0xFFFFFFFFu, wait_count(&sm.tiles_done, i - QD_AHEAD, sm, p.dev_err))) return;
        if (at >= 0 && elect_one()) bulk_prefetch_l2(p.slab + (size_t)at * QPAGE, QPAGE);
        __syncwarp();
    }
}

// The queries of this CTA's heads, by the softmax warps: all of them times one power of two 2^a that brings the largest finite
// latent entry to [2^7, 2^8) (less where the rope entries would leave bf16's range), as a sum of two e4m3 numbers, the second
// in units of 1 / 16.  A bf16 has 8 bits, the two numbers 4 each and a sign: exact down to 2^-14 of the largest, and within
// 2^-14 below.  Returns 2^-a.
__device__ __forceinline__ float qd_queries(QdSmem& sm, const QdParams& p, int b, int rank)
{
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint16_t* src = p.q_abs + ((size_t)b * H + rank * QD_HEADS) * ROW;
    constexpr int ITEMS = QD_HEADS * (LORA / 16) / (32 * QD_SOFTMAX);  // pieces of 16 entries a thread: 6
    uint4 v[ITEMS][2], vr[2];
    uint32_t most = 0, most_rope = 0;
    auto largest = [](uint32_t m, uint32_t w) {  // of bf16 pairs, NaN and infinities aside
        const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
        return max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    };
    auto of4 = [&](uint32_t m, const uint4& w) { return largest(largest(largest(largest(m, w.x), w.y), w.z), w.w); };
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int item = tid + 32 * QD_SOFTMAX * i, h = item >> 5, j = item & 31;
        const uint4* at = reinterpret_cast<const uint4*>(src + (size_t)h * ROW + 16 * j);
        v[i][0] = at[0];
        v[i][1] = at[1];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int item = tid + 32 * QD_SOFTMAX * i, h = item >> 3, j = item & 7;
        vr[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < QD_HEADS) vr[i] = *reinterpret_cast<const uint4*>(src + (size_t)h * ROW + LORA + 8 * j);
        most_rope = of4(most_rope, vr[i]);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) most = of4(of4(most, v[i][0]), v[i][1]);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    most_rope = __reduce_max_sync(0xFFFFFFFFu, most_rope);
    if (lane == 0) sm.most[warp][0] = most, sm.most[warp][1] = most_rope;
    if (tid < QD_HEADS) sm.m_ref[tid] = -INFINITY;
    named_bar(QB_ALL, 32 * QD_SOFTMAX);
#pragma unroll
    for (int w = 0; w < QD_SOFTMAX; ++w) {
        most = max(most, sm.most[w][0]);
        most_rope = max(most_rope, sm.most[w][1]);
    }
    // (exponent fields: a value in [2^(e - 127), 2^(e - 126)))
    int a = most ? 134 - (int)(most >> 7) : 0;
    a = max(min(min(a, 246 - (int)(most_rope >> 7)), 100), -120);
    const float up = __uint_as_float((uint32_t)(127 + a) << 23);
    auto two = [&](uint32_t w, uint32_t& first, uint32_t& second) {  // a bf16 pair -> the pairs of codes
        if ((w & 0x7F80u) == 0x7F80u) w |= 0x7Fu;
        if ((w & 0x7F800000u) == 0x7F800000u) w |= 0x7F0000u;
        const float x = bf16lo_to_f32(w) * up, y = bf16hi_to_f32(w) * up;
        first = pack_e4m3x2(x, y);
        float fx, fy;
        f16x2_parts(e4m3x2_to_f16x2(first), fx, fy);
        second = pack_e4m3x2((x - fx) * QD_LOW, (y - fy) * QD_LOW);
    };
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int item = tid + 32 * QD_SOFTMAX * i, h = item >> 5, j = item & 31;
        uint32_t f[8], s[8];
        two(v[i][0].x, f[0], s[0]), two(v[i][0].y, f[1], s[1]), two(v[i][0].z, f[2], s[2]), two(v[i][0].w, f[3], s[3]);
        two(v[i][1].x, f[4], s[4]), two(v[i][1].y, f[5], s[5]), two(v[i][1].z, f[6], s[6]), two(v[i][1].w, f[7], s[7]);
        uint8_t* at = sm.q[j >> 3] + h * 128 + (((j & 7) ^ (h & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = make_uint4(f[0] | f[1] << 16, f[2] | f[3] << 16, f[4] | f[5] << 16, f[6] | f[7] << 16);
        *reinterpret_cast<uint4*>(at + QD_HEADS * 128) =
            make_uint4(s[0] | s[1] << 16, s[2] | s[3] << 16, s[4] | s[5] << 16, s[6] | s[7] << 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int item = tid + 32 * QD_SOFTMAX * i, h = item >> 3, j = item & 7;
        if (h >= QD_HEADS) continue;
        float x[8];
        unpack8(vr[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= up;
        *reinterpret_cast<uint4*>(sm.q_rope + h * 128 + ((j ^ (h & 7)) << 4)) = pack8(x);
    }
    fence_proxy_async_cta();  // the MMAs read them through the async proxy
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_ready);
    return __uint_as_float((uint32_t)(127 - a) << 23);
}

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

// The references of this half's heads move to the largest s + k of the tile where that is larger, k a row's exponent; sums and
// O follow.  All four warps of the half come here together.  u: the raw scores; c: what makes log2 units of them.
__device__ __forceinline__ bool qd_move(QdSmem& sm, const QdParams& p, const float (&u)[QD_HALF], float (&l)[QD_HALF], float c,
                                     float k, bool seen, uint32_t tbase, int quarter, int half, int i)
{
    const int lane = (int)lane_id(), h0 = QD_HALF * half;
    int32_t mine = (int32_t)0x80000000;
#pragma unroll
    for (int h = 0; h < QD_HALF; ++h) {
        const int32_t m = __reduce_max_sync(0xFFFFFFFFu, seen ? qd_order(fmaf(u[h], c, k)) : (int32_t)0x80000000);
        if (lane == h) mine = m;
    }
    if (lane < QD_HALF) sm.part[quarter][h0 + lane] = qd_unorder(mine);
    named_bar(QB_HALF + half, 128);
    if (quarter == 0 && lane < QD_HALF) {
        const float old = sm.m_ref[h0 + lane];
        float m = old;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, sm.part[w][h0 + lane]);
        sm.m_ref[h0 + lane] = m;
        sm.alpha[h0 + lane] = m == old ? 1.f : ex2_approx(old - m);
    }
    named_bar(QB_HALF + half, 128);
#pragma unroll
    for (int h = 0; h < QD_HALF; ++h) l[h] *= sm.alpha[h0 + h];
    if (i == 0) return true;
    if (!__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.pv_done, i - 1))) return false;
    tc_fence_after();
    const uint32_t t0 = tbase + ((32u * (uint32_t)quarter) << 16) + 2u * (uint32_t)h0;
#pragma unroll 1
    for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            uint32_t v[16];
            const uint32_t at = t0 + (uint32_t)(QD_PAIRS * d + 16 * x);
            tmem_ld16(at, v);
            tmem_wait_ld();
            qd_pin(v);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                v[e] = __float_as_uint(__uint_as_float(v[e]) * sm.alpha[h0 + (16 * x + e) % QD_HALF]);
            tmem_st16(at, v);
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

// Softmax warp: the tokens of its quarter, a lane each, and the heads of its half.  A token's factor is its thread's, and the
// sums of exp stay in the thread until the end; what meets in every tile is one vote of the half's four warps, whether a row
// has passed its reference.
__device__ __forceinline__ void qd_softmax(QdSmem& sm, const QdParams& p, const QdUnit& g, int b, int s, int rank,
                                           uint32_t tbase, int tiles)
{
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id(), quarter = warp & 3, half = warp >> 2, h0 = QD_HALF * half;
    const int token = 32 * quarter + lane, line = token & (PAGE - 1), page = quarter >> 1;
    const float kq = qd_queries(sm, p, b, rank) * p.kscale;
    const uint32_t t_lane = tbase + ((32u * (uint32_t)quarter) << 16);
    QdLookup look;
    auto row_scale = [&](int i) {  // of this thread's token in tile i; 1 for tokens that are not there
        look(p, g, b, 2 * i, false);
        const int32_t at = __shfl_sync(0xFFFFFFFFu, look.block, (2 * i + page) & 31);
        return at < 0 ? (uint16_t)0x3F80u : *reinterpret_cast<const uint16_t*>(p.slab + (size_t)at * QPAGE + QSCALES + 2 * line);
    };
    float l[QD_HALF];
#pragma unroll
    for (int h = 0; h < QD_HALF; ++h) l[h] = 0.f;
    uint16_t next = row_scale(0);
    bool dead = false;  // a wait ran out: this warp only goes on to where the four can leave together
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
        const int e = 2 * i + page, t = PAGE * qd_logical(g, e) + line;
        const bool seen = e < g.npg && qd_seen(p, g.n, t);
        const float scale = seen ? __uint_as_float((uint32_t)next << 16) : 1.f;
        const float k = (float)((int)(__float_as_uint(scale) >> 23) - 127), c = kq * scale;
        if (i + 1 < tiles) next = row_scale(i + 1);
        dead = dead || !__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.s_full, i));
        float u[QD_HALF];
        {
            uint32_t a[QD_HALF], z[QD_HALF];
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
            for (int h = 0; h < QD_HALF; ++h) u[h] = fmaf(__uint_as_float(z[h]), 1.f / QD_LOW, __uint_as_float(a[h]));
        }
        float x[QD_HALF], most = -INFINITY;
#pragma unroll
        for (int h = 0; h < QD_HALF; ++h) {
            x[h] = fmaf(u[h], c, -sm.m_ref[h0 + h]);
            most = fmaxf(most, x[h]);
        }
        bool odd = false;
        if (!seen) {
#pragma unroll
            for (int h = 0; h < QD_HALF; ++h) odd = odd || (__float_as_uint(u[h]) & 0x7F800000u) == 0x7F800000u;
        }
        // (the first tile's references are -inf)
        if (named_bar_any(QB_HALF + half, 128, dead || i == 0 || (seen && !(most <= QD_TAU - k)))) {
            if (named_bar_any(QB_HALF + half, 128, dead)) return;
            dead = !qd_move(sm, p, u, l, c, k, seen, tbase, quarter, half, i);
#pragma unroll
            for (int h = 0; h < QD_HALF; ++h) {
                const float m = sm.m_ref[h0 + h];
                x[h] = fmaf(u[h], c, m == -INFINITY ? 0.f : -m);
            }
        }
        if (odd) qd_clear(sm, i, token);
        uint32_t w[QD_HALF / 2];  // 24 first numbers, 24 second ones
        const float up = scale * QD_UP;
#pragma unroll
        for (int y = 0; y < QD_HALF / 4; ++y) {
            uint32_t first[2], second[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int h = 4 * y + 2 * z;
                float e0 = ex2_approx(x[h]), e1 = ex2_approx(x[h + 1]);
                if (!seen) e0 = e1 = 0.f;
                l[h] += e0;
                l[h + 1] += e1;
                const uint32_t v = pack_f16x2(e0 * up, e1 * up);
                first[z] = pack_e4m3x2_f16(v);
                second[z] = pack_e4m3x2_f16(rest_f16x2(v, e4m3x2_to_f16x2(first[z])));
            }
            w[y] = first[0] | first[1] << 16;
            w[QD_HALF / 4 + y] = second[0] | second[1] << 16;
        }
        if (i > 0) dead = dead || !__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.pv_done, i - 1));
#pragma unroll
        for (int y = 0; y < 3; ++y)
            *reinterpret_cast<uint4*>(sm.p + token * 128 + (((3 * half + y) ^ (token & 7)) << 4)) =
                make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
        fence_proxy_async_cta();  // the MMAs read P, and what was cleared, through the async proxy
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
    }
    // the sums of exp: over the lanes, then over the quarters
    float mine = 0.f;
#pragma unroll
    for (int h = 0; h < QD_HALF; ++h) {
        float v = l[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == h) mine = v;
    }
    if (lane < QD_HALF) sm.part[quarter][h0 + lane] = mine;
    dead = dead || !__all_sync(0xFFFFFFFFu, qd_wait(sm, p, &sm.pv_done, tiles - 1));
    if (named_bar_any(QB_HALF + half, 128, dead)) return;
    tc_fence_after();
    // lane h has head h0 + h of this CTA's
    float total = 1.f;
    if (lane < QD_HALF)
        total = (sm.part[0][h0 + lane] + sm.part[1][h0 + lane]) + (sm.part[2][h0 + lane] + sm.part[3][h0 + lane]);
    const float r = (g.single ? 1.f / total : 1.f) * (1.f / QD_UP);
    // thread = dim 128 d + 32 quarter + lane of every block d
    float o[4][QD_HALF];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t v[3][16];
#pragma unroll
        for (int y = 0; y < 3; ++y) tmem_ld16(t_lane + (uint32_t)(QD_PAIRS * d + 2 * h0 + 16 * y), v[y]);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 3; ++y) qd_pin(v[y]);
#pragma unroll
        for (int h = 0; h < QD_HALF; ++h)
            o[d][h] = fmaf(__uint_as_float(v[(QD_HALF + h) / 16][(QD_HALF + h) % 16]), 1.f / QD_LOW,
                           __uint_as_float(v[h / 16][h % 16]));
    }
    uint32_t big = 0;
#pragma unroll
    for (int h = 0; h < QD_HALF; ++h) {
        const float f = __shfl_sync(0xFFFFFFFFu, r, h);
        float m = 0.f;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            o[d][h] *= f;
            m = fmaxf(m, fabsf(o[d][h]));
        }
        const uint32_t v = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
        if (lane == h) big = v;
    }
    named_bar(QB_HALF + half, 128);  // the sums have been read
    if (lane < QD_HALF) sm.part[quarter][h0 + lane] = __uint_as_float(big);
    named_bar(QB_HALF + half, 128);
    float up = 1.f;
    const int head = rank * QD_HEADS + h0 + lane;
    auto place = [&](int h) { return g.single ? (size_t)h * p.B + b : ((size_t)b * p.nsplit + s) * H + h; };
    if (lane < QD_HALF) {
        const float m = fmaxf(fmaxf(sm.part[0][h0 + lane], sm.part[1][h0 + lane]), fmaxf(sm.part[2][h0 + lane], sm.part[3][h0 + lane]));
        float inverse;
        up = w_row_scale(m, inverse);
        if (quarter == 0) {
            (g.single ? p.oscale : p.ws_oscale)[place(head)] = inverse;
            if (!g.single) p.ws_ml[place(head)] = make_float2(sm.m_ref[h0 + lane], total);
        }
    }
    // two lanes trade, so that each has a pair of neighbouring dims of every second block
    uint16_t* out = g.single ? p.olat : p.ws_o;
    const bool upper = lane & 1;
#pragma unroll
    for (int h = 0; h < QD_HALF; ++h) {
        const float f = __shfl_sync(0xFFFFFFFFu, up, h);
        uint16_t* row = out + place(rank * QD_HEADS + h0 + h) * LORA;
#pragma unroll
        for (int d = 0; d < 4; d += 2) {
            const float mine0 = o[d][h] * f, mine1 = o[d + 1][h] * f;
            const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? mine0 : mine1, 1);
            const int dim = 128 * (upper ? d + 1 : d) + 32 * quarter + (lane & ~1);
            *reinterpret_cast<uint32_t*>(row + w_dim_place(dim)) = upper ? pack_f16x2(other, mine1) : pack_f16x2(mine0, other);
        }
    }
}

// ---- the kernel ---------------------------------------------------------------------------

// A cluster a unit: split s of slot b; the CTAs take 48 heads each.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(QD_THREADS, 1)
    k3mla_quant_decode_kernel(const __grid_constant__ CUtensorMap tm_page, const QdParams p)
{
    extern __shared__ uint8_t smem_raw[];
    QdSmem& sm = *reinterpret_cast<QdSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int rank = (int)cluster_ctarank(), warp = (int)(threadIdx.x >> 5), unit = (int)(blockIdx.x >> 1);
    const int b = unit / p.nsplit, s = unit % p.nsplit;
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
    cluster_sync();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    griddep_wait();
    griddep_launch_dependents();
    const QdUnit g = qd_unit(p, b, s, s == 0 && rank == 0 && threadIdx.x == 0);
    if (s == 0 && g.n == 0 && threadIdx.x < QD_HEADS) p.oscale[(size_t)(rank * QD_HEADS + (int)threadIdx.x) * p.B + b] = 0.f;
    const int tiles = (g.npg + 1) / 2;
    if (tiles > 0) {
        if (warp < QD_SOFTMAX) qd_softmax(sm, p, g, b, s, rank, tbase, tiles);
        else if (warp == QW_LOAD) qd_produce(sm, tm_page, p, g, b, rank, tiles);
        else if (warp == QW_SCORE) qd_score(sm, p, tbase, tiles);
        else if (warp == QW_PV) qd_pv(sm, p, tbase, tiles);
        else if (warp == QW_AHEAD) qd_prefetch(sm, p, g, b, rank, tiles);
    }
    // After an abort a role leaves wherever it stands, with copies and MMAs under way: they land before the CTA gives its
    // shared memory and its TMEM back.
    if (aborted(sm)) drain_inflight();
    __syncwarp();
    tc_fence_before();
    cluster_sync();
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
    return k3mla_window_split_tokens(B, max_ctx, window, n_sink);
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
