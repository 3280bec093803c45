// norm_rope.cu -- what stands between the projections of an MLA layer and its cache: the norms of the
// queries (per head) and of the keys, the rotation by position, and the write of the cache rows.
//
// For token row r at position p (all in f32, one rounding to bf16 at the end):
//     q'[h]  = rot_p( q[h] * wq / sqrt(mean_192(q[h]^2) + eps) )     (the rotation turns entries 128..191)
//     c'     = c * wc / sqrt(mean_512(c^2) + eps)
//     k'     = rot_p( k * wk / sqrt(mean_64(k^2) + eps) )
//     cache row of p = c' | k'
// where a null weight leaves its norm out and rot_p turns pair i of the 64 rope entries -- (i, i + 32), or
// (2i, 2i + 1) when interleaved -- by the angle p * inv_freq[i].  A slot whose rows were compacted has two counts: the row
// goes to position p of its pages, and the angles go on from the positions its kept keys were rotated at
// (k3mla_norm_rope_append_at).
//
// The angle.  p * inv_freq[i] reaches 10^6 radians in long contexts, where an f32 product is off by
// 0.03; the product of an integer below 2^29 and an f32 is exact in f64, so the turn p * inv_freq / 2 pi
// is taken there, its nearest integer subtracted, and only the remainder in [-1/2, 1/2] is rounded to f32
// (an error of at most 2^-25 turns) for sincospi.  32 angles a row, computed once per CTA: 4 f64 operations
// each, against 18,432 query entries a row.
//
// Bound: HBM.  A row is 36,864 B of q in and out and 1,152 B of keys in and out at some 6 operations an
// entry.  A CTA takes one row's 32 heads, eight lanes a head, each lane three 16-byte vectors (the third
// one of the rope part: the lane holding the partner entries is lane ^ 4 of the eight, or the lane itself
// when interleaved), so that a head's norm is three shuffles and nothing is read twice.  Three CTAs a row
// rather than one keep the single row of a lone decode stream on more SMs.  The cache rows go to further
// CTAs of the grid, a warp each.
// Measured, device time in a graph of calls: 5,251 rows of 16 chunks 61.8 us (6.5 TB/s, 95 % of the copy rate); 64 rows of
// 64 slots 3.6 us, one row 2.9 us.  Called from Python, one row takes 22 us and 64 rows 26: the host's time.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace k3 {

constexpr int NR_WARPS = 8;
constexpr int NR_THREADS = 32 * NR_WARPS;
constexpr int NR_HEADS = 4 * NR_WARPS;       // heads of one CTA: eight lanes a head
constexpr int NR_QCTAS = H / NR_HEADS;       // CTAs of a row's queries
static_assert(NR_QCTAS * NR_HEADS == H, "whole heads");

struct NormRopeParams {
    const uint16_t* q;
    uint16_t* q_out;  // may be q
    const uint16_t *wq, *wc, *wk;  // null: that norm is left out
    uint16_t* slab;
    const int32_t *table, *pos0, *row_start;  // row_start null: row r is slot r's only one
    const int32_t* rope_pos0;                 // null: the angles' positions are pos0 as well
    const uint16_t *c_kv, *k_rope;
    int64_t c_stride, r_stride;
    const float* inv_freq;  // null: no rotation
    int32_t* dev_err;
    float eps;
    int interleaved, n_pages, n_layers, layer, max_pages, B, R;
    int q_ctas;  // NR_QCTAS * R, or 0 when the queries stay as they are
    int q_nope;  // 0: entries 0..127 of every head stay as they are (no norm, in place)
};

__device__ __forceinline__ void nr_unpack(const uint4& v, float (&x)[8])
{
    x[0] = bf16lo_to_f32(v.x), x[1] = bf16hi_to_f32(v.x);
    x[2] = bf16lo_to_f32(v.y), x[3] = bf16hi_to_f32(v.y);
    x[4] = bf16lo_to_f32(v.z), x[5] = bf16hi_to_f32(v.z);
    x[6] = bf16lo_to_f32(v.w), x[7] = bf16hi_to_f32(v.w);
}

__device__ __forceinline__ uint4 nr_pack(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ float nr_sumsq(const float (&x)[8])
{
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
    return s;
}

// x *= rs * w (eight weights from global memory; they stay in L1)
__device__ __forceinline__ void nr_scale(float (&x)[8], float rs, const uint16_t* w)
{
    float y[8];
    nr_unpack(*reinterpret_cast<const uint4*>(w), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= rs * y[e];
}

// The position that turns a row of slot b at position pos of its pages.
template <bool AT> __device__ __forceinline__ int64_t nr_rope_position(const NormRopeParams& p, int b, int64_t pos)
{
    return AT ? p.rope_pos0[b] + (pos - p.pos0[b]) : pos;
}

// (cos, sin) of the angle pos * inv_freq.
__device__ __forceinline__ float2 nr_angle(int64_t pos, float inv_freq)
{
    const double turns = (double)pos * (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    const float t = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * t, &s, &c);
    return make_float2(c, s);
}

// Rotate the eight rope entries 8 j .. 8 j + 7 of one vector, cs[i] the (cos, sin) of pair i.  Every lane
// of the warp takes part (the shuffle); lanes j and j ^ 4 of a group of eight hold partner vectors.
__device__ __forceinline__ void nr_rotate(float (&x)[8], int j, const float2* cs, bool interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float2 t = cs[4 * (j & 7) + m];
            const float a = x[2 * m], b = x[2 * m + 1];
            x[2 * m] = a * t.x - b * t.y;
            x[2 * m + 1] = a * t.y + b * t.x;
        }
    } else {
        const float sign = (j & 4) ? 1.f : -1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 t = cs[8 * (j & 3) + e];
            const float other = __shfl_xor_sync(0xFFFFFFFFu, x[e], 4);
            x[e] = x[e] * t.x + sign * other * t.y;
        }
    }
}

__device__ __forceinline__ void nr_query(const NormRopeParams& p, int r, int part, const float2* cs, bool norm,
                                         bool rot, const uint4 (&raw)[3])
{
    const int g = threadIdx.x >> 3, j = threadIdx.x & 7;
    float x[3][8];
#pragma unroll
    for (int k = 0; k < 3; ++k) nr_unpack(raw[k], x[k]);
    if (norm) {
        float s = nr_sumsq(x[0]) + nr_sumsq(x[1]) + nr_sumsq(x[2]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        const float rs = rsqrtf(s * (1.f / (float)QDIM) + p.eps);
#pragma unroll
        for (int k = 0; k < 3; ++k) nr_scale(x[k], rs, p.wq + 64 * k + 8 * j);
    }
    if (rot) nr_rotate(x[2], j, cs, p.interleaved != 0);
    uint4* dst = reinterpret_cast<uint4*>(p.q_out + ((size_t)r * H + part * NR_HEADS + g) * QDIM);
    if (p.q_nope) {
        dst[j] = nr_pack(x[0]);
        dst[j + 8] = nr_pack(x[1]);
    }
    dst[j + 16] = nr_pack(x[2]);
}

__device__ __forceinline__ void nr_key_row(const NormRopeParams& p, int r, int b, int64_t pos, const float2* cs)
{
    const int lane = (int)lane_id();
    const uint4* sc = reinterpret_cast<const uint4*>(p.c_kv + (int64_t)r * p.c_stride);
    const uint4* sk = reinterpret_cast<const uint4*>(p.k_rope + (int64_t)r * p.r_stride);
    float c0[8], c1[8], k[8];
    nr_unpack(sc[lane], c0);
    nr_unpack(sc[lane + 32], c1);
    nr_unpack(lane < 8 ? sk[lane] : make_uint4(0u, 0u, 0u, 0u), k);
    if (p.wc) {
        float s = nr_sumsq(c0) + nr_sumsq(c1);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        const float rs = rsqrtf(s * (1.f / (float)LORA) + p.eps);
        nr_scale(c0, rs, p.wc + 8 * lane);
        nr_scale(c1, rs, p.wc + 256 + 8 * lane);
    }
    if (p.wk) {
        float s = nr_sumsq(k);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);  // lanes 0..7 hold the key
        nr_scale(k, rsqrtf(s * (1.f / (float)ROPE) + p.eps), p.wk + 8 * (lane & 7));
    }
    if (p.inv_freq) nr_rotate(k, lane & 7, cs, p.interleaved != 0);
    const int64_t lp = pos / PAGE;
    const int32_t id = lp < p.max_pages ? p.table[(size_t)b * p.max_pages + lp] : -1;
    if (id < 0 || id >= p.n_pages) {
        if (lane == 0 && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_UNMAPPED);
        return;
    }
    const size_t row = ((size_t)id * (size_t)p.n_layers + (size_t)p.layer) * PAGE + (size_t)(pos % PAGE);
    uint4* dst = reinterpret_cast<uint4*>(p.slab + row * ROW);
    dst[lane] = nr_pack(c0);
    dst[lane + 32] = nr_pack(c1);
    if (lane < 8) dst[lane + 64] = nr_pack(k);
}

// Grid: q_ctas CTAs of a row's 32 heads each, then ceil(R / 8) CTAs of eight cache rows.  AT: with rope_pos0 (asking for
// it in the one kernel took 5,251 rows from 61.8 to 62.3 us).
template <bool AT>
__global__ void __launch_bounds__(NR_THREADS) k3mla_norm_rope_kernel(const NormRopeParams p)
{
    __shared__ float2 cs[NR_WARPS][ROPE / 2];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = (int)lane_id();
    if ((int)blockIdx.x < p.q_ctas) {
        const int r = blockIdx.x / NR_QCTAS, part = blockIdx.x % NR_QCTAS;
        const int g = threadIdx.x >> 3, j = threadIdx.x & 7;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)r * H + part * NR_HEADS + g) * QDIM);
        uint4 raw[3];
        raw[0] = raw[1] = make_uint4(0u, 0u, 0u, 0u);
        if (p.q_nope) {
            raw[0] = src[j];
            raw[1] = src[j + 8];
        }
        raw[2] = src[j + 16];
        int b;
        int64_t pos;
        if (!row_position(p.row_start, p.pos0, p.B, r, b, pos)) return;  // left as it is (uniform in the CTA)
        if (p.inv_freq) {
            if (warp == 0) cs[0][lane] = nr_angle(nr_rope_position<AT>(p, b, pos), p.inv_freq[lane]);
            __syncthreads();
        }
        nr_query(p, r, part, cs[0], p.wq != nullptr, p.inv_freq != nullptr, raw);
    } else {
        const int r = ((int)blockIdx.x - p.q_ctas) * NR_WARPS + warp;
        if (r >= p.R) return;
        int b;
        int64_t pos;
        if (!row_position(p.row_start, p.pos0, p.B, r, b, pos)) return;
        if (p.inv_freq) {
            cs[warp][lane] = nr_angle(nr_rope_position<AT>(p, b, pos), p.inv_freq[lane]);
            __syncwarp();
        }
        nr_key_row(p, r, b, pos, cs[warp]);
    }
}

}  // namespace k3

using namespace k3;

extern "C" int k3mla_norm_rope_append_at(const uint16_t* q, uint16_t* q_out, const uint16_t* q_weight, uint16_t* slab,
                                         int n_pages, int n_layers, int layer, const int32_t* block_table,
                                         int max_pages_per_slot, const int32_t* pos0, const int32_t* row_start,
                                         const int32_t* rope_pos0, const uint16_t* c_kv, int64_t c_stride,
                                         const uint16_t* c_weight, const uint16_t* k_rope, int64_t r_stride,
                                         const uint16_t* k_weight, float eps, const float* inv_freq, int interleaved, int B,
                                         int R, int32_t* dev_err, void* stream)
{
    if (B < 0 || R < 0 || n_pages <= 0 || n_layers <= 0 || layer < 0 || layer >= n_layers || max_pages_per_slot <= 0 ||
        c_stride < LORA || r_stride < ROPE || (c_stride & 7) || (r_stride & 7) || !(eps >= 0.f) || (!row_start && R != B)) {
        set_error("k3mla_norm_rope_append: invalid sizes, strides or eps");
        return K3MLA_E_INVALID;
    }
    if (B == 0 || R == 0) return K3MLA_OK;
    if ((long long)NR_QCTAS * R + (R + NR_WARPS - 1) / NR_WARPS > 0x7FFFFFFFll) {
        set_error("k3mla_norm_rope_append: too many rows");
        return K3MLA_E_INVALID;
    }
    if (!q || !q_out || !slab || !block_table || !pos0 || !c_kv || !k_rope || !aligned(q, 16) || !aligned(q_out, 16) ||
        !aligned(slab, 16) || !aligned(c_kv, 16) || !aligned(k_rope, 16) || !aligned(q_weight, 16) ||
        !aligned(c_weight, 16) || !aligned(k_weight, 16) || !aligned(inv_freq, 4)) {
        set_error("k3mla_norm_rope_append: null or misaligned pointer");
        return K3MLA_E_INVALID;
    }
    const uintptr_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(q_out);
    if (from != to && (from < to ? to - from : from - to) < (size_t)R * H * QDIM * 2) {
        set_error("k3mla_norm_rope_append: q_out overlaps q in part");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    NormRopeParams p;
    p.q = q, p.q_out = q_out, p.wq = q_weight, p.wc = c_weight, p.wk = k_weight;
    p.slab = slab, p.table = block_table, p.pos0 = pos0, p.row_start = row_start, p.rope_pos0 = rope_pos0;
    p.c_kv = c_kv, p.k_rope = k_rope, p.c_stride = c_stride, p.r_stride = r_stride;
    p.inv_freq = inv_freq, p.dev_err = dev_err, p.eps = eps, p.interleaved = interleaved;
    p.n_pages = n_pages, p.n_layers = n_layers, p.layer = layer, p.max_pages = max_pages_per_slot, p.B = B, p.R = R;
    const bool stays = q == q_out && !q_weight;  // entries 0..127 of every head
    p.q_nope = stays ? 0 : 1;
    p.q_ctas = stays && !inv_freq ? 0 : NR_QCTAS * R;
    return launch_pdl(rope_pos0 ? k3mla_norm_rope_kernel<true> : k3mla_norm_rope_kernel<false>,
                      dim3(p.q_ctas + (R + NR_WARPS - 1) / NR_WARPS), dim3(NR_THREADS), 0,
                      reinterpret_cast<cudaStream_t>(stream), "k3mla_norm_rope_kernel", p);
}

extern "C" int k3mla_norm_rope_append(const uint16_t* q, uint16_t* q_out, const uint16_t* q_weight, uint16_t* slab,
                                      int n_pages, int n_layers, int layer, const int32_t* block_table,
                                      int max_pages_per_slot, const int32_t* pos0, const int32_t* row_start,
                                      const uint16_t* c_kv, int64_t c_stride, const uint16_t* c_weight,
                                      const uint16_t* k_rope, int64_t r_stride, const uint16_t* k_weight, float eps,
                                      const float* inv_freq, int interleaved, int B, int R, int32_t* dev_err,
                                      void* stream)
{
    return k3mla_norm_rope_append_at(q, q_out, q_weight, slab, n_pages, n_layers, layer, block_table, max_pages_per_slot,
                                     pos0, row_start, nullptr, c_kv, c_stride, c_weight, k_rope, r_stride, k_weight, eps,
                                     inv_freq, interleaved, B, R, dev_err, stream);
}
