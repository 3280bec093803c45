// quant_pages.cu -- whole pages of the bf16 cache into the 8-bit one (quant.cuh), and back.
//
// In: per row the largest latent, the row's power of two, 512 codes and 64 rope entries in its units.  Back: code and rope
// entry times the power of two, exact in bf16.  Both are one pass over the rows at a handful of operations an entry; bound:
// HBM, 73,728 + 41,088 B a page and layer.  A warp takes a row (8 latents a lane, twice: the row's maximum is one warp
// reduction) and asks for four rows' data before it turns the first, 4.6 KB under way a warp.
// Measured, in a graph of calls: 64 pages x 24 layers in 30.1 us (176 MB, 5.9 TB/s, 0.86 of the copy rate; 27.5 us by itself),
// 63 back 28.6 us (6.1 TB/s; 25 us by itself), one page 2.3 us; from Python some 15 us of the host's.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace k3 {

constexpr int QP_THREADS = 256;
constexpr int QP_ROWS = 4;                              // rows of a warp
constexpr int QP_CTA = QP_ROWS * QP_THREADS / 32;       // ... of a CTA: half a page
static_assert(PAGE % QP_CTA == 0, "a CTA's rows lie in one page");

struct QuantPagesParams {
    uint16_t* slab;
    uint8_t* quant;
    const int32_t *src_ids, *dst_ids;
    int32_t* dev_err;
    int n_pages, quant_pages, n_layers, layer0;
};

// The larger of m and x's bf16 magnitudes, NaN and infinities aside; with LATENT these become NaN.
template <bool LATENT> __device__ __forceinline__ uint32_t qp_finite(uint32_t m, uint32_t& x)
{
    const uint32_t lo = x & 0x7FFFu, hi = (x >> 16) & 0x7FFFu;
    if (lo < 0x7F80u) m = max(m, lo);
    else if (LATENT) x |= 0x7Fu;
    if (hi < 0x7F80u) m = max(m, hi);
    else if (LATENT) x |= 0x7F0000u;
    return m;
}

// quant_store_row for a row of bf16: lane l has the latents 8 l .. and 256 + 8 l .. and the rope entries 2 l, 2 l + 1.  The
// same results in half the instructions (what bounds this direction): maxima of two magnitudes at a time, products in pairs.
__device__ __forceinline__ void qp_store_row(uint8_t* block, int line, const uint4& c0, const uint4& c1, uint32_t k)
{
    const int lane = (int)lane_id();
    uint32_t x[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    constexpr uint32_t A = 0x7FFF7FFFu;
    uint32_t m = x[0] & A, r = k & A;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_u16x2(m, x[i] & A);
    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
    r = __reduce_max_sync(0xFFFFFFFFu, max(r & 0xFFFFu, r >> 16));
    if (m >= 0x7F80u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = qp_finite<true>(m, x[i]);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
    }
    if (r >= 0x7F80u) r = __reduce_max_sync(0xFFFFFFFFu, qp_finite<false>(0u, k));
    const int n = quant_exponent(m << 16, r << 16);
    const float d = __uint_as_float((uint32_t)(127 - n) << 23);
    const uint64_t down = f32x2(d, d);
    auto two = [&](uint32_t w, float& a, float& b) { f32x2_parts(mul_f32x2(f32x2(bf16lo_to_f32(w), bf16hi_to_f32(w)), down), a, b); };
    float a, b;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        two(x[i], a, b);
        c[i] = pack_e4m3x2(a, b);
    }
    uint8_t* row = block + line * QROW;
    *reinterpret_cast<uint2*>(row + 8 * lane) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    *reinterpret_cast<uint2*>(row + 256 + 8 * lane) = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
    two(k, a, b);
    *reinterpret_cast<uint32_t*>(row + LORA + 4 * lane) = pack_bf16x2(a, b);
    if (lane == 0) *reinterpret_cast<uint16_t*>(block + QSCALES + 2 * line) = (uint16_t)((n + 127) << 7);
}

// grid (PAGE / QP_CTA, layers, pairs).  BACK: from the 8-bit cache.
template <bool BACK>
__global__ void __launch_bounds__(QP_THREADS) k3mla_quant_pages_kernel(const QuantPagesParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = (int)lane_id(), line0 = (int)blockIdx.x * QP_CTA + QP_ROWS * ((int)threadIdx.x >> 5);
    const int layer = p.layer0 + (int)blockIdx.y;
    const int32_t s = p.src_ids[blockIdx.z], d = p.dst_ids[blockIdx.z];
    if (s < 0 || s >= (BACK ? p.quant_pages : p.n_pages) || d < 0 || d >= (BACK ? p.n_pages : p.quant_pages)) {
        if (blockIdx.x == 0 && layer == 0 && threadIdx.x == 0 && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_BAD_PAGE);
        return;
    }
    uint16_t* rows = p.slab + (((size_t)(BACK ? d : s) * p.n_layers + layer) * PAGE + line0) * ROW;
    uint8_t* block = p.quant + ((size_t)(BACK ? s : d) * p.n_layers + layer) * QPAGE;
    if constexpr (BACK) {
        uint2 v[QP_ROWS][2];
        uint4 k[QP_ROWS];
        float scale[QP_ROWS];
#pragma unroll
        for (int i = 0; i < QP_ROWS; ++i) {
            const uint8_t* row = block + (line0 + i) * QROW;
            v[i][0] = *reinterpret_cast<const uint2*>(row + 8 * lane);
            v[i][1] = *reinterpret_cast<const uint2*>(row + 256 + 8 * lane);
            k[i] = lane < 8 ? *reinterpret_cast<const uint4*>(row + LORA + 16 * lane) : make_uint4(0u, 0u, 0u, 0u);
            scale[i] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(block + QSCALES + 2 * (line0 + i)) << 16);
        }
#pragma unroll
        for (int i = 0; i < QP_ROWS; ++i) {
            uint4* dst = reinterpret_cast<uint4*>(rows + (size_t)i * ROW);
            float x[8];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                e4m3x8_to_f32(v[i][half], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= scale[i];
                dst[32 * half + lane] = pack8(x);
            }
            if (lane < 8) {
                unpack8(k[i], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= scale[i];
                dst[64 + lane] = pack8(x);
            }
        }
    } else {
        uint4 v[QP_ROWS][2];
        uint32_t k[QP_ROWS];
#pragma unroll
        for (int i = 0; i < QP_ROWS; ++i) {
            const uint4* src = reinterpret_cast<const uint4*>(rows + (size_t)i * ROW);
            v[i][0] = src[lane];
            v[i][1] = src[32 + lane];
            k[i] = reinterpret_cast<const uint32_t*>(src + 64)[lane];
        }
#pragma unroll
        for (int i = 0; i < QP_ROWS; ++i) qp_store_row(block, line0 + i, v[i][0], v[i][1], k[i]);
    }
}

static int quant_pages(const char* who, bool back, uint16_t* slab, int n_pages, uint8_t* quant, int quant_n_pages, int n_layers,
                       const int32_t* src_ids, const int32_t* dst_ids, int n, int32_t* dev_err, void* stream)
{
    if (n < 0 || n_layers <= 0 || n_pages <= 0 || quant_n_pages <= 0 || n > 65535) {
        set_error("%s: invalid sizes (n must be in [0, 65535])", who);
        return K3MLA_E_INVALID;
    }
    if (n == 0) return K3MLA_OK;
    if (!slab || !quant || !src_ids || !dst_ids || !aligned(slab, 16) || !aligned(quant, 16)) {
        set_error("%s: null or misaligned pointer", who);
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    QuantPagesParams p;
    p.slab = slab, p.quant = quant, p.src_ids = src_ids, p.dst_ids = dst_ids, p.dev_err = dev_err;
    p.n_pages = n_pages, p.quant_pages = quant_n_pages, p.n_layers = n_layers;
    constexpr int MOST = 65535;  // a grid's extent in y
    for (p.layer0 = 0; p.layer0 < n_layers; p.layer0 += MOST) {
        const int rc = launch_pdl(back ? k3mla_quant_pages_kernel<true> : k3mla_quant_pages_kernel<false>,
                                  dim3(PAGE / QP_CTA, n_layers - p.layer0 < MOST ? n_layers - p.layer0 : MOST, n),
                                  dim3(QP_THREADS), 0, reinterpret_cast<cudaStream_t>(stream), "k3mla_quant_pages_kernel", p);
        if (rc) return rc;
    }
    return K3MLA_OK;
}

}  // namespace k3

using namespace k3;

extern "C" int k3mla_quant_write_pages(uint8_t* dst_slab, int dst_n_pages, const uint16_t* src_slab, int src_n_pages,
                                       int n_layers, const int32_t* src_ids, const int32_t* dst_ids, int n, int32_t* dev_err,
                                       void* stream)
{
    return quant_pages("k3mla_quant_write_pages", false, const_cast<uint16_t*>(src_slab), src_n_pages, dst_slab, dst_n_pages,
                       n_layers, src_ids, dst_ids, n, dev_err, stream);
}

extern "C" int k3mla_quant_read_pages(uint16_t* dst_slab, int dst_n_pages, const uint8_t* src_slab, int src_n_pages,
                                      int n_layers, const int32_t* src_ids, const int32_t* dst_ids, int n, int32_t* dev_err,
                                      void* stream)
{
    return quant_pages("k3mla_quant_read_pages", true, dst_slab, dst_n_pages, const_cast<uint8_t*>(src_slab), src_n_pages,
                       n_layers, src_ids, dst_ids, n, dev_err, stream);
}
