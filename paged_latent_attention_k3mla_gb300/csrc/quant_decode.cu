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
__device__ __forceinline__ int64_t qd_block(const QdParams& p, int b, int lp)
{
    const int32_t id = p.table[(size_t)b * p.max_pages + lp];
    if (id >= 0 && id < p.n_pages) return (int64_t)id * p.n_layers + p.layer;
    if (id != -1 && p.dev_err) atomicOr(p.dev_err, (int)K3MLA_DEV_BAD_PAGE);
    return -1;
}

__device__ __forceinline__ bool qd_seen(const QdParams& p, int n, int t) { return t < n && (t < p.n_sink || t >= n - p.window); }

// A warp a head; lane l has the latents 16 l .. and the rope entries 2 l, 2 l + 1.
constexpr int QD_WARPS = 8;
__global__ void __launch_bounds__(32 * QD_WARPS) k3mla_quant_decode_kernel(const QdParams p)
{
    const int lane = (int)lane_id(), h = QD_WARPS * (int)blockIdx.x + (int)(threadIdx.x >> 5);
    const int s = (int)blockIdx.y, b = (int)blockIdx.z;
    griddep_wait();
    griddep_launch_dependents();
    const QdUnit g = qd_unit(p, b, s, s == 0 && threadIdx.x == 0 && blockIdx.x == 0);
    if (s == 0 && g.n == 0 && lane == 0) p.oscale[(size_t)h * p.B + b] = 0.f;
    if (g.npg == 0) return;
    float q[16], qr[2], o[16];
    {
        const uint16_t* src = p.q_abs + ((size_t)b * H + h) * ROW;
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            unpack8(reinterpret_cast<const uint4*>(src)[2 * lane + i], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[8 * i + e] = x[e], o[8 * i + e] = 0.f;
        }
        const uint32_t r = reinterpret_cast<const uint32_t*>(src + LORA)[lane];
        qr[0] = bf16lo_to_f32(r), qr[1] = bf16hi_to_f32(r);
    }
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < g.npg; ++i) {
        const int lp = qd_logical(g, i);
        const int64_t at = qd_block(p, b, lp);
        const uint8_t* block = p.slab + at * QPAGE;
        for (int line = 0; line < PAGE; ++line) {
            if (!qd_seen(p, g.n, PAGE * lp + line)) continue;
            float c[16], dot = 0.f, scale = 1.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) c[e] = 0.f;
            if (at >= 0) {
                const uint4 v = *reinterpret_cast<const uint4*>(block + line * QROW + 16 * lane);
                const uint32_t r = *reinterpret_cast<const uint32_t*>(block + line * QROW + LORA + 4 * lane);
                scale = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(block + QSCALES + 2 * line) << 16);
                float x[8];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    e4m3x8_to_f32(half ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y), x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        c[8 * half + e] = x[e];
                        dot = fmaf(q[8 * half + e], x[e], dot);
                    }
                }
                dot = fmaf(qr[0], bf16lo_to_f32(r), fmaf(qr[1], bf16hi_to_f32(r), dot));
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
            const float score = dot * scale * p.kscale;
            if (score > m) {
                const float a = ex2_approx(m - score);
                l *= a;
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= a;
                m = score;
            }
            const float w = ex2_approx(score - (m == -INFINITY ? 0.f : m));
            l += w;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(w * scale, c[e], o[e]);
        }
    }
    const float r = g.single ? 1.f / l : 1.f;
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        o[e] *= r;
        most = fmaxf(most, fabsf(o[e]));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, x));
    float inverse;
    const float up = w_row_scale(most, inverse);
    const size_t at = g.single ? (size_t)h * p.B + b : ((size_t)b * p.nsplit + s) * H + h;
    uint16_t* out = (g.single ? p.olat : p.ws_o) + at * LORA;
#pragma unroll
    for (int e = 0; e < 16; e += 2)
        *reinterpret_cast<uint32_t*>(out + w_dim_place(16 * lane + e)) = pack_f16x2(o[e] * up, o[e + 1] * up);
    if (lane == 0) {
        (g.single ? p.oscale : p.ws_oscale)[at] = inverse;
        if (!g.single) p.ws_ml[at] = make_float2(m, l);
    }
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

extern "C" int k3mla_quant_decode(const uint16_t* q_abs, const uint8_t* slab, int n_pages, int n_layers, int layer,
                                  const int32_t* block_table, int max_pages_per_slot, const int32_t* ctx_len,
                                  const uint16_t* w_kv_b, uint16_t scale_bf16, uint16_t* out, void* workspace,
                                  size_t ws_bytes, int B, int max_ctx, int window, int n_sink, int split_tokens,
                                  int32_t* dev_err, void* stream)
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
    if (B > 65535 || (long long)B * ns * H > 0x7FFFFFFFll || ns > 65535) {
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
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int rc = launch_pdl(k3mla_quant_decode_kernel, dim3(H / QD_WARPS, ns, B), dim3(32 * QD_WARPS), 0, st,
                        "k3mla_quant_decode_kernel", p);
    if (rc) return rc;
    TailArgs t;
    t.ctx_len = ctx_len, t.olat = p.olat, t.oscale = p.oscale, t.ws_o = p.ws_o, t.ws_oscale = p.ws_oscale, t.ws_ml = p.ws_ml;
    t.w_kv_b = w_kv_b, t.out = out, t.dev_err = dev_err, t.B = B, t.cap = p.cap, t.window = window, t.n_sink = n_sink;
    t.split_tokens = split_tokens, t.nsplit = ns;
    return launch_window_tail(t, st);
}
