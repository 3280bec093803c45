// pages.cu -- whole-page copies between page-first slabs.
//
// pegainfer PR #869, "K3: paged latent MLA KV + absorbed decode", M1 commit: a
// prefilled sequence is adopted into a decode slot by copying its pages whole.
// In the page-first slab [page][layer][64][576] bf16 a page is one contiguous
// block of n_layers * 64 * 576 elements (every layer's rows of those 64 tokens),
// so adopting a page, or un-sharing a page that two slots map (copy on write),
// is one contiguous block copy.  The copy is HBM-bound (read + write of
// n_layers * 73,728 bytes per page); each CTA moves 16-byte vectors, eight in
// flight per thread, over one page of one (src, dst) pair.
//
// Row compaction (k3mla_compact_rows): the kept tokens of a slot move to the front of its pages, in
// place.  Entry i of a slot's ascending list of kept positions goes to position i, and i <= keep[i], so
// a walk over i in ascending order never writes a row that a later step still has to read: rows up to i
// are written only after entries up to i have been read.  Within one column of the rows (128 or 64 bytes
// of the 1,152) this order is one CTA's: it reads a step's rows, waits at a barrier, and writes them
// while the next ones are on their way -- reading ahead is always safe.  The columns, the layers and the
// slots are independent, so even a lone slot of 24 layers fills the GPU.  Bound: HBM, 2,304 bytes a
// moved row and layer; rows that stay in place are neither read nor written.
// Measured: 16 slots x 24 layers, 827 MB, 147 us (5.6 TB/s, 83 % of the copy rate); one slot, 1,028 rows kept, 57 MB, 15.9 us:
// eight steps of 144 rows behind each other, some 1.7 us each, where the step's 8 MB would take 1.2 at the copy rate.  A
// step asks for its data one step ahead and ends at a barrier; in a profile a warp spends 29 % of its cycles on loads and
// 12 % at the barrier, the schedulers issue in half of the cycles (the addresses of 16-byte pieces), and 432 CTAs are two
// on some SMs and three on others.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace k3 {

constexpr int CP_THREADS = 256;
constexpr int CP_VEC = 8;  // 16-byte vectors in flight per thread

// grid (chunks of a page, pairs); block CP_THREADS.  A pair with an id outside its slab is skipped
// and flagged (K3MLA_DEV_BAD_PAGE, once per pair by the first CTA of the pair).
__global__ void __launch_bounds__(CP_THREADS) k3mla_copy_pages_kernel(uint16_t* __restrict__ dst_slab, int dst_n_pages,
                                                                      const uint16_t* __restrict__ src_slab,
                                                                      int src_n_pages, const int32_t* __restrict__ src_ids,
                                                                      const int32_t* __restrict__ dst_ids,
                                                                      size_t page_vecs, int32_t* dev_err)
{
    griddep_wait();
    griddep_launch_dependents();
    const int pair = blockIdx.y;
    const int32_t s = src_ids[pair], d = dst_ids[pair];
    if (s < 0 || s >= src_n_pages || d < 0 || d >= dst_n_pages) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && dev_err) atomicOr(dev_err, (int)K3MLA_DEV_BAD_PAGE);
        return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(src_slab) + (size_t)s * page_vecs;
    uint4* dst = reinterpret_cast<uint4*>(dst_slab) + (size_t)d * page_vecs;
    const size_t step = (size_t)gridDim.x * CP_THREADS * CP_VEC;
    for (size_t base = (size_t)blockIdx.x * CP_THREADS * CP_VEC + threadIdx.x; base < page_vecs; base += step) {
        uint4 v[CP_VEC];
#pragma unroll
        for (int k = 0; k < CP_VEC; ++k) {
            const size_t i = base + (size_t)k * CP_THREADS;
            if (i < page_vecs) v[k] = src[i];
        }
#pragma unroll
        for (int k = 0; k < CP_VEC; ++k) {
            const size_t i = base + (size_t)k * CP_THREADS;
            if (i < page_vecs) dst[i] = v[k];
        }
    }
}

// COLS columns of a row, a CTA of THREADS each; UNROLL rows a thread and step.
template <int COLS, int UNROLL, int THREADS> struct Compact {
    static constexpr int VECS = ROW * 2 / (16 * COLS);     // 16-byte vectors of a row's column
    static constexpr int GROUP = THREADS / VECS;        // rows that the CTA's threads cover at once
    static constexpr int ROWS = GROUP * UNROLL;            // rows a step
    static_assert(COLS * VECS * 16 == ROW * 2 && GROUP * VECS == THREADS, "whole columns and rows");
};

struct CompactParams {
    uint16_t* slab;
    const int32_t *table, *keep, *keep_start;
    int64_t keep_stride;  // entries from a layer's list to the next layer's, 0: one list for all
    int32_t* dev_err;
    int n_pages, n_layers, max_pages, n_keep, layer0, slot0;
};

// One thread's part of a step: UNROLL rows, GROUP apart, of one 16-byte piece each.
template <int UNROLL> struct CompactRows {
    int64_t src[UNROLL], dst[UNROLL];  // rows of the slab; dst -1: nothing to move, src -1: zeros
};

// grid (columns, layers, slots); block THREADS.
template <int COLS, int UNROLL, int THREADS>
__global__ void __launch_bounds__(THREADS) k3mla_compact_rows_kernel(const CompactParams p)
{
    using C = Compact<COLS, UNROLL, THREADS>;
    griddep_wait();
    griddep_launch_dependents();
    const int b = p.slot0 + (int)blockIdx.z, layer = p.layer0 + (int)blockIdx.y;
    const int first = max(0, p.keep_start[b]);
    const int n = min(p.n_keep, p.keep_start[b + 1]) - first;
    const int32_t* keep = p.keep + (int64_t)layer * p.keep_stride + first;
    const int32_t* table = p.table + (int64_t)b * p.max_pages;
    const int at = (int)threadIdx.x / C::VECS, vec = (int)blockIdx.x * C::VECS + (int)threadIdx.x % C::VECS;
    if (n <= 0) return;

    // A row takes three loads in a chain (its old position, the two pages, its data), so three steps are under way:
    // the positions of step k + 3, the pages of step k + 2 and the data of step k + 1 are fetched while step k is
    // written.
    auto positions = [&](int i0, int (&t)[UNROLL]) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int i = i0 + at + u * C::GROUP;
            t[u] = i < n ? keep[i] : i;
        }
    };
    auto places = [&](int i0, const int (&t)[UNROLL], CompactRows<UNROLL>& r) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int i = i0 + at + u * C::GROUP;
            r.src[u] = r.dst[u] = -1;
            if (t[u] == i) continue;  // the row stays where it is
            const int32_t d = i / PAGE < p.max_pages ? table[i / PAGE] : -1;
            const bool inside = t[u] >= 0 && t[u] / PAGE < p.max_pages;
            const int32_t s = inside ? table[t[u] / PAGE] : -1;
            if (d >= 0 && d < p.n_pages) r.dst[u] = ((int64_t)d * p.n_layers + layer) * PAGE + i % PAGE;
            if (s >= 0 && s < p.n_pages) r.src[u] = ((int64_t)s * p.n_layers + layer) * PAGE + t[u] % PAGE;
            const int bits = (r.dst[u] < 0 ? (int)K3MLA_DEV_UNMAPPED : 0) | (inside ? 0 : (int)K3MLA_DEV_CTX) |
                             (s < -1 || s >= p.n_pages ? (int)K3MLA_DEV_BAD_PAGE : 0);
            if (bits && p.dev_err) atomicOr(p.dev_err, bits);
        }
    };
    auto load = [&](const CompactRows<UNROLL>& r, uint4 (&v)[UNROLL]) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            v[u] = r.dst[u] >= 0 && r.src[u] >= 0 ? reinterpret_cast<const uint4*>(p.slab + r.src[u] * ROW)[vec]
                                                  : make_uint4(0u, 0u, 0u, 0u);
    };
    int t[UNROLL];
    CompactRows<UNROLL> now, next;
    uint4 v[UNROLL];
    positions(0, t);
    places(0, t, now);
    positions(C::ROWS, t);
    load(now, v);
    places(C::ROWS, t, next);
    positions(2 * C::ROWS, t);
    for (int i = 0; i < n; i += C::ROWS) {
        uint4 w[UNROLL];
        CompactRows<UNROLL> later;
        load(next, w);
        places(i + 2 * C::ROWS, t, later);
        positions(i + 3 * C::ROWS, t);
        __syncthreads();  // every thread holds its rows of this step: what they leave may be overwritten
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (now.dst[u] >= 0) reinterpret_cast<uint4*>(p.slab + now.dst[u] * ROW)[vec] = v[u];
            v[u] = w[u];
        }
        now = next;
        next = later;
    }
}

}  // namespace k3

using namespace k3;

extern "C" int k3mla_copy_pages(uint16_t* dst_slab, int dst_n_pages, const uint16_t* src_slab, int src_n_pages,
                                int n_layers, const int32_t* src_ids, const int32_t* dst_ids, int n,
                                int32_t* dev_err, void* stream)
{
    if (n < 0 || n_layers <= 0 || dst_n_pages <= 0 || src_n_pages <= 0 || n > 65535) {
        set_error("k3mla_copy_pages: invalid sizes (n must be in [0, 65535])");
        return K3MLA_E_INVALID;
    }
    if (n == 0) return K3MLA_OK;
    if (!dst_slab || !src_slab || !src_ids || !dst_ids || !aligned(dst_slab, 16) || !aligned(src_slab, 16)) {
        set_error("k3mla_copy_pages: null or misaligned pointer");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    const size_t page_vecs = (size_t)n_layers * PAGE * ROW * 2 / 16;  // 4,608 16-byte vectors per layer
    const size_t per_cta = (size_t)CP_THREADS * CP_VEC;
    size_t chunks = (page_vecs + per_cta - 1) / per_cta;
    if (chunks > 1024) chunks = 1024;  // a grid-stride loop covers the rest of a very deep page
    return launch_pdl(k3mla_copy_pages_kernel, dim3((unsigned)chunks, (unsigned)n), dim3(CP_THREADS), 0,
                      reinterpret_cast<cudaStream_t>(stream), "k3mla_copy_pages_kernel", dst_slab, dst_n_pages,
                      src_slab, src_n_pages, src_ids, dst_ids, page_vecs, dev_err);
}

extern "C" int k3mla_compact_rows(uint16_t* slab, int n_pages, int n_layers, const int32_t* block_table,
                                  int max_pages_per_slot, const int32_t* keep, int64_t keep_layer_stride, int n_keep,
                                  const int32_t* keep_start, int B, int32_t* dev_err, void* stream)
{
    if (B < 0 || n_pages <= 0 || n_layers <= 0 || max_pages_per_slot <= 0 || n_keep < 0 ||
        n_keep > 0x3FFFFFFF ||  // (a step's positions are counted a few steps past the list)
        (keep_layer_stride != 0 && keep_layer_stride < n_keep)) {
        set_error("k3mla_compact_rows: invalid sizes");
        return K3MLA_E_INVALID;
    }
    if (B == 0 || n_keep == 0) return K3MLA_OK;
    if (!slab || !block_table || !keep || !keep_start || !aligned(slab, 16)) {
        set_error("k3mla_compact_rows: null or misaligned pointer");
        return K3MLA_E_INVALID;
    }
    if (!device_ok()) return K3MLA_E_DEVICE;
    CompactParams p;
    p.slab = slab, p.table = block_table, p.keep = keep, p.keep_start = keep_start, p.keep_stride = keep_layer_stride;
    p.dev_err = dev_err, p.n_pages = n_pages, p.n_layers = n_layers, p.max_pages = max_pages_per_slot, p.n_keep = n_keep;
    constexpr int MOST = 65535;  // a grid's extent in y and z
    for (p.slot0 = 0; p.slot0 < B; p.slot0 += MOST)
        for (p.layer0 = 0; p.layer0 < n_layers; p.layer0 += MOST) {
            const int ny = n_layers - p.layer0 < MOST ? n_layers - p.layer0 : MOST;
            const int nz = B - p.slot0 < MOST ? B - p.slot0 : MOST;
            // Few columns in all (less than eight CTAs of 128 bytes an SM): half as wide ones and two rows a thread, since
            // the steps' latency is what counts -- one slot of 24 layers 15.9 us against 24.8.  Else whole lines and one
            // row a thread, for more CTAs an SM -- 16 slots 147 us against 164 (eight CTAs of 256 threads fill an SM; of 288 155 us).
            int dev = 0, sms = 152;
            if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            const bool few = 9ll * ny * nz < 8ll * sms;
            const int rc = launch_pdl(few ? k3mla_compact_rows_kernel<18, 2, 288> : k3mla_compact_rows_kernel<9, 1, 256>,
                                      dim3(few ? 18 : 9, ny, nz), dim3(few ? 288 : 256), 0, reinterpret_cast<cudaStream_t>(stream),
                                      "k3mla_compact_rows_kernel", p);
            if (rc) return rc;
        }
    return K3MLA_OK;
}
