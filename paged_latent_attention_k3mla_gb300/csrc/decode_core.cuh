// decode_core.cuh -- what the split kernel (decode.cu) and the windowed kernel (window.cu) share: the page
// tiles of their two rings, the bounded waits, and the issue of the two contractions.  Both run as
// clusters of two CTAs, the score CTA (rank 0) and the PV CTA (rank 1); S is the shared-memory layout of
// the kernel at hand, with an abort_flag and the wait_ns limit of its waits.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace k3 {

constexpr int CHUNK = PAGE * 128;              // 8192 B per chunk of a page slot
constexpr int HALF = 32;                       // PV CTA: tokens per half-page box
constexpr int THIRD = 3 * 8192;  // score CTA: a third of a page (3 chunks), one TMA box
constexpr int SLOT1 = 8 * HALF * 128;          // 32768 B: [8 chunks][32 rows][128 B], chunks 0..7 only
constexpr int HCHUNK = HALF * 128;             // 4096 B per chunk of a half-page slot
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 0;                  // score CTA: S^T buffers r = 0..2 at 64 r
constexpr uint32_t Q_COL = 192;                // score CTA: Q, 288 columns (576 bf16)
constexpr float TAU = 16.0f;                   // max growth (natural log) before a rescale: p~ <= e^16,
                                               // l <= n e^16 stays far inside f32 for any context here
constexpr uint64_t WAIT_NS = 1000000000ull;    // bounded waits: 1 s
constexpr uint32_t IDESC_S = make_idesc_bf16(128, PAGE, 0, 0);  // S^T page = Q . C^T
constexpr uint32_t IDESC_PV = make_idesc_bf16(128, 256, 0, 1);  // O half = P . C (B MN-major)

template <class S> __device__ __forceinline__ bool aborted(const S& sm)
{
    return *reinterpret_cast<const volatile int32_t*>(&sm.abort_flag) != 0;
}

// Bounded mbarrier wait, slow path: gives up after the CTA's wait limit or when this CTA aborted.
template <class S>
__device__ __noinline__ bool wait_bar_slow(uint64_t* bar, uint32_t parity, S& sm, int32_t* dev_err,
                                           bool cluster_scope)
{
    const uint32_t a = smem_u32(bar);
    if (cluster_scope ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (cluster_scope ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity)) return true;
        if ((n & 127u) == 0) {
            if (aborted(sm)) return false;
            if (globaltimer() - t0 > sm.wait_ns) {
                *reinterpret_cast<volatile int32_t*>(&sm.abort_flag) = 1;
                if (dev_err) atomicOr(dev_err, (int)K3MLA_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

// Bounded mbarrier wait: an inline non-blocking test first (most waits are already
// satisfied when they are reached), then the suspending slow path.
template <class S>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, S& sm, int32_t* dev_err,
                                         bool cluster_scope = false)
{
    const uint32_t a = smem_u32(bar);
    if (cluster_scope ? mbar_test_wait_cluster(a, parity) : mbar_test_wait(a, parity)) return true;
    return wait_bar_slow(bar, parity, sm, dev_err, cluster_scope);
}

// Bounded wait until a shared counter of this CTA reaches `target` (written by another thread of
// the CTA with a plain store); false when this CTA aborted or the wait timed out.
template <class S>
__device__ __noinline__ bool wait_count(const int32_t* counter, int32_t target, S& sm, int32_t* dev_err)
{
    const volatile int32_t* v = counter;
    if (*v >= target) return true;
    const uint64_t t0 = globaltimer();
    while (*v < target) {
        if (aborted(sm)) return false;
        if (globaltimer() - t0 > sm.wait_ns) {
            *reinterpret_cast<volatile int32_t*>(&sm.abort_flag) = 1;
            if (dev_err) atomicOr(dev_err, (int)K3MLA_DEV_TIMEOUT);
            return false;
        }
        __nanosleep(32);
    }
    return true;
}

// After an abort: let this thread's in-flight TMA copies / MMAs land (bounded, ~2 ms).
static __device__ __noinline__ void drain_inflight()
{
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
}

// Score CTA: the 12 K steps of third t (chunks 3t .. 3t+2, at third_addr) of the same product.
__device__ __forceinline__ void issue_score_third(uint32_t tbase, uint32_t d_col, uint32_t third_addr, int t)
{
    uint64_t bd = make_sdesc(third_addr, 16, 1024);
    uint32_t a = tbase + Q_COL + 96u * (uint32_t)t;
    const uint32_t d = tbase + d_col;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) umma_ts(d, a + 8u * ks, bd + 2u * ks, IDESC_S, (t | c | ks) != 0);
        a += 32u;
        bd += (uint64_t)(CHUNK >> 4);
    }
}

// PV CTA: O[128 rows = heads (rows 96.. unused) x 512 dims] (+)= P . C over one 64-token page held as
// two half-page slots ([8 chunks][32 rows][128 B] each).  A = P, K-major (the P buffer's rows are heads,
// 64 tokens each; rows 96..127 read whatever follows the buffer in this CTA's shared memory and only
// land in TMEM lanes nobody reads); B = C, MN-major (dims contiguous).  Two N = 256 halves of the dims
// x 4 K-steps of 16 tokens.
// Half hh of the page (tokens 32 hh .. 32 hh + 31, held in one slot): 4 MMAs.
__device__ __forceinline__ void issue_pv_half(uint32_t tbase, uint32_t half_addr, uint32_t pt_addr, int hh,
                                              bool accumulate_first)
{
    const uint64_t a0 = make_sdesc(pt_addr, 16, 1024);
    const uint64_t b0 = make_sdesc(half_addr, HCHUNK, 1024);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const uint64_t ad = a0 + (uint64_t)((uint32_t)((2 * hh + ks) * 32) >> 4);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const uint64_t bd = b0 + (uint64_t)((uint32_t)(4 * n * HCHUNK + ks * 2048) >> 4);
            umma_ss(tbase + 256u * n, ad, bd, IDESC_PV, (accumulate_first || hh > 0 || ks > 0) ? 1u : 0u);
        }
    }
}

// Byte offset in a P^T buffer of the 16-byte chunk with tokens 8j .. 8j+7 of head h.
__device__ __forceinline__ uint32_t pt_chunk_off(int h, int j) { return (uint32_t)(h * 128 + ((j ^ (h & 7)) << 4)); }

static void set_smem_attr(const void* fn, size_t bytes, bool* done)
{
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
}

}  // namespace k3
