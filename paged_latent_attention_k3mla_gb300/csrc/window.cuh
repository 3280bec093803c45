// window.cuh -- what the kernels that attend by lists of pages share (window.cu, quant_decode.cu): the list of the pages that a
// row sees, the splits of it and their records, and what turns those into outputs.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "common.cuh"

namespace k3 {

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

inline size_t w_up(size_t x) { return (x + 255) & ~size_t(255); }

// The most pages a slot of at most cap tokens can see, and the splits that makes.
inline long long w_max_pages(int cap, int window, int n_sink)
{
    const long long all = ((long long)cap + PAGE - 1) / PAGE;
    const long long sink = ((long long)std::min(n_sink, cap) + PAGE - 1) / PAGE;
    const long long win = ((long long)std::min(window, cap) + PAGE - 2) / PAGE + 1;
    return std::min(all, sink + win);
}

inline int w_nsplit(int cap, int window, int n_sink, int split_tokens)
{
    return launch_nsplit((int)std::min<long long>(w_max_pages(cap, window, n_sink) * PAGE, 0x7FFFFF00), split_tokens);
}

struct WinWs {
    size_t olat, scale, o, oscale, ml, total;
};
inline WinWs w_layout(long long rows, int nsplit)
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

inline int sm_count()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

inline bool w_scale(uint16_t bits, float* kscale)
{
    uint32_t u = (uint32_t)bits << 16;
    float f;
    std::memcpy(&f, &u, 4);
    if (!(f > 0.f) || (bits & 0x7F80) == 0x7F80) return false;
    const double k = (double)f * 1.4426950408889634;
    *kscale = (float)k;
    return k <= 3.4028234663852886e38;  // (an infinite factor would make NaN of every score of 0)
}

// When the last of S units of a us, then O units of b us, has ended, each taken by the first free of `workers`.
inline double units_span(long long S, double a, long long O, double b, long long workers)
{
    const long long q = S / workers, r = S % workers;  // r workers are free after q + 1 rounds, the others after q
    const double early = q * a, late = r ? early + a : early;
    auto ends = [&](double base) {
        long long lo = 0, hi = O;
        while (lo < hi) {
            const long long k = (lo + hi) / 2;
            const double t = base + k * b;
            long long room = (workers - r) * (long long)((t - early) / b + 1e-9);
            if (r && t >= late) room += r * (long long)((t - late) / b + 1e-9);
            if (room >= O) hi = k;
            else lo = k + 1;
        }
        return base + lo * b;
    };
    return std::max(late, std::min(ends(early), ends(late)));
}

// A unit's pages take up to 0.85 us each, and its write-out waits for all of them within WAIT_NS: half of that is allowed.
constexpr long long W_UNIT_PAGES = 1 << 19;

inline bool w_unit_fits(const char* who, long long pages)
{
    if (pages <= W_UNIT_PAGES) return true;
    set_error("%s: %lld pages in one unit of work, more than %lld", who, pages, W_UNIT_PAGES);
    return false;
}

// Splits -> o_lat -> W_UV expansion of one token row per slot (window.cu), behind a kernel that left either a slot's o_lat
// (all it sees in one split) or its splits' records.  Two kernels on the stream, or one.
struct TailArgs {
    const int32_t* ctx_len;   // [B]; no output of the kernels of the call
    uint16_t* olat;           // [96][B][512] f16: o_lat times a power of two per row, each 64 dims in the write-out's order
    float* oscale;            // [96][B]: what undoes it; 0 for rows that see nothing
    uint16_t* ws_o;           // [B][nsplit][96][512] f16, the same order: a split's O (null for nsplit == 1) ...
    float* ws_oscale;         // [B][nsplit][96]: ... what undoes its power of two
    float2* ws_ml;            // [B][nsplit][96]: reference max (in log2 units), sum of exp
    const uint16_t* w_kv_b;
    uint16_t* out;            // [B][96][128]
    int32_t* dev_err;
    int B, cap, window, n_sink, split_tokens, nsplit;
};
int launch_window_tail(const TailArgs& t, cudaStream_t st);

// The write-out's order of 64 dims: 8 n + 2 j + e lies at 16 j + 2 n + e.
__host__ __device__ inline int w_dim_place(int d) { return (d & ~63) | ((d & 6) << 3) | ((d & 56) >> 2) | (d & 1); }

}  // namespace k3
