// rows.cuh -- which slot a packed token row belongs to, and at which position it stands.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace k3 {

// The number of entries of the non-decreasing v[0 .. n) that are <= x, by a 32-way search of the whole
// warp: one load a lane and step, ceil(log32(n)) steps.  Every lane gets the answer.
__device__ __forceinline__ int warp_count_le(const int32_t* v, int n, int x)
{
    const int lane = (int)lane_id();
    int lo = 0;  // v[0 .. lo) <= x, and the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = min(step * (lane + 1), n) - 1;  // the last entry of this lane's piece
        const unsigned le = __ballot_sync(0xFFFFFFFFu, v[lo + i] <= x);
        const int pieces = __popc(le);  // whole pieces that are <= x (a prefix: v is non-decreasing)
        if (pieces == 32) return lo + n;
        const int done = pieces * step;
        lo += done;
        n = step > 1 ? min(step, n - done) - 1 : 0;  // the next piece's last entry is > x
    }
    return lo;
}

// The last slot b with row_start[b] <= r (slot 0 when there is none; row_start is non-decreasing), by one thread.
__device__ __forceinline__ int last_slot_from(const int32_t* row_start, int B, int r)
{
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_start[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Row r of the packed rows: slot b, position pos.  False when the row lies outside every slot or its
// position is negative.  row_start null: row r is the only one of slot r.  A whole warp calls it.
__device__ __forceinline__ bool row_position(const int32_t* row_start, const int32_t* pos0, int B, int r, int& b,
                                             int64_t& pos)
{
    if (!row_start) {
        b = r;
        pos = pos0[r];
        return pos >= 0;
    }
    b = warp_count_le(row_start + 1, B, r);
    if (b >= B) return false;
    const int first = row_start[b];
    if (r < first) return false;
    pos = (int64_t)pos0[b] + (r - first);
    return pos >= 0;
}

}  // namespace k3
