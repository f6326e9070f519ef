// pkv_partition.cuh -- the token-balanced partition of a decode call and the
// waits of its copy pipelines, shared by the decode kernels of the bf16 and
// the 8-bit cache.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr float kLn2f = 0.693147180559945309f;
constexpr float kLog2ef = 1.4426950408889634f;
constexpr int kSmemLimit = 232448;        // opt-in shared memory per block, sm_100 family
constexpr unsigned kFull = 0xffffffffu;

// Wait for phase `parity` of `bar` (limit_ns as mbar_wait_bounded: zero is one
// non-blocking probe); false if the limit ran out or another warp aborted
// (*abort set).  The abort word is read only once the phase is not already
// complete: a warp that fails stops its part of the pipeline, so every other
// warp's next wait that blocks sees the word.
__device__ __forceinline__ bool mbar_wait_or_abort(uint64_t *bar, uint32_t parity,
                                                   unsigned long long limit_ns,
                                                   volatile int *abort)
{
    if (limit_ns == 0)
        return mbar_test_wait(bar, parity) && !*abort;
    if (mbar_try_wait(bar, parity))
        return true;
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort || global_timer_ns() - t0 > limit_ns)
            return false;
    }
    return true;
}

// Block owning flattened token x under the partition x in [c*T/G, (c+1)*T/G).
__device__ __forceinline__ int block_of(long long x, long long T, int G)
{
    return (int)(((x + 1) * G + T - 1) / T) - 1;
}

// ---- the partition, shared by the decode kernel and the per-step plan -----
// Token count of virtual row r after the checks: a negative length counts as
// zero, one above max_seq_len as max_seq_len, and a row whose table is
// malformed or does not cover its length is cut to what the table covers.
// The failed checks' flags go to `bad`.
__device__ __forceinline__ int checked_row_len(const FusedParams &p, int r, unsigned &bad)
{
    const int b = r % p.B;
    int L = p.seq_lens[b];
    const int pg0 = p.kv_indptr[b];
    const int pg1 = p.kv_indptr[b + 1];
    if (L < 0 || L > p.max_seq_len) {
        bad |= kFlagBadLen;
        L = L < 0 ? 0 : p.max_seq_len;
    }
    if (pg0 < 0 || pg1 < pg0 || pg1 > p.num_indices) {
        bad |= kFlagBadPage;
        L = 0;
    } else if ((long long)(pg1 - pg0) * p.page_size < (long long)L) {
        bad |= kFlagBadPage;
        L = (pg1 - pg0) * p.page_size;
    }
    return L;
}

// prefix[0..n] of n rows' partition weights (a non-empty row weighs its tokens
// plus row_cost), computed by every thread of the block; row i of them is
// virtual row row_of(i); report: OR the flags of the first B virtual rows into
// the status word.
template <typename RowOf>
__device__ __forceinline__ void row_prefix(const FusedParams &p, int *prefix, int n, RowOf row_of,
                                           bool report)
{
    const int Bv = n, lane = threadIdx.x & 31;
    for (int r = threadIdx.x; r < Bv; r += blockDim.x) {
        unsigned bad = 0;
        const int L = checked_row_len(p, row_of(r), bad);
        if (bad && report && row_of(r) < p.B)
            atomicOr(p.status, bad);
        prefix[r + 1] = L > 0 ? L + p.row_cost : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int carry = 0;
        for (int base = 0; base < Bv; base += 32) {
            const int i = base + lane;
            int v = i < Bv ? prefix[i + 1] : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int n = __shfl_up_sync(kFull, v, off);
                if (lane >= off)
                    v += n;
            }
            v += carry;
            if (i < Bv)
                prefix[i + 1] = v;
            carry = __shfl_sync(kFull, v, 31);
        }
        if (lane == 0)
            prefix[0] = 0;
    }
    __syncthreads();
}

// The same of all virtual rows.
__device__ __forceinline__ void row_prefix(const FusedParams &p, int *prefix, bool report)
{
    row_prefix(p, prefix, p.Bv, [](int r) { return r; }, report);
}

// Blocks that get work: at least kFusedMinTokens positions each, at most the
// grid, at least one.
__device__ __forceinline__ unsigned active_blocks(unsigned T, unsigned grid)
{
    unsigned Gu = (T + kFusedMinTokens - 1) / kFusedMinTokens;
    if (Gu > grid)
        Gu = grid;
    return Gu < 1 ? 1 : Gu;
}

// First row whose positions reach past `start` (never an empty row).
__device__ __forceinline__ int first_row(const int *prefix, int Bv, long long start)
{
    int lo = 0, hi = Bv - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((long long)prefix[mid + 1] > start)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// The per-step plan (int32 words): [0] T, [1] active blocks G, [2] grid,
// [3] virtual rows Bv, [4] rows B, [5] page_size, [6] row_cost, [7..15] unused; then
// prefix[0..Bv] (padded to a multiple of 4 words); then one entry of
// kPlanEntryInts words per block of the grid: [0] its first row r0 (-1: no
// work), [1] the base wb of that row's page-table window, [2] the row's
// first table entry kv_indptr[b], [3] its entry count, [4] and [5] the
// positions of the row's first and last-plus-one token, [6] and [7] the
// block's positions [start, end), [8..71] the window (the row's table
// entries wb .. wb + 63, 0 past the table).  A plan of the 8-bit cache's decode
// has no entries.
constexpr int kPlanHeaderInts = 16;
constexpr int kPlanEntryInts = 72;

__device__ __forceinline__ const int32_t *plan_entry(const int32_t *plan, int Bv, int c)
{
    return plan + kPlanHeaderInts + ((Bv + 1 + 3) & ~3) + (size_t)c * kPlanEntryInts;
}

// Whether a plan is of this grid, shape and row cost.
__device__ __forceinline__ bool plan_fits(const int32_t *plan, int grid, int Bv, int B,
                                          int page_size, int row_cost)
{
    const int g = plan[2], bv = plan[3], b = plan[4], ps = plan[5], rc = plan[6];   // at once
    return (g == grid) & (bv == Bv) & (b == B) & (ps == page_size) & (rc == row_cost);
}

} // namespace pkv
