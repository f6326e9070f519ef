// pkv_q8_read.cu -- the rows of an 8-bit cache read back as bf16.
//
// bf16(code * 2^e) is exact: a code has four significant bits, a bf16 eight.
// Token t of row b moves from pool page kv_indices[kv_indptr[b] + t / ps] to
// output page kv_indptr[b] + t / ps, so the output has the table's order and
// a thread needs, for one 16-code vector, its table entry's row, that row's
// length, and the page id.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// Eight codes times 2^(sb - 127) as eight bf16.
__device__ __forceinline__ uint4 decode8(uint2 c, float f)
{
    uint4 r;
    const uint32_t h[4] = {f16x2_of_e4m3x2(c.x), f16x2_of_e4m3x2_hi(c.x), f16x2_of_e4m3x2(c.y),
                           f16x2_of_e4m3x2_hi(c.y)};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        o[j] = pack_bf16x2(x.x * f, x.y * f);
    }
    r.x = o[0]; r.y = o[1]; r.z = o[2]; r.w = o[3];
    return r;
}

// One block per table entry (page): the entry's row is found once, then the
// block's threads move the page's valid tokens, K and V.
__global__ void __launch_bounds__(kThreads) read_q8_kernel(const ReadQ8Params p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    // the rows' own checks, each reported once
    for (long long b = blockIdx.x * (long long)kThreads + threadIdx.x; b < p.B;
         b += (long long)gridDim.x * kThreads) {
        const int L = p.seq_lens[b], pg0 = p.kv_indptr[b], pg1 = p.kv_indptr[b + 1];
        unsigned bad = 0;
        if (L < 0 || L > p.max_seq_len)
            bad |= kFlagBadLen;
        else if (L > 0 && (pg0 < 0 || pg1 < pg0 || pg1 > p.num_indices ||
                           (long long)(pg1 - pg0) * p.page_size < L))
            bad |= kFlagBadPage;
        if (bad && p.status != nullptr)
            atomicOr(p.status, bad);
    }
    for (int j = blockIdx.x; j < p.num_indices; j += gridDim.x) {
        int lo = 0, hi = p.B - 1;        // the last row whose entries start at or before j
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.kv_indptr[mid] <= j)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int pg0 = p.kv_indptr[lo], pg1 = p.kv_indptr[lo + 1], L = p.seq_lens[lo];
        if (pg0 < 0 || j < pg0 || j >= pg1 || pg1 > p.num_indices || L < 0 || L > p.max_seq_len)
            continue;
        const long long left = (long long)L - (long long)(j - pg0) * p.page_size;
        if (left <= 0)
            continue;
        const int page = p.kv_indices[j];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0 && p.status != nullptr)
                atomicOr(p.status, kFlagBadPage);
            continue;
        }
        const long long n = left < p.page_size ? left : p.page_size;
        const int vph = p.D / 8;                       // 8-value vectors of a head
        const long long vecs = n * p.Hkv * vph;
        const size_t src = (size_t)page * p.page_size * p.Hkv;
        const size_t dst = (size_t)j * p.page_size * p.Hkv;
        for (long long i = threadIdx.x; i < 2 * vecs; i += kThreads) {
            const bool v = i >= vecs;
            const long long at = v ? i - vecs : i;
            const long long head = at / vph;
            const uint8_t *codes = v ? p.v_codes : p.k_codes;
            const float f = q8_scale((v ? p.v_scale : p.k_scale)[src + head]);
            const uint2 c = *reinterpret_cast<const uint2 *>(codes + src * p.D + at * 8);
            *reinterpret_cast<uint4 *>((v ? p.v_out : p.k_out) + dst * p.D + at * 8) =
                decode8(c, f);
        }
    }
}

} // namespace

cudaError_t launch_read_q8(const ReadQ8Params &p, cudaStream_t stream)
{
    if (p.num_indices <= 0)
        return cudaSuccess;
    const int blocks = p.num_indices < (1 << 20) ? p.num_indices : (1 << 20);
    return launch_pdl(read_q8_kernel, dim3(blocks), dim3(kThreads), 0, stream, p);
}

} // namespace pkv
