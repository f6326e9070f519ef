// pkv_q8_read.cu -- the rows of an 8-bit cache read back as bf16.
//
// bf16(code * 2^e) is exact: a code has four significant bits, a bf16 eight.
// Token t of row b moves from pool page kv_indices[kv_indptr[b] + t / ps] to
// output page kv_indptr[b] + t / ps, so the output, taken as one list of token
// slots (entry * ps + slot), has the table's order.  A block takes a few
// consecutive slots of that list: a thread a slot finds the entry's row, its
// length and the page, then all threads stream the slots' heads, 16 codes of K
// and the 16 of V beside them at a time.  3 bytes of traffic a value and
// nothing else to do: bound by memory.  32 ragged rows, 73,728 tokens of 8 heads
// of 128, 454 MB: 75.0 us, 6,060 GB/s, 89% of the copy bandwidth (86.4 us with
// two 16-byte stores in place of each 32-byte one, 92 with four vectors of one
// pool a thread, 105 with 8-byte loads).
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlots = 64;            // token slots a block takes at most
constexpr int kBlockValues = 16384;      // values of K (and of V) a block aims at

// Eight codes times f as eight bf16.
__device__ __forceinline__ uint4 decode8(uint32_t lo, uint32_t hi, float f)
{
    const uint32_t h[4] = {f16x2_of_e4m3x2(lo), f16x2_of_e4m3x2_hi(lo), f16x2_of_e4m3x2(hi),
                           f16x2_of_e4m3x2_hi(hi)};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        o[j] = pack_bf16x2(x.x * f, x.y * f);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 codes times f to dst: one 32-byte store where the outputs are so aligned
// (two of 16 bytes write each 32-byte sector in halves, a warp apart).
template <bool WIDE>
__device__ __forceinline__ void store16(__nv_bfloat16 *dst, uint4 c, float f)
{
    const uint4 a = decode8(c.x, c.y, f), b = decode8(c.z, c.w, f);
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                     "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z),
                     "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = a;
        reinterpret_cast<uint4 *>(dst)[1] = b;
    }
}

// Pool slot of output slot `at`, or -1 if no token of a row is there.
__device__ __forceinline__ long long source_of(const ReadQ8Params &p, long long at)
{
    const int j = p.ps_shift >= 0     ? (int)(at >> p.ps_shift)
                  : at < (1ll << 31) ? (int)at / p.page_size
                                     : (int)(at / p.page_size);
    const int sl = (int)(at - (long long)j * p.page_size);
    const int page = p.kv_indices[j];
    int lo = 0, hi = p.B - 1;            // the last row whose entries start at or before j
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.kv_indptr[mid] <= j)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int pg0 = p.kv_indptr[lo], pg1 = p.kv_indptr[lo + 1], L = p.seq_lens[lo];
    if (pg0 < 0 || j < pg0 || j >= pg1 || pg1 > p.num_indices || L < 0 || L > p.max_seq_len ||
        (long long)(j - pg0) * p.page_size + sl >= L)
        return -1;
    if (page < 0 || page >= p.num_pages) {
        if (p.status != nullptr)
            atomicOr(p.status, kFlagBadPage);
        return -1;
    }
    return (long long)page * p.page_size + sl;
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) read_q8_kernel(const ReadQ8Params p)
{
    constexpr int VPH = D / 16;          // 16-code vectors of a head
    __shared__ long long s_src[kMaxSlots];
    grid_dependency_wait();
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
    const long long slots = (long long)p.num_indices * p.page_size;
    const int per_tok = p.Hkv * VPH;     // vectors of a token, of K or of V
    for (long long s0 = (long long)blockIdx.x * p.per_block; s0 < slots;
         s0 += (long long)gridDim.x * p.per_block) {
        const int n = (int)(slots - s0 < p.per_block ? slots - s0 : p.per_block);
        if (threadIdx.x < n)
            s_src[threadIdx.x] = source_of(p, s0 + threadIdx.x);
        __syncthreads();
        const int vecs = n * per_tok;
        for (int i = threadIdx.x; i < vecs; i += kThreads) {
            const int tok = i / per_tok, k = i - tok * per_tok;
            const long long src = s_src[tok];
            if (src < 0)
                continue;
            const size_t head = (size_t)src * p.Hkv + k / VPH;
            const size_t from = head * D + (k % VPH) * 16;
            const size_t to = ((size_t)(s0 + tok) * per_tok + k) * 16;
            const uint4 kc = __ldcs(reinterpret_cast<const uint4 *>(p.k_codes + from));
            const uint4 vc = __ldcs(reinterpret_cast<const uint4 *>(p.v_codes + from));
            const float fk = q8_scale(p.k_scale[head]), fv = q8_scale(p.v_scale[head]);
            store16<WIDE>(p.k_out + to, kc, fk);
            store16<WIDE>(p.v_out + to, vc, fv);
        }
        __syncthreads();
    }
    grid_launch_dependents();
}

} // namespace

cudaError_t launch_read_q8(const ReadQ8Params &params, int D, cudaStream_t stream)
{
    ReadQ8Params p = params;
    const long long slots = (long long)p.num_indices * p.page_size;
    if (slots <= 0)
        return cudaSuccess;
    const int per = kBlockValues / (p.Hkv * D > kBlockValues ? kBlockValues : p.Hkv * D);
    p.per_block = per < kMaxSlots ? per : kMaxSlots;
    const long long blocks = (slots + p.per_block - 1) / p.per_block;
    const dim3 grid((unsigned)(blocks < (1ll << 30) ? blocks : (1ll << 30)));
    const bool wide = ((reinterpret_cast<uintptr_t>(p.k_out) |
                        reinterpret_cast<uintptr_t>(p.v_out)) & 31) == 0;
    auto run = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, p); };
    if (D == 64)
        return wide ? run(read_q8_kernel<64, true>) : run(read_q8_kernel<64, false>);
    return wide ? run(read_q8_kernel<128, true>) : run(read_q8_kernel<128, false>);
}

} // namespace pkv
