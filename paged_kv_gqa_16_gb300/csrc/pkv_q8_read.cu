// pkv_q8_read.cu -- the rows of an 8-bit cache read back as bf16.
//
// bf16(code * 2^e) is exact: a code has four significant bits, a bf16 eight.
// (Scales under 2^-124 and over 2^119, which the writes do not choose, leave bf16's
// range: the result is then the nearest bf16, past its largest value infinity.)
// Token t of row b moves from pool page kv_indices[kv_indptr[b] + t / ps] to
// output page kv_indptr[b] + t / ps, so the output, taken as one list of token
// slots (entry * ps + slot), has the table's order.  A warp takes a few consecutive
// slots of that list: a lane a slot finds the entry's row, its length and the page,
// then all lanes stream the slots' heads, 16 codes of K and the 16 of V beside them
// at a time.  3 bytes of traffic a value and nothing else to do: bound by memory.
// 32 ragged rows, 73,728 tokens of 8 heads of 128, 454 MB: 71.7 us, 6,330 GB/s, 93% of
// the copy bandwidth.  Variants, measured against 73.4 us for this layout at the time:
// 86.4 us with two 16-byte stores in place of each 32-byte one, 92 with four vectors of
// one pool a thread, 105 with 8-byte loads.  Blocks of 256 threads that look up their
// slots together took 74.6; 9.9 in place of 8.4 for 6,152 tokens, 7.0 in place of 4.9
// for those of D = 64, 3.0 in place of 2.2 for 137, 4.8 in place of 5.5 for 48,000 of
// one head of 64 at page size 1.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

// 12 blocks an SM, at most 42 registers: 76.6 us with the 48 that the compiler takes
// by itself, 80.0 with 36; 64 threads: 75.7.
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Values of K (and of V) a warp takes at most (1024: 77.8 us, 4096: 78.7), and the
// warps that a small call is spread over (half and twice as many: within 1%).
constexpr int kWarpValues = 2048;
constexpr int kShare = 4864;

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

// The scale of any e8m0 byte: 0 stands for 2^-127, 255 for NaN.
__device__ __forceinline__ float any_scale(unsigned byte)
{
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
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
__global__ void __launch_bounds__(kThreads, 12) read_q8_kernel(const ReadQ8Params p)
{
    constexpr int VPH = D / 16;          // 16-code vectors of a head
    grid_dependency_wait();
    // the rows' own checks, each reported once
    for (long long b = blockIdx.x * (long long)kThreads + threadIdx.x; b < p.B;
         b += (long long)gridDim.x * kThreads) {
        const int L = p.seq_lens[b], pg0 = p.kv_indptr[b], pg1 = p.kv_indptr[b + 1];
        unsigned bad = 0;
        if (L < 0 || L > p.max_seq_len)
            bad |= kFlagBadLen;
        // (an idle row's offsets too: the search for a slot's row goes by them)
        if (pg0 < 0 || pg1 < pg0 || pg1 > p.num_indices ||
            ((bad & kFlagBadLen) == 0 && (long long)(pg1 - pg0) * p.page_size < L))
            bad |= kFlagBadPage;
        if (bad && p.status != nullptr)
            atomicOr(p.status, bad);
    }
    const long long slots = (long long)p.num_indices * p.page_size;
    const int per_tok = p.Hkv * VPH;     // vectors of a token, of K or of V
    const int lane = threadIdx.x & 31;
    const long long warp = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    for (long long s0 = warp * p.per_warp; s0 < slots;
         s0 += (long long)gridDim.x * kWarps * p.per_warp) {
        const int n = (int)(slots - s0 < p.per_warp ? slots - s0 : p.per_warp);
        const long long mine = lane < n ? source_of(p, s0 + lane) : -1;
        const int vecs = n * per_tok;
        for (int i0 = 0; i0 < vecs; i0 += 32) {
            const int i = i0 + lane, tok = min(i / per_tok, n - 1), k = i - tok * per_tok;
            const long long src = __shfl_sync(0xffffffffu, mine, tok);
            if (src < 0 || i >= vecs)
                continue;
            const size_t head = (size_t)src * p.Hkv + k / VPH;
            const size_t from = head * D + (k % VPH) * 16;
            const size_t to = ((size_t)(s0 + tok) * per_tok + k) * 16;
            const uint4 kc = __ldcs(reinterpret_cast<const uint4 *>(p.k_codes + from));
            const uint4 vc = __ldcs(reinterpret_cast<const uint4 *>(p.v_codes + from));
            const float fk = any_scale(p.k_scale[head]), fv = any_scale(p.v_scale[head]);
            store16<WIDE>(p.k_out + to, kc, fk);
            store16<WIDE>(p.v_out + to, vc, fv);
        }
    }
    grid_launch_dependents();
}

} // namespace

cudaError_t launch_read_q8(const ReadQ8Params &params, int D, cudaStream_t stream)
{
    ReadQ8Params p = params;
    const long long slots = (long long)p.num_indices * p.page_size;
    const int most = p.Hkv * D > kWarpValues ? 1 : kWarpValues / (p.Hkv * D);   // up to 32
    // a slot's share, in whole rounds of 32 lanes (one head of 64: 6.0 us without)
    const int per_tok = p.Hkv * (D / 16), round = per_tok < 32 ? 32 / per_tok : 1;
    const long long share = slots / kShare / round * round;
    p.per_warp = share >= most ? most : share > round ? (int)share : round;
    const long long per_block = (long long)p.per_warp * kWarps;
    const long long blocks = (slots + per_block - 1) / per_block;
    // (an empty table: one block, for the rows' checks)
    const dim3 grid((unsigned)(blocks < 1 ? 1 : blocks < (1ll << 30) ? blocks : (1ll << 30)));
    const bool wide = ((reinterpret_cast<uintptr_t>(p.k_out) |
                        reinterpret_cast<uintptr_t>(p.v_out)) & 31) == 0;
    auto run = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, p); };
    if (D == 64)
        return wide ? run(read_q8_kernel<64, true>) : run(read_q8_kernel<64, false>);
    return wide ? run(read_q8_kernel<128, true>) : run(read_q8_kernel<128, false>);
}

} // namespace pkv
