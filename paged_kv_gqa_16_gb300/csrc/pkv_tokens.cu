// pkv_tokens.cu -- new tokens into the cache, normalised, rotated and (for
// the 8-bit cache) quantised in one pass.
//
// For a head vector x of D values (fp32 throughout, one rounding at the end):
//   norm      x <- x * rsqrt(mean(x^2) + eps) * w          (q and k, optional)
//   rotation  (x[2i], x[2i+1]) <- (x[2i] c - x[2i+1] s, x[2i] s + x[2i+1] c),
//             (c, s) of the token's position and pair i     (q and k, optional)
//   store     bf16, or e4m3 codes of x 2^-e with the power of two
//             e = clamp(ceil(log2(amax / 448)), -40, 40) of the vector.  Codes
//             are floating point, so a power of two keeps the precision of an
//             arbitrary scale, costs one byte, and scales without rounding.
//
// A head vector belongs to a group of D / 8 lanes with eight values each, so
// the norm's sum and the largest magnitude are log2(D / 8) shuffles, and every
// load is 16 bytes.  A block takes a few consecutive tokens: their rows,
// positions and slots are looked up once into shared memory, then its groups
// run over the tokens' Hq + 2 Hkv vectors.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;        // tokens a block takes at most

struct TokenPlace {
    int pos;                         // -1: the token writes nothing
    unsigned slot_hi, slot_lo;       // flat pool slot (page * page_size + slot)
};

// Row, position and slot of token t; flags in `bad` (kFlag*), pos -1 if it
// writes nothing.
template <bool EXTEND>
__device__ __forceinline__ TokenPlace place_token(const TokenWriteParams &p, int t, unsigned &bad)
{
    TokenPlace r{-1, 0, 0};
    int b = t, pos;
    if constexpr (EXTEND) {
        int lo = 0, hi = p.B - 1;    // the last row that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.qo_indptr[mid] <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
        const int a = p.qo_indptr[b], e = p.qo_indptr[b + 1];
        const int L = p.seq_lens[b];
        if (t < a || t >= e || e - a > L || L > p.max_seq_len) {
            bad |= kFlagBadLen;
            return r;
        }
        pos = L - (e - a) + (t - a);
    } else {
        const int L = p.seq_lens[b];
        if (L <= 0 || L > p.max_seq_len) {
            if (L != 0)
                bad |= kFlagBadLen;
            return r;
        }
        pos = L - 1;
    }
    const int pg0 = p.kv_indptr[b], pg1 = p.kv_indptr[b + 1];
    const int pi = pos / p.page_size;
    int page = -1;
    if (pg0 >= 0 && pg1 >= pg0 && pg1 <= p.num_indices && pi < pg1 - pg0)
        page = p.kv_indices[pg0 + pi];
    if (page < 0 || page >= p.num_pages)
        bad |= kFlagBadPage;
    if (p.rope != nullptr && pos >= p.rope_max_pos)
        bad |= kFlagBadPos;
    if (bad)
        return r;
    const unsigned long long slot =
        (unsigned long long)page * p.page_size + (unsigned)(pos - pi * p.page_size);
    r.pos = pos;
    r.slot_hi = (unsigned)(slot >> 32);
    r.slot_lo = (unsigned)slot;
    return r;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1)
        x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

template <int LANES>
__device__ __forceinline__ float group_max(float x)
{
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1)
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}

template <int D, bool Q8, bool EXTEND>
__global__ void __launch_bounds__(kThreads) token_write_kernel(const TokenWriteParams p)
{
    constexpr int LANES = D / 8;             // lanes of a head vector
    constexpr int GROUPS = kThreads / LANES;
    __shared__ TokenPlace s_place[kMaxTokens];
    grid_dependency_wait();
    const int t0 = blockIdx.x * p.per_block;
    const int nt = min(p.per_block, p.T - t0);
    if (threadIdx.x < nt) {
        unsigned bad = 0;
        s_place[threadIdx.x] = place_token<EXTEND>(p, t0 + threadIdx.x, bad);
        if (bad && p.status != nullptr)
            atomicOr(p.status, bad);
    }
    __syncthreads();
    grid_launch_dependents();

    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int nv = p.Hq + 2 * p.Hkv;         // vectors of a token: q, k, v heads
    const int total = nt * nv;
    // every lane runs the same number of rounds: the shuffles need whole warps
    for (int i0 = 0; i0 < total; i0 += GROUPS) {
        const int i = i0 + group;
        const bool in = i < total;
        const int tok = in ? i / nv : 0;
        int h = in ? i - tok * nv : 0;
        const TokenPlace place = s_place[tok];
        const bool live = in && place.pos >= 0;
        const size_t t = (size_t)(t0 + tok);
        const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;   // q, k, v
        h -= kind == 0 ? 0 : kind == 1 ? p.Hq : p.Hq + p.Hkv;
        const __nv_bfloat16 *src = kind == 0   ? p.q + t * p.q_stride
                                   : kind == 1 ? p.k + t * p.k_stride
                                               : p.v + t * p.v_stride;
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (live)
            raw = *reinterpret_cast<const uint4 *>(src + h * D + lane * 8);
        float x[8];
        x[0] = bf16_lo(raw.x); x[1] = bf16_hi(raw.x);
        x[2] = bf16_lo(raw.y); x[3] = bf16_hi(raw.y);
        x[4] = bf16_lo(raw.z); x[5] = bf16_hi(raw.z);
        x[6] = bf16_lo(raw.w); x[7] = bf16_hi(raw.w);

        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss = fmaf(x[j], x[j], ss);
        ss = group_sum<LANES>(ss);
        const __nv_bfloat16 *w = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
        if (w != nullptr) {
            const uint4 wr = *reinterpret_cast<const uint4 *>(w + lane * 8);
            const float f = rsqrtf(ss * (1.f / D) + p.norm_eps);
            x[0] *= f * bf16_lo(wr.x); x[1] *= f * bf16_hi(wr.x);
            x[2] *= f * bf16_lo(wr.y); x[3] *= f * bf16_hi(wr.y);
            x[4] *= f * bf16_lo(wr.z); x[5] *= f * bf16_hi(wr.z);
            x[6] *= f * bf16_lo(wr.w); x[7] *= f * bf16_hi(wr.w);
        }
        if (kind != 2 && p.rope != nullptr && live) {
            const float4 *cs = reinterpret_cast<const float4 *>(p.rope + (size_t)place.pos * D) +
                               lane * 2;
            const float4 c01 = cs[0], c23 = cs[1];
            rotate(x[0], x[1], c01.x, c01.y);
            rotate(x[2], x[3], c01.z, c01.w);
            rotate(x[4], x[5], c23.x, c23.y);
            rotate(x[6], x[7], c23.z, c23.w);
        }
        const size_t slot = ((size_t)place.slot_hi << 32) | place.slot_lo;
        if constexpr (Q8) {
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                amax = fmaxf(amax, fabsf(x[j]));
            amax = group_max<LANES>(amax);
            if (kind != 0) {
                const int sb = q8_scale_byte(amax);
                const uint2 codes = q8_encode8(x, sb);
                if (live) {
                    uint8_t *dst = static_cast<uint8_t *>(kind == 1 ? p.k_pool : p.v_pool);
                    *reinterpret_cast<uint2 *>(dst + (slot * p.Hkv + h) * D + lane * 8) = codes;
                    if (lane == 0)
                        (kind == 1 ? p.k_scale : p.v_scale)[slot * p.Hkv + h] = (uint8_t)sb;
                }
            }
        }
        if (kind == 0 || !Q8) {
            uint4 y = raw;                       // V: unchanged
            if (kind != 2) {
                y.x = pack_bf16x2(x[0], x[1]);
                y.y = pack_bf16x2(x[2], x[3]);
                y.z = pack_bf16x2(x[4], x[5]);
                y.w = pack_bf16x2(x[6], x[7]);
            }
            __nv_bfloat16 *dst =
                kind == 0 ? p.q_out + (t * p.Hq + h) * D
                          : static_cast<__nv_bfloat16 *>(kind == 1 ? p.k_pool : p.v_pool) +
                                (slot * p.Hkv + h) * D;
            if (live)
                *reinterpret_cast<uint4 *>(dst + lane * 8) = y;
        }
    }
}

template <int D, bool Q8, bool EXTEND>
cudaError_t launch(const TokenWriteParams &params, cudaStream_t stream)
{
    TokenWriteParams p = params;
    p.per_block = EXTEND ? 4 : 1;
    const unsigned blocks = (unsigned)((p.T + p.per_block - 1) / p.per_block);
    return launch_pdl(token_write_kernel<D, Q8, EXTEND>, dim3(blocks), dim3(kThreads), 0, stream,
                      p);
}

template <int D>
cudaError_t launch_d(const TokenWriteParams &p, cudaStream_t stream)
{
    const bool q8 = p.k_scale != nullptr, extend = p.qo_indptr != nullptr;
    if (q8)
        return extend ? launch<D, true, true>(p, stream) : launch<D, true, false>(p, stream);
    return extend ? launch<D, false, true>(p, stream) : launch<D, false, false>(p, stream);
}

} // namespace

cudaError_t launch_token_write(const TokenWriteParams &p, int D, cudaStream_t stream)
{
    if (p.T <= 0)
        return cudaSuccess;
    return D == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

} // namespace pkv
