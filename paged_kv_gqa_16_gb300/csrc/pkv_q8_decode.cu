// pkv_q8_decode.cu -- split-free decode attention over the 8-bit cache.
//
// out[b, h] = sum_t w_t V_t / sum_t w_t, w_t = exp(scale q.K_t - max), with
// K_t = 2^ek code, V_t = 2^ev code.  One block per (row, kv head): chunks of
// 128 tokens, a thread a token for the scores, a thread a column for the sum.
#include <cmath>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

constexpr int kChunk = 128;

template <int D>
__global__ void __launch_bounds__(kChunk) decode_q8_kernel(const FusedParams p)
{
    __shared__ float s_q[16][D];
    __shared__ float s_p[16][kChunk];
    __shared__ float s_m[16], s_l[16], s_a[16];
    __shared__ long long s_slot[kChunk];
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x % p.Hkv, tid = threadIdx.x;
    const int rep = p.n_rep;
    int L = p.seq_lens[b];
    const int pg0 = p.kv_indptr[b], pg1 = p.kv_indptr[b + 1];
    unsigned bad = 0;
    if (L < 0 || L > p.max_seq_len) {
        bad |= kFlagBadLen;
        L = L < 0 ? 0 : p.max_seq_len;
    }
    if (pg0 < 0 || pg1 < pg0 || pg1 > p.num_indices) {
        bad |= kFlagBadPage;
        L = 0;
    } else if ((long long)(pg1 - pg0) * p.page_size < L) {
        bad |= kFlagBadPage;
        L = (pg1 - pg0) * p.page_size;
    }
    if (bad && kvh == 0 && tid == 0)
        atomicOr(p.status, bad);
    const size_t q0 = ((size_t)b * p.Hq + (size_t)kvh * rep) * D;
    for (int i = tid; i < rep * D; i += kChunk)
        s_q[i / D][i % D] = __bfloat162float(p.q[q0 + i]) * p.scale_log2;
    if (tid < 16) {
        s_m[tid] = -INFINITY;
        s_l[tid] = 0.f;
    }
    const int g = tid / D, col = tid % D;        // PV: column col, tokens g, g + groups
    constexpr int kGroups = kChunk / D;
    float acc[16];
    for (int h = 0; h < 16; ++h)
        acc[h] = 0.f;
    __syncthreads();
    for (int c0 = 0; c0 < L; c0 += kChunk) {
        const int t = c0 + tid;
        long long slot = -1;
        if (t < L) {
            int page = p.kv_indices[pg0 + t / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                atomicOr(p.status, kFlagBadPage);
                page = 0;
            }
            slot = (long long)page * p.page_size + t % p.page_size;
            const size_t row = (size_t)slot * p.Hkv + kvh;
            const float f = q8_scale(p.k_scale[row]);
            const uint32_t *k = reinterpret_cast<const uint32_t *>(p.k_codes + row * D);
            float s[16];
            for (int h = 0; h < 16; ++h)
                s[h] = 0.f;
            for (int d = 0; d < D / 4; ++d) {
                const uint32_t w = k[d];
                const uint32_t a = f16x2_of_e4m3x2(w), c = f16x2_of_e4m3x2_hi(w);
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
                const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&c));
#pragma unroll
                for (int h = 0; h < 16; ++h)
                    if (h < rep)
                        s[h] += x.x * s_q[h][4 * d] + x.y * s_q[h][4 * d + 1] +
                                y.x * s_q[h][4 * d + 2] + y.y * s_q[h][4 * d + 3];
            }
#pragma unroll
            for (int h = 0; h < 16; ++h)
                if (h < rep)
                    s_p[h][tid] = s[h] * f;
        } else {
            for (int h = 0; h < rep; ++h)
                s_p[h][tid] = -INFINITY;
        }
        s_slot[tid] = slot;
        __syncthreads();
        for (int h = tid / 32; h < rep; h += kChunk / 32) {
            const int lane = tid % 32;
            float m = s_m[h];
            for (int i = lane; i < kChunk; i += 32)
                m = fmaxf(m, s_p[h][i]);
            for (int o = 1; o < 32; o <<= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float base = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            for (int i = lane; i < kChunk; i += 32) {
                const float e = exp2f(s_p[h][i] - base);
                s_p[h][i] = e;
                l += e;
            }
            for (int o = 1; o < 32; o <<= 1)
                l += __shfl_xor_sync(0xffffffffu, l, o);
            __syncwarp();
            if (lane == 0) {
                const float a = exp2f(s_m[h] - base);
                s_a[h] = a;
                s_l[h] = s_l[h] * a + l;
                s_m[h] = m;
            }
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 16; ++h)
            if (h < rep)
                acc[h] *= s_a[h];
        for (int i = g; i < kChunk && c0 + i < L; i += kGroups) {
            const size_t row = (size_t)s_slot[i] * p.Hkv + kvh;
            const uint32_t a = f16x2_of_e4m3x2(p.v_codes[row * D + col]);
            const float v = __low2float(*reinterpret_cast<const __half2 *>(&a)) *
                            q8_scale(p.v_scale[row]);
#pragma unroll
            for (int h = 0; h < 16; ++h)
                if (h < rep)
                    acc[h] = fmaf(s_p[h][i], v, acc[h]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 16; ++h) {
        if (h >= rep)
            break;
        float o = acc[h];
        if (kGroups > 1) {                // the column's other groups
            s_p[h][tid] = o;
            __syncthreads();
            if (g == 0)
                for (int k = 1; k < kGroups; ++k)
                    o += s_p[h][k * D + col];
        }
        if (g == 0)
            p.out[q0 + (size_t)h * D + col] =
                __float2bfloat16_rn(s_l[h] > 0.f ? o / s_l[h] : 0.f);
    }
}

} // namespace

cudaError_t launch_decode_q8(const FusedParams &p, int D, int grid, cudaStream_t stream)
{
    (void)grid;
    const dim3 blocks((unsigned)(p.B * p.Hkv));
    if (D == 64)
        return launch_pdl(decode_q8_kernel<64>, blocks, dim3(kChunk), 0, stream, p);
    return launch_pdl(decode_q8_kernel<128>, blocks, dim3(kChunk), 0, stream, p);
}

} // namespace pkv
