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
// The pass reads and writes every value once and is bound by memory, if the
// arithmetic is kept small: a head vector belongs to a group of D / 8 lanes with
// eight values each (16-byte loads; the norm's sum and the largest magnitude
// are log2(D / 8) shuffles), a group keeps one token, and the norm's weight
// and the rotation become four coefficients a pair that its lanes form once for
// all the token's query heads (and once for its K heads):
//   y[2i]   = r (x[2i] (w c) - x[2i+1] (w' s)),
//   y[2i+1] = r (x[2i] (w s) + x[2i+1] (w' c)),   r = rsqrt(mean + eps),
// in two-wide fp32 operations.  `width` groups share a token.  Every warp looks up
// its own tokens' rows, pages and rotations while their first vectors are already
// on their way.  (Each dependent load of a look-up queues behind the stream: by a
// block for all its tokens, behind a barrier, 9,537 tokens of D = 64 took 23.8 us in
// place of 22.7 at the same block size, one token of 8 rows 3.0 in place of 2.6.)
//
// Measured (CUDA-graph replay): 4 prompts of 4,096 tokens, 32 + 8 heads of 128,
// norms, 405 MB: 66.5 us, 6,090 GB/s, 90% of the copy bandwidth; the 8-bit form on
// 18,425 tokens, 416 MB: 67.7 us, 91%; 9,537 tokens of 32 + 8 heads of 64, 108 MB:
// 21.3 us, 75% (an elementwise kernel of as many bytes takes 18 us); one token of 8
// to 128 rows: 2.4 to 3.6 us, the launch and three dependent loads.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

// Threads of a block: those of one token, at least kMinThreads.  Few threads keep
// the SMs' shares even at the end: 64 against 128 and 256 gain up to 2% and 5%.
constexpr int kMinThreads = 64;
constexpr int kMaxThreads = 256;
// Query vectors, and K and V vectors, that a group has in flight, at 80 registers
// (768 threads an SM).  Extends of 16,384 tokens, 9,537 of D = 64 and 512 tokens: 4
// and 1 take 67.1, 21.6 and 4.8 us; 2 and 1 71.9, 23.3 and 4.8; 3 and 1 69.3, 22.5
// and 5.0; 4 and 2 66.3, 22.5 and 5.1; 2 and 1 at 64 registers 67.5, 21.1 and 5.1.
// One token of 8 and of 32 rows: 4 and 1 2.8 and 2.9 us, 2 and 1 2.4 and 2.6.
constexpr int kQExtend = 4;
constexpr int kQAppend = 2;
constexpr int kKv = 1;
// From this many threads on, a token gets fewer groups (1,456 tokens of D = 64: 5.6
// us with 16384 or 32768 here, 5.2 with 65536; 364: 3.5, 3.7, 4.6; 1,024 of 8 + 1
// heads of 64: 3.3, 3.5, 4.6; one token of 128 rows of 64 + 8 heads of 128: 4.5, 3.4,
// 3.5).
constexpr long long kManyThreads = 32768;

// What a token's row says of it.
struct TokenRow {
    int pos;                             // position, -1: the token writes nothing
    int at;                              // its entry of kv_indices, -1: none
    int in_page;                         // its place in that page
    unsigned bad;                        // kFlag*
};

template <bool EXTEND>
__device__ __forceinline__ TokenRow token_row(const TokenWriteParams &p, int t, int a, int e, int L,
                                              int pg0, int pg1)
{
    TokenRow r{-1, -1, 0, 0};
    int pos = L - 1;
    if constexpr (EXTEND) {
        if (a < 0 || e > p.T || t < a || t >= e || e - a > L || L > p.max_seq_len) {
            r.bad = kFlagBadLen;
            return r;
        }
        pos = L - (e - a) + (t - a);
    } else if (L <= 0 || L > p.max_seq_len) {
        r.bad = L != 0 ? kFlagBadLen : 0;
        return r;
    }
    const int pi = pos / p.page_size;
    if (pg0 >= 0 && pg1 >= pg0 && pg1 <= p.num_indices && pi < pg1 - pg0)
        r.at = pg0 + pi;
    if (p.rope != nullptr && pos >= p.rope_max_pos)
        r.bad = kFlagBadPos;
    r.pos = pos;
    r.in_page = pos - pi * p.page_size;
    return r;
}

// The row of each lane's token t, whose least in the warp is t0 (lane 0's); every
// lane calls it.  Dependent loads are the time of a small call, and of a warp that
// waits for them: a row's words are loaded at once, and for an extend those of 32
// rows from the first token's on, of which a lane takes its own by shuffles.
template <bool EXTEND>
__device__ __forceinline__ TokenRow row_of_token(const TokenWriteParams &p, int t)
{
    constexpr unsigned kAll = 0xffffffffu;
    if constexpr (!EXTEND) {
        return token_row<false>(p, t, 0, 0, p.seq_lens[t], p.kv_indptr[t], p.kv_indptr[t + 1]);
    } else {
        const int lane = threadIdx.x & 31, t0 = __shfl_sync(kAll, t, 0);
        int lo = 0, n = p.B;             // the first token's row is in [lo, lo + n)
        while (n > 32) {
            const int step = (n + 31) / 32, i = lane * step;
            const int hits = __popc(__ballot_sync(kAll, i < n && p.qo_indptr[lo + i] <= t0));
            const int to = hits > 0 ? (hits - 1) * step : 0;
            lo += to;
            n = min(step, n - to);
        }
        const int row = min(lo + lane, p.B - 1);
        int a = p.qo_indptr[row], e = p.qo_indptr[row + 1], L = p.seq_lens[row];
        int pg0 = p.kv_indptr[row], pg1 = p.kv_indptr[row + 1];
        int k = 0;                       // the last of the rows that starts at or before t
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) {
            const int start = __shfl_sync(kAll, a, k + s);
            if (lo + k + s < p.B && start <= t)
                k += s;
        }
        const int next = __shfl_sync(kAll, e, 31);
        a = __shfl_sync(kAll, a, k);
        e = __shfl_sync(kAll, e, k);
        L = __shfl_sync(kAll, L, k);
        pg0 = __shfl_sync(kAll, pg0, k);
        pg1 = __shfl_sync(kAll, pg1, k);
        int b = lo + k;
        if (k == 31 && b + 1 < p.B && next <= t) {
            // past the 32 rows: steps that double while rows start at or before the
            // token, and halve behind the last of them
            int by = 1;
            while (b + by < p.B && p.qo_indptr[b + by] <= t) {
                b += by;
                by <<= 1;
            }
            while (by >>= 1)
                if (b + by < p.B && p.qo_indptr[b + by] <= t)
                    b += by;
            a = p.qo_indptr[b], e = p.qo_indptr[b + 1], L = p.seq_lens[b];
            pg0 = p.kv_indptr[b], pg1 = p.kv_indptr[b + 1];
        }
        return token_row<true>(p, t, a, e, L, pg0, pg1);
    }
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

// Two fp32 values in one 64-bit register.
struct F2 {
    unsigned long long v;
};

__device__ __forceinline__ F2 f2(float x, float y)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float2 parts(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Eight values of a head vector: the pairs' first and second values.
struct Eight {
    F2 a[2], b[2];
};

__device__ __forceinline__ Eight unpack(uint4 r)
{
    return {{f2(bf16_lo(r.x), bf16_lo(r.y)), f2(bf16_lo(r.z), bf16_lo(r.w))},
            {f2(bf16_hi(r.x), bf16_hi(r.y)), f2(bf16_hi(r.z), bf16_hi(r.w))}};
}

// The lane's coefficients: y = (a ca + b nsb, a sa + b cb).
struct Turn {
    F2 ca[2], nsb[2], sa[2], cb[2];
};

__device__ __forceinline__ Turn turn_of(float4 c01, float4 c23, const Eight &w)
{
    const F2 c[2] = {f2(c01.x, c01.z), f2(c23.x, c23.z)};
    const F2 s[2] = {f2(c01.y, c01.w), f2(c23.y, c23.w)};
    const F2 minus = f2(-1.f, -1.f);
    Turn t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        t.ca[i] = mul2(w.a[i], c[i]);
        t.sa[i] = mul2(w.a[i], s[i]);
        t.cb[i] = mul2(w.b[i], c[i]);
        t.nsb[i] = mul2(minus, mul2(w.b[i], s[i]));
    }
    return t;
}

// Without a rotation the other value of a pair stays out of it (0 times an
// infinity would be NaN).
__device__ __forceinline__ void apply(Eight &x, const Turn &t, bool rotate)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const F2 a = x.a[i], b = x.b[i];
        if (!rotate) {
            x.a[i] = mul2(a, t.ca[i]);
            x.b[i] = mul2(b, t.cb[i]);
            continue;
        }
        x.a[i] = fma2(a, t.ca[i], mul2(b, t.nsb[i]));
        x.b[i] = fma2(a, t.sa[i], mul2(b, t.cb[i]));
    }
}

// rsqrt(mean(x^2) + eps) over the group.
template <int D>
__device__ __forceinline__ float norm_factor(const Eight &x, float eps)
{
    F2 s = mul2(x.a[0], x.a[0]);
    s = fma2(x.a[1], x.a[1], s);
    s = fma2(x.b[0], x.b[0], s);
    s = fma2(x.b[1], x.b[1], s);
    const float2 p = parts(s);
    return rsqrtf(group_sum<D / 8>(p.x + p.y) * (1.f / D) + eps);
}

__device__ __forceinline__ uint4 pack(const Eight &x, float f)
{
    const F2 ff = f2(f, f);
    const float2 a0 = parts(mul2(x.a[0], ff)), a1 = parts(mul2(x.a[1], ff));
    const float2 b0 = parts(mul2(x.b[0], ff)), b1 = parts(mul2(x.b[1], ff));
    return make_uint4(pack_bf16x2(a0.x, b0.x), pack_bf16x2(a0.y, b0.y),
                      pack_bf16x2(a1.x, b1.x), pack_bf16x2(a1.y, b1.y));
}

// x f as codes and the scale byte of the group's vector.
template <int D>
__device__ __forceinline__ uint2 quantise(const Eight &x, float f, int &sb)
{
    const float2 a0 = parts(x.a[0]), a1 = parts(x.a[1]), b0 = parts(x.b[0]), b1 = parts(x.b[1]);
    const float y[8] = {a0.x, b0.x, a0.y, b0.y, a1.x, b1.x, a1.y, b1.y};
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        amax = fmaxf(amax, fabsf(y[j]));
    amax = group_max<D / 8>(amax) * f;
    sb = q8_scale_byte(amax);
    // (a power of two: x (f 2^-e) rounds as (x f) 2^-e does)
    return q8_encode8(y, f, sb, amax == INFINITY);
}

// A block takes GROUPS / p.width tokens, p.width groups (a power of two) each.
template <int D, bool Q8, bool EXTEND>
__global__ void __launch_bounds__(kMaxThreads, 3) token_write_kernel(const TokenWriteParams p)
{
    constexpr int LANES = D / 8;             // lanes of a head vector
    constexpr int kQ = EXTEND ? kQExtend : kQAppend;
    grid_dependency_wait();
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int at_once = (int)blockDim.x / LANES >> p.width_shift;
    const int t0 = blockIdx.x * at_once, tok = group >> p.width_shift;
    const int nt = min(at_once, p.T - t0);
    const int width = 1 << p.width_shift, v0 = group & (width - 1);
    // (a group behind the last token reads that token and writes nothing)
    const size_t t = (size_t)(t0 + min(tok, nt - 1));
    const __nv_bfloat16 *q = p.q + t * p.q_stride + lane * 8;
    const __nv_bfloat16 *k = p.k + t * p.k_stride + lane * 8;
    const __nv_bfloat16 *v = p.v + t * p.v_stride + lane * 8;

    // (a vector past the last keeps what it held and is not stored)
    auto load = [&](uint4 &to, const __nv_bfloat16 *src, int h, int H) {
        if (h < H)
            to = __ldcs(reinterpret_cast<const uint4 *>(src + h * D));
    };
    // the first vectors do not wait for the look-up
    uint4 rq[kQ] = {}, rk[kKv] = {}, rv[kKv] = {};
#pragma unroll
    for (int u = 0; u < kQ; ++u)
        load(rq[u], q, v0 + u * width, p.Hq);
#pragma unroll
    for (int u = 0; u < kKv; ++u) {
        load(rk[u], k, v0 + u * width, p.Hkv);
        load(rv[u], v, v0 + u * width, p.Hkv);
    }
    const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    uint4 wq = ones, wk = ones;
    if (p.q_norm != nullptr)
        wq = *(reinterpret_cast<const uint4 *>(p.q_norm) + lane);

    // (an extend reads the keys' weight when it needs it: its registers would spill,
    // 69.2 us in place of 67.1)
    if (!EXTEND && p.k_norm != nullptr)
        wk = *(reinterpret_cast<const uint4 *>(p.k_norm) + lane);
    TokenRow row = row_of_token<EXTEND>(p, (int)t);
    const int page = row.at >= 0 ? p.kv_indices[row.at] : -1;
    grid_launch_dependents();
    float4 c01 = make_float4(1.f, 0.f, 1.f, 0.f), c23 = c01;
    if (p.rope != nullptr && row.pos >= 0 && row.bad == 0) {
        const float4 *cs =
            reinterpret_cast<const float4 *>(p.rope + (size_t)row.pos * D) + lane * 2;
        c01 = cs[0];
        c23 = cs[1];
    }
    if (row.pos >= 0 && (page < 0 || page >= p.num_pages))
        row.bad |= kFlagBadPage;
    if (row.bad != 0 && lane == 0 && v0 == 0 && p.status != nullptr)
        atomicOr(p.status, row.bad);
    const bool live = tok < nt && row.pos >= 0 && row.bad == 0;
    const long long slot = (long long)page * p.page_size + row.in_page;

    // query heads; every lane runs the same rounds, as the shuffles need whole warps
    {
        const Turn turn = turn_of(c01, c23, unpack(wq));
        __nv_bfloat16 *dst = p.q_out + (t * p.Hq) * D + lane * 8;
        for (int h0 = 0; h0 < p.Hq; h0 += kQ * width) {
#pragma unroll
            for (int u = 0; u < kQ; ++u) {
                const int h = h0 + u * width + v0;
                Eight x = unpack(rq[u]);
                load(rq[u], q, h + kQ * width, p.Hq);
                const float f = p.q_norm != nullptr ? norm_factor<D>(x, p.norm_eps) : 1.f;
                apply(x, turn, p.rope != nullptr);
                if (live && h < p.Hq)
                    *reinterpret_cast<uint4 *>(dst + h * D) = pack(x, f);
            }
        }
    }
    // K and V heads
    if (EXTEND && p.k_norm != nullptr)
        wk = *(reinterpret_cast<const uint4 *>(p.k_norm) + lane);
    // (codes: a key's products with the weight are formed by themselves, exactly, 16
    // bits of 24: of 4.9 M codes 4.6 lie across a tie from the 64-bit ones, 5.3 with
    // the weight in the coefficients, 7.7 in plain 32-bit operations, at the same time)
    const Eight wk8 = unpack(wk);
    const Turn turn = turn_of(c01, c23, Q8 ? unpack(ones) : wk8);
    for (int h0 = 0; h0 < p.Hkv; h0 += kKv * width) {
#pragma unroll
        for (int u = 0; u < kKv; ++u) {
            const int h = h0 + u * width + v0;
            const uint4 vraw = rv[u];
            Eight x = unpack(rk[u]);
            load(rk[u], k, h + kKv * width, p.Hkv);
            load(rv[u], v, h + kKv * width, p.Hkv);
            const float f = p.k_norm != nullptr ? norm_factor<D>(x, p.norm_eps) : 1.f;
            if constexpr (Q8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    x.a[i] = mul2(x.a[i], wk8.a[i]);
                    x.b[i] = mul2(x.b[i], wk8.b[i]);
                }
            }
            apply(x, turn, p.rope != nullptr);
            const bool store = live && h < p.Hkv;
            const size_t head = (size_t)slot * p.Hkv + h;
            if constexpr (Q8) {
                int sk, sv;
                const uint2 kc = quantise<D>(x, f, sk);
                const uint2 vc = quantise<D>(unpack(vraw), 1.f, sv);
                if (store) {
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.k_pool) + head * D +
                                               lane * 8) = kc;
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.v_pool) + head * D +
                                               lane * 8) = vc;
                    if (lane == 0) {
                        p.k_scale[head] = (uint8_t)sk;
                        p.v_scale[head] = (uint8_t)sv;
                    }
                }
            } else if (store) {
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.k_pool) + head * D +
                                           lane * 8) = pack(x, f);
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.v_pool) + head * D +
                                           lane * 8) = vraw;
            }
        }
    }
}

template <int D, bool Q8, bool EXTEND>
cudaError_t launch(const TokenWriteParams &params, cudaStream_t stream)
{
    constexpr int kLanes = D / 8;
    TokenWriteParams p = params;
    // As many groups a token as it has vectors of a kind, for few tokens; with
    // more, fewer (of 8 vectors at least: with 4, 16,384 tokens of 32 heads of 128
    // take 74.7 us in place of 67.1; with 16, they take 66.6, 9,537 of D = 64 23.9 in
    // place of 21.6), which then share the coefficients among more vectors.
    const int heads = p.Hq > p.Hkv ? p.Hq : p.Hkv;
    p.width_shift = 0;
    while (kLanes << p.width_shift < kMaxThreads && (1 << p.width_shift) < heads)
        ++p.width_shift;
    while (p.width_shift > 0 && (heads >> p.width_shift) < 8 &&
           (long long)p.T * (kLanes << p.width_shift >> 1) >= kManyThreads)
        --p.width_shift;
    const int wide = kLanes << p.width_shift;            // threads of a token
    const int threads = wide > kMinThreads ? wide : kMinThreads;
    const unsigned at_once = threads / wide;
    const unsigned blocks = ((unsigned)p.T + at_once - 1) / at_once;
    return launch_pdl(token_write_kernel<D, Q8, EXTEND>, dim3(blocks), dim3(threads), 0, stream, p);
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
