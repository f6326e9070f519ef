// pkv_q8_decode.cu -- decode attention over the 8-bit cache.
//
// out[b, h] = sum_t w_t V_t / sum_t w_t, w_t = exp(scale q.K_t - max), with
// K_t = 2^ek_t code, V_t = 2^ev_t code of the token's kv head.  A step reads
// every cached token once and does 4 Hq/Hkv D operations for 2 D + 2 bytes,
// so it is bound by memory; the work is split over the cache's length as in
// the bf16 decode (pkv_fused.cu): one persistent block per SM takes an equal
// range of all rows' tokens laid end to end, producer warps stream the tokens
// of HPC kv heads into a ring of shared-memory stages, and the piece combine
// joins the rows that several blocks share.
//
// What the 8-bit cache changes:
//  - Half the bytes a token means twice the tokens a second, so the tensor
//    products must waste less: here the tokens are the M rows of the
//    products (S^T = K Q^T, O^T = V^T P^T, m16n8k16) and the query heads the
//    eight columns, which a group of 8 heads fills and a group of 4 fills
//    half -- half the products and half the accumulators of heads as rows.
//    NT = 2 column tiles serve groups of 9 to 16 heads.
//  - Codes become f16 exactly (one cvt for two codes).  q is scaled by a
//    power of two to the top of f16's range, which keeps the eight significant
//    bits of every element down to 2^-32 of its head's largest (smaller ones
//    are off by 2^-40 of the largest); that power and the softmax scale go into
//    the score's factor in fp32.  (e4m3 x e4m3 products, with q and the weights
//    as two codes each, were slower: 62.8 us for the serving batch below, at
//    twice the tensor pipe's time -- this GPU makes them out of f16 products.)
//  - Both scales act on the scores: x_t = 2^ek_t (s_t c) and y_t = x_t + ev_t
//    in the log2 domain.  The weights used for O are 2^(y_t - base), base
//    following the largest y_t; the sum of softmax weights takes each of them,
//    in fp32, times 2^-ev_t (a power of two, exact).  Both sums carry 2^-base.
//    A weight is rounded to f16 for the product: to 11 significant bits, or,
//    under f16's normal range, to steps of 2^-24.  base is therefore kept 7
//    under the largest y_t, which leaves those steps at 2^-31 of the largest
//    weight: a long tail of small weights still adds up.  A token 2^32 below
//    the largest is lost from O, which shows where all larger ones have zero
//    codes in a channel.
//  - base is raised only when some y_t exceeds it by more than 15: a weight is
//    then at most 2^15 (f16 ends at 2^16) and the usual tile needs no maximum
//    over its lanes and no rescaling.
//  - Short rows (kQ8WholeBytes) are not split: a block takes whole rows and
//    writes their outputs, and there is no combine.
//  - A kv head has WPH = 8 / HPC warps, which take 16 tokens each of every
//    stage and have sums of their own, joined in pairs through shared memory at
//    the end of a piece.  A warp takes two stages at a time: the products and
//    exponentials of one overlap those of the other.
//  - Copies.  The producers' lanes copy 16 bytes each (cp.async), 32 lines of
//    consecutive tokens' rows at a time, and permute the 16-byte units of a row
//    so that eight tokens' vectors of a head are in different banks.  It serves
//    every page size and head count alike.  Copies by the copy engine were
//    slower: one bulk copy a token, as the bf16 decode makes them, sets the pace
//    at 1 KB a copy (86 us of copies alone for 322 MB, the serving batch of 128,
//    against 47.5 us at the measured copy bandwidth; at 64 bytes a copy, seven
//    times this kernel's time); boxes of 16 tokens x 128 bytes x heads took
//    59.4 us for that batch against 58.3, 20.4 against 20.0 for a row of 32,768
//    tokens, 54.5 against 44.4 for one kv head of 128, and no odd pages.
//
// Measured (CUDA-graph replay, K and V larger than L2 or rotating): 128 rows,
// lognormal, 154,103 tokens, 64 over 8 heads of 128, 322 MB: 57.3 us, 5,620 GB/s,
// 83% of the copy bandwidth (0.4 us less with the products left out: the copies
// set the pace; 53.2 without the combine); one row of 32,768: 19.6 us, 10 of them
// the stream, 3.5 the combine and its launch; 8 rows of 513 to 1,025, heads of 64:
// 8.7 us, latency (2.8 the combine).
#include <cmath>

#include "pkv_partition.cuh"
#include "pkv_q8.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;                 // consumer warps
constexpr float kRaise = 15.f;            // how far a score may exceed its base
constexpr float kUnder = 7.f;             // a raised base's distance to the largest score

template <int D, int HPC, int NT>
struct Q8Cfg {
    static constexpr int kWph = kWarps / HPC;         // warps of a kv head
    static constexpr int kTok = 16 * kWph;            // tokens of a stage
    // stages a warp takes at a time: two chains of products and exponentials
    // to overlap, where the registers allow it
    static constexpr int kTake = NT == 1 ? 2 : 1;
    // producer warps, a stage each in turn (of 2, 3 and 4, as far as the stages
    // are a multiple: 66.4 us with 4 and four stages, 58.3 with 3 and six for the
    // serving batch at D = 128; one kv head of 64: 69 us with 3, 52 with 4)
    static constexpr int kProducers = D == 64 ? 4 : 3;
    static constexpr int kThreads = (kWarps + kProducers) * 32;
    static constexpr int kRowBytes = HPC * D;         // one token, HPC kv heads
    static constexpr int kStageBytes = 2 * kTok * kRowBytes;
    static constexpr int kScaleBytes = 2 * kTok * 8;  // 8 bytes a token, K then V
    // joining parts: half of them leave half of their registers, a slot a warp
    static constexpr int kJoinFloats = NT * (D / 16 * 2 + 2);
    static constexpr int kJoinBytes = kWph == 1 ? 0 : kWarps / 2 * kJoinFloats * 32 * 4;
    static constexpr int kFixedBytes = kJoinBytes + (kQ8MaxRows + 1) * 4 + 16;
    static constexpr int kStagesFit =
        (kSmemLimit - kFixedBytes) / (kStageBytes + kScaleBytes + 16);
    // A multiple of the producers: a slot then always belongs to the same one.
    // Otherwise a producer could reach a slot before another had filled it for
    // its previous use, and take the parity of the use before that for its own.
    static constexpr int kStages =
        (kStagesFit > 10 ? 10 : kStagesFit) / kProducers * kProducers;
    static_assert(kStages >= 4 && kStages % kProducers == 0, "a slot has one producer");
    static constexpr int kScaleOffset = kStages * kStageBytes;
    static constexpr int kJoinOffset = kScaleOffset + kStages * kScaleBytes;
    static constexpr int kBarOffset = kJoinOffset + kJoinBytes;
    static constexpr int kAbortOffset = kBarOffset + 2 * kStages * 8;
    static constexpr int kPrefixOffset = kAbortOffset + 16;
    static constexpr int kSmemBytes = kPrefixOffset + (kQ8MaxRows + 1) * 4;
    static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
    static_assert(kStageBytes % 1024 == 0, "swizzled rows");
    static_assert(kJoinBytes % 16 == 0, "alignment");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two floats to f16x2, the first in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float exp2_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// This thread's earlier cp.async copies arrive on `bar` when they have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// 16 bytes global -> shared.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(src), "l"(policy)
                 : "memory");
}

// Four or eight bytes global -> shared, of which the first `bytes` are read
// (the others are zero).
template <int SIZE>
__device__ __forceinline__ void cp_async(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src),
                 "n"(SIZE), "r"(bytes)
                 : "memory");
}

template <int D, int HPC, int NT>
__global__ void __launch_bounds__(Q8Cfg<D, HPC, NT>::kThreads, 1)
    decode_q8_kernel(const __grid_constant__ FusedParams p)
{
    using C = Q8Cfg<D, HPC, NT>;
    constexpr int kProducers = C::kProducers;
    constexpr int NST = C::kStages;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    uint64_t *empty = full + NST;
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kAbortOffset);
    int *prefix = reinterpret_cast<int *>(smem + C::kPrefixOffset);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const int Bv = p.Bv;
    // byte b of token t's row, 16-byte units permuted within 128 bytes so
    // that the units of eight tokens at one column are in different banks
    auto line_addr = [](int t, int b) {
        return (uint32_t)(t * C::kRowBytes + b) ^
               (uint32_t)((C::kRowBytes >= 128 ? t : t >> 1) & 7) << 4;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 33);     // a producer warp, and each of its lanes' copies
            mbar_init(&empty[i], kWarps);
        }
        fence_mbar_init();
        *abort = 0;
    }
    grid_dependency_wait();

    // the partition, from the step's plan or computed here (as in pkv_fused.cu);
    // or whole rows, of which this block takes every gridDim.x-th: its row r
    // (of n_rows) is virtual row row_of(r)
    const int n_rows = p.whole_rows ? (Bv - cta + (int)gridDim.x - 1) / (int)gridDim.x : Bv;
    auto row_of = [&](int r) { return p.whole_rows ? cta + r * (int)gridDim.x : r; };
    bool planned = false;
    if (p.whole_rows) {
        row_prefix(p, prefix, n_rows, row_of, true);
    } else if (p.plan != nullptr) {
        planned = plan_fits(p.plan, (int)gridDim.x, Bv, p.B, p.page_size, p.row_cost);
        for (int i = threadIdx.x; i <= Bv; i += C::kThreads)
            prefix[i] = p.plan[kPlanHeaderInts + i];
        __syncthreads();
    }
    if (!planned && !p.whole_rows)
        row_prefix(p, prefix, cta == 0);

    const unsigned T = (unsigned)prefix[n_rows];
    const unsigned Gu = active_blocks(T, gridDim.x);
    const int G = (int)Gu;

    // rows with no tokens: zero output, no pieces (owner: block r mod grid)
    for (int r = p.whole_rows ? 0 : cta; r < n_rows; r += p.whole_rows ? 1 : gridDim.x) {
        if (prefix[r + 1] == prefix[r]) {
            const int b = row_of(r) % p.B, hg = row_of(r) / p.B;
            uint4 *o = reinterpret_cast<uint4 *>(
                p.out + ((size_t)b * p.Hq + (size_t)hg * HPC * p.n_rep) * D);
            for (int i = threadIdx.x; i < HPC * p.n_rep * D / 8; i += blockDim.x)
                o[i] = make_uint4(0u, 0u, 0u, 0u);
            if (threadIdx.x == 0 && !planned && !p.whole_rows) {
                p.row_info[2 * r] = 0;
                p.row_info[2 * r + 1] = 0;
            }
        }
    }
    // an unplanned call leaves its partition behind as the step's plan (the prefix
    // sums and the rows' pieces: this kernel reads no blocks' entries)
    if (p.plan_out != nullptr && cta == 0) {
        for (int i = threadIdx.x; i <= Bv; i += blockDim.x)
            p.plan_out[kPlanHeaderInts + i] = prefix[i];
        if (threadIdx.x == 0) {
            p.plan_out[0] = (int)T;
            p.plan_out[1] = G;
            p.plan_out[2] = (int)gridDim.x;
            p.plan_out[3] = Bv;
            p.plan_out[4] = p.B;
            p.plan_out[5] = p.page_size;
            p.plan_out[6] = p.row_cost;
        }
    }
    const unsigned t_q = T / Gu, t_r = T % Gu;
    // (T < 2^31)
    const int start = p.whole_rows ? 0 : (int)(t_q * cta + t_r * (unsigned)cta / Gu);
    const int end = p.whole_rows
                        ? (int)T
                        : (int)(t_q * (cta + 1) + t_r * (unsigned)(cta + 1) / Gu);
    if ((cta >= G && !p.whole_rows) || start >= end)
        return;
    const int r0 = first_row(prefix, n_rows, start);

    if (warp >= kWarps) {
        // ======================= producer warps ===========================
        // Stage i belongs to warp i % kProducers.  Lane l looks up the stage's
        // tokens l, 32 + l, ... and copies their scales; the copies of the codes
        // take the tokens' slots from it.
        const int pw = warp - kWarps;
        const uint64_t policy = policy_evict_first();
        const size_t scale_bytes = (size_t)p.num_pages * p.page_size * p.Hkv;
        constexpr int IDS = (C::kTok + 31) / 32;      // page ids a lane holds
        int it = 0;
        bool aborted = false;
        auto page_of_tok = [&](int t) {
            return p.ps_shift >= 0 ? (t >> p.ps_shift) : (t / p.page_size);
        };
        for (int r = r0; r < n_rows && !aborted; ++r) {
            // [lo, hi): the positions of the row's tokens
            const int lo = prefix[r] + p.row_cost, hi = prefix[r + 1];
            if (lo >= end)
                break;
            if (hi == prefix[r])
                continue;
            const int t0 = max(start, lo) - lo, t1 = min(end, hi) - lo;
            const int b = row_of(r) % p.B, hg = row_of(r) / p.B;
            const int pg0 = p.kv_indptr[b];
            int npg = p.kv_indptr[b + 1] - pg0;
            if (pg0 < 0 || npg < 0 || pg0 > p.num_indices - npg)
                npg = 0;                               // a table changed since the plan
            // the table's entry for this lane's token k of the stage at tok
            auto load_id = [&](int tok, int k) {
                const int at = k * 32 + lane;
                const bool there = at < C::kTok && tok + at < t1;
                const int pi = page_of_tok(there ? tok + at : 0);
                return there && pi < npg ? p.kv_indices[pg0 + pi] : 0;
            };
            // the ids of this warp's next stage are loaded a stage ahead
            int ids[IDS];
            const int skip = (pw - it % kProducers + kProducers) % kProducers;
#pragma unroll
            for (int k = 0; k < IDS; ++k)
                ids[k] = load_id(t0 + skip * C::kTok, k);
            for (int tok = t0; tok < t1; tok += C::kTok, ++it) {
                if (it % kProducers != pw)
                    continue;
                const int st = it % NST;
                int next[IDS];
#pragma unroll
                for (int k = 0; k < IDS; ++k)
                    next[k] = load_id(tok + kProducers * C::kTok, k);
                if (it >= NST) {
                    // (a consumer that gave up releases its stages without having
                    // waited for them, after it has set the abort word)
                    const bool ok =
                        mbar_wait_or_abort(&empty[st], (uint32_t)(((it / NST) - 1) & 1),
                                           p.handoff_wait_ns, abort) &&
                        !*abort;
                    if (!__all_sync(kFull, ok)) {
                        aborted = true;
                        if (lane == 0) {
                            *abort = 1;
                            atomicOr(p.status, kFlagTimeout);
                        }
                        break;
                    }
                }
                unsigned char *stage = smem + st * C::kStageBytes;
                unsigned char *sc0 = smem + C::kScaleOffset + st * C::kScaleBytes;
                const int nvalid = min(C::kTok, t1 - tok);
                // a page id of a token that is there, checked
                auto checked = [&](int page, bool there) {
                    if (page < 0 || page >= p.num_pages) {
                        if (there)
                            atomicOr(p.status, kFlagBadPage);
                        page = 0;
                    }
                    return page;
                };
                // a token's HPC scale bytes of one pool
                auto copy_scale = [&](const uint8_t *scales, int row, size_t head) {
                    unsigned char *sc = sc0 + row * 8;
                    if constexpr (HPC == 8) {
                        cp_async<8>(sc, scales + head, 8);
                    } else if constexpr (HPC == 4) {
                        cp_async<4>(sc, scales + head, 4);
                    } else {
                        // the aligned word around the HPC bytes, and where they are in it
                        const size_t word = head & ~(size_t)3;
                        const size_t left = scale_bytes - word;
                        cp_async<4>(sc, scales + word, left < 4 ? (int)left : 4);
                        sc[4] = (unsigned char)(head & 3);
                    }
                };
                constexpr int CH = C::kRowBytes / 16;      // 16-byte lines of a token
                const size_t line0 = (size_t)hg * C::kRowBytes;
                const unsigned tok_bytes = (unsigned)(p.Hkv * D);
#pragma unroll
                for (int k = 0; k < IDS; ++k) {
                    if (k * 32 >= nvalid)
                        break;
                    const int row = k * 32 + lane, t = tok + row;
                    const bool there = row < nvalid;
                    const int page = checked(ids[k], there);
                    const int slot = page * p.page_size +
                                     (there ? t - page_of_tok(t) * p.page_size : 0);
                    if (there) {
                        const size_t head = (size_t)slot * p.Hkv + (size_t)hg * HPC;
                        copy_scale(p.k_scale, row, head);
                        copy_scale(p.v_scale, C::kTok + row, head);
                    }
                    // 32 lines at a time, 32 / CH tokens' (or part of one): line
                    // 32 j + lane lies at byte 16 (32 j + lane) of these tokens'
                    // rows, its swizzle that of the lane and of j (no carry)
                    constexpr int ROUNDS = (C::kTok < 32 ? C::kTok : 32) * CH / 32;
                    constexpr int HALF = C::kRowBytes >= 128 ? 0 : 1;
                    const uint32_t lane_key = (uint32_t)((lane / CH) >> HALF & 7) << 4;
                    const uint32_t to = smem_addr(stage) + k * 32 * C::kRowBytes;
#pragma unroll
                    for (int j = 0; j < ROUNDS; ++j) {
                        const int from = (j * 32 + lane) / CH, ch = (j * 32 + lane) % CH;
                        const unsigned s_ = (unsigned)__shfl_sync(kFull, slot, from);
                        if (k * 32 + from < nvalid) {
                            const size_t off = (size_t)s_ * tok_bytes + (line0 + ch * 16);
                            const uint32_t dst =
                                to + j * 512 +
                                ((lane * 16u) ^ lane_key ^
                                 (uint32_t)((j * 32 / CH) >> HALF & 7) << 4);
                            cp_async16(dst, p.k_codes + off, policy);
                            cp_async16(dst + C::kTok * C::kRowBytes, p.v_codes + off, policy);
                        }
                    }
                }
                cp_async_arrive(&full[st]);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[st]);
#pragma unroll
                for (int k = 0; k < IDS; ++k)
                    ids[k] = next[k];
            }
        }
        // Let this warp's copies land before it exits, with the full time
        // limit: a consumer that gave up skips its stages, and the block must
        // not exit while a copy into its shared memory is in flight.
        for (int k = (it > NST ? it - NST : 0); k < it; ++k)
            if (k % kProducers == pw)
                (void)mbar_wait_bounded(&full[k % NST], (uint32_t)((k / NST) & 1));
        grid_launch_dependents();
        return;
    }

    // ========================= consumer warps ===============================
    const int hw = warp % HPC, tg = warp / HPC;   // kv head, its part
    const int g = lane >> 2, c = lane & 3;
    const uint32_t smem_s = smem_addr(smem);
    // Matrix loads: lane l addresses token l % 16 of the warp's 16 and the
    // 16-byte column l / 16 of each two.
    // the 32-byte column i of a row whose first is at `addr`: the swizzle is in
    // the same bits
    auto column = [](uint32_t addr, int i) { return addr ^ (i * 32u); };
    const uint32_t k_off =
        smem_s + line_addr(tg * 16 + (lane & 15), hw * D + (lane >> 4) * 16);
    const uint32_t v_off = k_off + C::kTok * C::kRowBytes;
    // lane (g, c)'s elements of head 8 nt + g of the heads from qrow0 on (plain
    // loads, here and for the tables: the grid before may have written them
    // while this one was already on the GPU)
    auto load_q = [&](uint2 (&raw)[D / 16], size_t qrow0, int nt) {
        const int h = nt * 8 + g;
        const __nv_bfloat16 *src = p.q + (qrow0 + h) * D;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            raw[j] = h < p.n_rep ? reinterpret_cast<const uint2 *>(src)[j * 4 + c]
                                 : make_uint2(0u, 0u);
    };
    int it = 0;
    bool aborted = false;

    for (int r = r0; r < n_rows; ++r) {
        const int lo = prefix[r] + p.row_cost, hi = prefix[r + 1];
        if (lo >= end)
            break;
        if (hi == prefix[r])
            continue;
        const int t0 = max(start, lo) - lo, t1 = min(end, hi) - lo;
        const int b = row_of(r) % p.B, hg = row_of(r) / p.B;
        const size_t qrow0 = (size_t)b * p.Hq + (size_t)(hg * HPC + hw) * p.n_rep;

        // q as the products' B operand: lane (g, c) holds elements 4c .. 4c + 3
        // of each 16 of head g, the order in which a K word's four codes come
        uint32_t qf[NT][D / 16][2];
        float cq[NT][2];                   // factors of heads 2c, 2c + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint2 raw[D / 16];
            load_q(raw, qrow0, nt);
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(raw[j].x)), fabsf(bf16_hi(raw[j].x))),
                                         fmaxf(fabsf(bf16_lo(raw[j].y)), fabsf(bf16_hi(raw[j].y)))));
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
            // 2^(15 - n), n the exponent of amax, both powers kept in the normal range
            // (the largest, 2^16 less a bf16 step, is within f16; infinity stays)
            const int n = min(max((int)(__float_as_uint(amax) >> 23) - 127, -111), 127);
            const float down = __uint_as_float((unsigned)(127 + 15 - n) << 23);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                qf[nt][j][0] = pack_f16x2(bf16_lo(raw[j].x) * down, bf16_hi(raw[j].x) * down);
                qf[nt][j][1] = pack_f16x2(bf16_lo(raw[j].y) * down, bf16_hi(raw[j].y) * down);
            }
            const float up = __uint_as_float((unsigned)(127 - 15 + n) << 23) * p.scale_log2;
            cq[nt][0] = __shfl_sync(kFull, up, (2 * c) * 4);
            cq[nt][1] = __shfl_sync(kFull, up, (2 * c + 1) * 4);
        }

        float m_run[NT][2], l_run[NT][2];
        float oacc[NT][D / 16][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m_run[nt][0] = m_run[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                oacc[nt][j][0] = oacc[nt][j][1] = oacc[nt][j][2] = oacc[nt][j][3] = 0.f;
        }

        for (int tok = t0; tok < t1;) {
            constexpr int U = C::kTake;
            // this turn's stages: U, or as many as the piece has left
            const int take = U == 1 ? 1 : min(U, (t1 - tok + C::kTok - 1) / C::kTok);
            uint32_t stage[U];
            const unsigned char *sc[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int st = (it + u) % NST;
                stage[u] = (uint32_t)st * C::kStageBytes;
                sc[u] = smem + C::kScaleOffset + st * C::kScaleBytes + tg * 16 * 8;
                if (!aborted && u < take) {
                    const bool ok = mbar_wait_or_abort(&full[st], (uint32_t)(((it + u) / NST) & 1),
                                                       p.handoff_wait_ns, abort);
                    if (!__all_sync(kFull, ok)) {
                        aborted = true;
                        if (lane == 0) {
                            *abort = 1;
                            atomicOr(p.status, kFlagTimeout);
                        }
                    }
                }
            }
            // tokens [v0, v1) of this warp's 16 of the first stage belong to the
            // piece, [v0, v1) - u kTok of stage u (none of a stage not taken)
            const int v0 = t0 - tok - tg * 16, v1 = t1 - tok - tg * 16;
            if (!aborted && v1 > 0 && v0 < 16 + (U - 1) * C::kTok) {
                // S^T = K q, in two sums: a word of four codes gives two pairs of f16,
                // places 2c, 2c + 1 and 2c + 8, 2c + 9 of a product's depth
                float sacc[NT][U][2][4] = {};
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        uint32_t r0_, r1_, r2_, r3_;
                        ldmatrix_x4(r0_, r1_, r2_, r3_, column(stage[u] + k_off, i));
                        const uint32_t a0[4] = {f16x2_of_e4m3x2(r0_), f16x2_of_e4m3x2(r1_),
                                                f16x2_of_e4m3x2_hi(r0_), f16x2_of_e4m3x2_hi(r1_)};
                        const uint32_t a1[4] = {f16x2_of_e4m3x2(r2_), f16x2_of_e4m3x2(r3_),
                                                f16x2_of_e4m3x2_hi(r2_), f16x2_of_e4m3x2_hi(r3_)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(sacc[nt][u][0], a0, qf[nt][2 * i][0], qf[nt][2 * i][1]);
                            mma_f16(sacc[nt][u][1], a1, qf[nt][2 * i + 1][0],
                                    qf[nt][2 * i + 1][1]);
                        }
                    }
                // the scales of this lane's tokens, rows g and g + 8
                float y[NT][U][4], inv_v[U][2];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const unsigned char *sk = sc[u] + (g + k * 8) * 8;
                        const unsigned char *sv = sk + C::kTok * 8;
                        const unsigned bk = HPC >= 4 ? sk[hw] : sk[(sk[4] & 3) + hw];
                        const unsigned bv = HPC >= 4 ? sv[hw] : sv[(sv[4] & 3) + hw];
                        const float fk = q8_scale(bk);
                        const float ev = __uint_as_float(0x4b000000u | bv) - 8388735.f;  // bv - 127
                        inv_v[u][k] = __uint_as_float((254u - bv) << 23);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int x = 2 * k + e;
                                y[nt][u][x] = fmaf(sacc[nt][u][0][x] + sacc[nt][u][1][x],
                                                   fk * cq[nt][e], ev);
                            }
                    }
                // some of the tokens are of no piece: no weight, and V's bytes (which
                // may be NaN) masked
                const bool cut = v0 > 0 || v1 < 16 + (U - 1) * C::kTok;
                unsigned sel[U][2];                    // byte selectors of V's words, below
#pragma unroll
                for (int u = 0; u < U; ++u)
                    sel[u][0] = sel[u][1] = 0x3120;
                if (cut) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        auto in = [&](int t) {
                            return t + u * C::kTok >= v0 && t + u * C::kTok < v1;
                        };
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (!in(g + k * 8)) {
                                inv_v[u][k] = 0.f;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    y[nt][u][2 * k] = y[nt][u][2 * k + 1] = -INFINITY;
                            }
                            // (selector 4: a zero byte)
                            sel[u][k] = (in(2 * c + k * 8) ? 0x0100u : 0x0404u) |
                                        (in(2 * c + 1 + k * 8) ? 0x3020u : 0x4040u);
                        }
                    }
                }
                bool raise = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            raise |= y[nt][u][x] > m_run[nt][x & 1] + kRaise;
                if (__any_sync(kFull, raise)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(y[nt][0][e], y[nt][0][e + 2]);
#pragma unroll
                            for (int u = 1; u < U; ++u)
                                mx = fmaxf(mx, fmaxf(y[nt][u][e], y[nt][u][e + 2]));
                            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                            const float mn = fmaxf(m_run[nt][e], mx - kUnder);
                            const float a = mn == -INFINITY ? 1.f : exp2_ftz(m_run[nt][e] - mn);
                            m_run[nt][e] = mn;
                            l_run[nt][e] *= a;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                oacc[nt][j][e] *= a;
                                oacc[nt][j][e + 2] *= a;
                            }
                        }
                }
                uint32_t pb[NT][U][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float base0 = m_run[nt][0] == -INFINITY ? 0.f : m_run[nt][0];
                    const float base1 = m_run[nt][1] == -INFINITY ? 0.f : m_run[nt][1];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            w[x] = exp2_ftz(y[nt][u][x] - (x & 1 ? base1 : base0));
                            l_run[nt][x & 1] = fmaf(w[x], inv_v[u][x >> 1], l_run[nt][x & 1]);
                        }
                        // S^T's layout has a token's heads in a lane, P^T's B operand a
                        // head's tokens: transpose the two 8 x 8 halves
                        pb[nt][u][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
                        pb[nt][u][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
                    }
                }
                // O^T += V^T P^T: a transposed 8-token x 16-byte matrix gives lane (g, c)
                // the codes (t, d), (t, d+1), (t+1, d), (t+1, d+1) of t = 2c, d = 2g:
                // swapping the middle two leaves the token pairs of column d and of
                // column d + 1
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        uint32_t r0_, r1_, r2_, r3_;
                        ldmatrix_x4_trans(r0_, r1_, r2_, r3_, column(stage[u] + v_off, i));
                        r0_ = __byte_perm(r0_, 0, sel[u][0]);
                        r1_ = __byte_perm(r1_, 0, sel[u][1]);
                        r2_ = __byte_perm(r2_, 0, sel[u][0]);
                        r3_ = __byte_perm(r3_, 0, sel[u][1]);
                        const uint32_t a0[4] = {f16x2_of_e4m3x2(r0_), f16x2_of_e4m3x2_hi(r0_),
                                                f16x2_of_e4m3x2(r1_), f16x2_of_e4m3x2_hi(r1_)};
                        const uint32_t a1[4] = {f16x2_of_e4m3x2(r2_), f16x2_of_e4m3x2_hi(r2_),
                                                f16x2_of_e4m3x2(r3_), f16x2_of_e4m3x2_hi(r3_)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(oacc[nt][2 * i], a0, pb[nt][u][0], pb[nt][u][1]);
                            mma_f16(oacc[nt][2 * i + 1], a1, pb[nt][u][0], pb[nt][u][1]);
                        }
                    }
            }
            __syncwarp();
            if (lane < take)
                mbar_arrive(&empty[(it + lane) % NST]);
            tok += take * C::kTok;
            it += take;
        }

        // ---- end of the piece: join the head's parts in pairs -----------------
        if constexpr (C::kWph > 1) {
            float *slots = reinterpret_cast<float *>(smem + C::kJoinOffset) + lane;
#pragma unroll
            for (int s = C::kWph / 2; s >= 1; s >>= 1)
#pragma unroll
                for (int e = 0; e < 2; ++e) {              // heads 2c, then 2c + 1
                    if (tg >= s && tg < 2 * s) {
                        float *to = slots + ((tg - s) * HPC + hw) * (C::kJoinFloats * 32);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            *to = m_run[nt][e], to += 32;
                            *to = l_run[nt][e], to += 32;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                *to = oacc[nt][j][e], to += 32;
                                *to = oacc[nt][j][e + 2], to += 32;
                            }
                        }
                    }
                    named_bar_sync(1, kWarps * 32);
                    if (tg < s) {
                        const float *from = slots + (tg * HPC + hw) * (C::kJoinFloats * 32);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float m = *from;
                            const float mn = fmaxf(m_run[nt][e], m);
                            const float base = mn == -INFINITY ? 0.f : mn;
                            const float fa = exp2_ftz(m_run[nt][e] - base), fb = exp2_ftz(m - base);
                            m_run[nt][e] = mn;
                            l_run[nt][e] = l_run[nt][e] * fa + from[32] * fb;
                            from += 64;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                oacc[nt][j][e] = oacc[nt][j][e] * fa + *from * fb;
                                oacc[nt][j][e + 2] = oacc[nt][j][e + 2] * fa + from[32] * fb;
                                from += 64;
                            }
                        }
                    }
                    named_bar_sync(1, kWarps * 32);
                }
        }
        if (tg != 0)
            continue;
        // oacc[nt][j][e]: head 8 nt + 2c + (e & 1), column 16 j + 2g + (e >> 1)
        const bool whole = t0 == 0 && t1 == hi - lo;
        if (t0 == 0 && warp == 0 && lane == 0 && !planned && !p.whole_rows) {
            p.row_info[2 * r] = cta;
            p.row_info[2 * r + 1] = whole ? 1 : block_of(hi - 1, T, G) - cta + 1;
        }
        const size_t slot0 = (size_t)(cta + r) * (HPC * p.n_rep) + (size_t)hw * p.n_rep;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nt][e], m = m_run[nt][e];
                l += __shfl_xor_sync(kFull, l, 4);
                l += __shfl_xor_sync(kFull, l, 8);
                l += __shfl_xor_sync(kFull, l, 16);
                const int h = nt * 8 + 2 * c + e;
                if (h >= p.n_rep)
                    continue;
                if (l != l)                  // NaN: kept through the combine
                    l = 1.f, m = 0.f;
                const float inv = l > 0.f ? 1.f / l : 0.f;
                if (whole) {
                    __nv_bfloat16 *o = p.out + (qrow0 + h) * D + 2 * g;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        *reinterpret_cast<uint32_t *>(o + 16 * j) =
                            pack_bf16x2(oacc[nt][j][e] * inv, oacc[nt][j][e + 2] * inv);
                } else {
                    float *o = p.o_part + (slot0 + h) * D + 2 * g;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        *reinterpret_cast<float2 *>(o + 16 * j) =
                            make_float2(oacc[nt][j][e] * inv, oacc[nt][j][e + 2] * inv);
                    if (g == 0)
                        reinterpret_cast<float2 *>(p.ml_part)[slot0 + h] =
                            l > 0.f ? make_float2(m * kLn2f, l) : make_float2(-INFINITY, 0.f);
                }
            }
    }
    grid_launch_dependents();
}

template <int D, int HPC, int NT>
cudaError_t launch(const FusedParams &p, int grid, cudaStream_t stream)
{
    using C = Q8Cfg<D, HPC, NT>;
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        cudaError_t r = cudaFuncSetAttribute(decode_q8_kernel<D, HPC, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmemBytes);
        if (r != cudaSuccess)
            return r;
        return cudaFuncSetAttribute(decode_q8_kernel<D, HPC, NT>,
                                    cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess)
        return e;
    return launch_pdl(decode_q8_kernel<D, HPC, NT>, dim3(grid), dim3(C::kThreads), C::kSmemBytes,
                      stream, p);
}

template <int D, int HPC>
cudaError_t launch_nt(const FusedParams &p, int grid, cudaStream_t stream)
{
    return p.n_rep <= 8 ? launch<D, HPC, 1>(p, grid, stream) : launch<D, HPC, 2>(p, grid, stream);
}

template <int D>
cudaError_t launch_d(const FusedParams &p, int grid, cudaStream_t stream)
{
    switch (p.hpc) {
    case 8:
        return launch_nt<D, 8>(p, grid, stream);
    case 4:
        return launch_nt<D, 4>(p, grid, stream);
    case 2:
        return launch_nt<D, 2>(p, grid, stream);
    default:
        return launch_nt<D, 1>(p, grid, stream);
    }
}

} // namespace

cudaError_t launch_decode_q8(const FusedParams &params, int D, int grid, cudaStream_t stream)
{
    FusedParams p = params;
    p.handoff_wait_ns = handoff_wait_ns();
    return D == 64 ? launch_d<64>(p, grid, stream) : launch_d<128>(p, grid, stream);
}

} // namespace pkv
