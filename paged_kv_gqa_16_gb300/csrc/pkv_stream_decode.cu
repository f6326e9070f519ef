// pkv_stream_decode.cu -- decode attention over the 4-bit cache, and through a
// sliding window over either that or the bf16 pools.
//
// out[b, h] = sum_t w_t V_t / sum_t w_t, w_t = exp(scale q.K_t - max), over the
// tokens t that the row's last one sees: all L, or with a window the last `window`
// and the first `sinks`.  A step reads each of them once, so it is bound by memory.
// The work is split as in the 8-bit decode (pkv_q8_decode.cu): one persistent block
// per SM takes an equal range of the seen tokens of all rows laid end to end;
// producer warps copy the tokens of HPC kv heads in 16-byte lines (2 KB rows: one bulk
// copy each) into a ring of stages, and the piece combine joins the rows that several
// blocks share.  The i-th seen token of a row is its token i for i < sinks, i + L -
// seen behind: only the producers know, as they look up each token's page, a stage of
// their own ahead, over the ends of rows too; several fill a stage together.  Pages without a seen token are not
// looked up.
//
// The tokens are the M rows of the products (S^T = K Q^T, O^T = V^T P^T, m16n8k16)
// and the query heads the eight columns; a kv head has WPH = 8 / HPC warps with sums
// of their own, joined at a piece's end.
//
// bf16 pools: K and V go into the products as they are, the weights are rounded to
// bf16 and summed as rounded.
//
// 4-bit cache: a 16-byte unit of a row is 32 codes of one scale.
//  - Scores: a lane's word of a unit is eight codes, four pairs of f16 (one
//    conversion each, exact).  The products of a unit have sums of their own, which
//    take the unit's scale in fp32: x = sum_u 2^ek_u s_u.  q is scaled by a power of
//    two to the top of f16's range, as in the 8-bit decode.
//  - Output: a transposed word holds four codes of two tokens; a token's weight is
//    multiplied with each unit's scale before it is rounded to f16 and transposed,
//    once a unit.  y = x + ev, ev the largest exponent of the token's units, decides
//    the base, so a weight of a unit is at most 2^15; under f16's normal range it is
//    rounded to steps of 2^-24, 2^-31 of the largest.
//
// What bounds it.  The windows over bf16 pools: memory.  The 4-bit cache: instructions.
// A warp makes 350 for 16 tokens of a head of 128, of which 160 go to the
// arithmetic-logic pipe at two cycles each (64 conversions, 16 to gather two tokens'
// codes, 16 for scales, 8 to round weights); of the kernel's time issue slots are busy
// 53%, that pipe 53%, the tensor cores 21%.  On the serving batch the copies alone take 35.6 us, the
// arithmetic alone 44, neither 18.
//
// Measured (CUDA-graph replay, K and V larger than L2 or rotating): 4 bits, 128 rows,
// lognormal, 154,103 tokens, 64 over 8 heads of 128, 168 MB: 47.7 us, 3,520 GB/s, 53% of
// the copy bandwidth (the 8-bit cache's 322 MB: 57.7, bf16's 631 MB: 97); one row of
// 32,768, 32 heads: 17.0 us; 32 rows through a window of 1,024 and 4 sinks: 17.0; 8 rows of
// 513 to 1,025, heads of 64: 8.6.  bf16, 128 rows of at most 1,028 seen tokens, 312 MB:
// 55.9 us, 5,580 GB/s, 84%; 64 rows of 4,100 seen tokens, 1,076 MB: 158.6 us, 6,785 GB/s.
#include <cmath>
#include <type_traits>

#include "pkv_decode.cuh"
#include "pkv_partition.cuh"
#include "pkv_q4.cuh"

namespace pkv {

namespace {

constexpr float kRaise = 15.f;            // how far a score may exceed its base

template <int BITS, int D, int HPC, int NT>
struct StreamCfg {
    static constexpr bool kCodes = BITS == 4;
    static constexpr int kWarps = 8;                      // consumer warps
    static constexpr int kWph = kWarps / HPC;             // warps of a kv head
    // Tiles of 16 tokens that a warp takes at a time: with two, the loop's steps serve
    // both (68 instructions of 700), and the products of one overlap the other's
    // exponentials.  The serving batch of 4 bits: 52.0 us, one tile 59.3, 16 warps of one
    // 57.9, four tiles 55.
    static constexpr int kTiles = kCodes && NT == 1 ? 2 : 1;
    static constexpr int kTok = 16 * kTiles * kWph;       // tokens of a stage
    // Rows of 2 KB go by one bulk copy each, with a pitch that spreads them over the
    // banks: a lane's instruction in place of four of a warp.  (Shorter ones would be
    // slower so: the copy engine takes about 24 copies a microsecond and SM.)
    static constexpr bool kBulk = BITS == 16 && HPC * D * BITS / 8 >= kBulkRowBytes;
    static_assert(!kBulk || kTok == 16, "a stage is one tile, zeroed to its end");
    // Producer warps, and how many fill a stage together, a part of its tokens each.
    // Together they bring the first stage sooner and issue more in flight: bf16, 512 rows
    // of 2048 tokens, 8 heads of D = 64, 402 us -> 330 with four a stage, one row of 64 8.0
    // -> 5.8; 8 heads of 128 by bulk copies, 76 rows of 256, 20.0 (three warps, a stage
    // each in turn) -> 17.0, one row of 64 7.2 -> 6.6, the windows' serving batch 56.8 ->
    // 55.9.  A stage of codes is smaller, and each share costs its own steps: two a
    // stage 17.45 us -> 17.1 for a row of 32768, 4 bits, and four 16.5, but a batch of 512
    // 166 us -> 198.  (Two tiles of heads at D = 128 take 437 us with three warps and 462
    // with four.)
    static constexpr int kProducers = BITS == 4 && kTok == 16 && D == 128 ? 3 : 4;
    static constexpr int kSplit = BITS == 16 ? 4 : kTok >= 32 ? 2 : 1;
    // Barriers of a full stage.  By bulk copies one for each of its producers: each can
    // then wait for its own copies, whatever the others did.
    static constexpr int kFulls = kBulk ? kSplit : 1;
    static constexpr int kShare = kTok / kSplit;           // tokens of a warp
    static constexpr int kTurn = kProducers / kSplit;      // stages from a warp's one to its next
    static constexpr int kThreads = (kWarps + kProducers) * 32;
    static constexpr int kHeadBytes = D * BITS / 8;
    static constexpr int kRowBytes = HPC * kHeadBytes;    // one token, HPC kv heads
    static constexpr int kPitch = kBulk ? kRowBytes + 16 : kRowBytes;
    static constexpr int kStageBytes = 2 * kTok * kPitch;
    // a token's scale bytes (of K, and of V), and its room for them
    static constexpr int kScaleRow = kCodes ? HPC * D / kQ4Group : 0;
    static constexpr int kScalePitch = kScaleRow == 2 ? 8 : kScaleRow;
    static constexpr int kScaleBytes = 2 * kTok * kScalePitch;
    // joining parts: half of them leave half of their registers, a slot a warp
    static constexpr int kJoinFloats = NT * (D / 16 * 2 + 2);
    static constexpr int kJoinBytes = kWph == 1 ? 0 : kWarps / 2 * kJoinFloats * 32 * 4;
    // the abort word and the producer warps' ends, 16 bytes for either
    static constexpr int kEndBytes = 32;
    static_assert(kProducers <= 4, "room for their ends");
    static constexpr int kFixedBytes = kJoinBytes + (kQ8MaxRows + 1) * 4 + 16 + kEndBytes;
    static constexpr int kStagesFit =
        (kSmemLimit - kFixedBytes) / (kStageBytes + kScaleBytes + 8 * (kFulls + 1));
    // A multiple of the turns: a slot then always belongs to the same producers.
    static constexpr int kStages = (kStagesFit > 12 ? 12 : kStagesFit) / kTurn * kTurn;
    static_assert(kStages >= 3 && kStages % kTurn == 0, "a slot has its producers");
    static_assert(!kBulk || (2 * kShare <= 32 && kTurn == 1), "a lane copies a row of K or of V");
    static_assert(kShare >= 4 && (kShare & (kShare - 1)) == 0, "no carry in the swizzle");
    static constexpr int kScaleOffset = kStages * kStageBytes;
    static constexpr int kJoinOffset = kScaleOffset + kStages * kScaleBytes;
    static constexpr int kBarOffset = kJoinOffset + kJoinBytes;
    static constexpr int kAbortOffset = kBarOffset + (((kFulls + 1) * kStages * 8 + 15) & ~15);
    static constexpr int kPrefixOffset = kAbortOffset + kEndBytes;
    static constexpr int kSmemBytes = kPrefixOffset + (kQ8MaxRows + 1) * 4;
    static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
    static_assert(kBulk || kStageBytes % 1024 == 0, "swizzled rows");
    static_assert(kScaleBytes % 16 == 0 && kJoinBytes % 16 == 0, "alignment");
};

// 16 bytes global -> shared, of which the first `bytes` are read (the others zero).
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void *src, int bytes,
                                                uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}

// d = A B, f16 products in fp32 (mma_f16 from zero: no registers to clear).
__device__ __forceinline__ void mma_f16_from_zero(float (&d)[4], const uint32_t (&a)[4],
                                                  uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Left shifts as products: the arithmetic-logic pipe, which makes the conversions,
// sets this kernel's pace, and the multiply-add pipe has time.  (The factors come
// from a place that the compiler does not see through.)
struct Shifts {
    uint32_t by4, by7, by12, by15, by16, by23;
};

__device__ __forceinline__ Shifts shifts()
{
    uint32_t one;
    asm volatile("mov.u32 %0, 1;" : "=r"(one));
    return {one << 4, one << 7, one << 12, one << 15, one << 16, one << 23};
}

// The bytes' low halves of a, their high halves of b.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xe4;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float fmax3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A transposed word holds four codes of two tokens, A0 .. A3 in its low half, B0 ..
// B3 in its high half.  `even` and `odd` hold (A0, B0), (A2, B2) and (A1, B1), (A3, B3)
// in bytes 2 and 3.
__device__ __forceinline__ void two_tokens(uint32_t w, const Shifts &by, uint32_t &even,
                                           uint32_t &odd)
{
    even = low_halves(w * by.by16, w * by.by4);
    odd = low_halves(w * by.by12, w);
}

template <int N>
using Const = std::integral_constant<int, N>;

// Byte B of a scale word as 2^(byte - 127) (infinity for 255).
template <int B>
__device__ __forceinline__ float scale_of(uint32_t w, const Shifts &by)
{
    if constexpr (B == 3)
        return __uint_as_float(__byte_perm(w, 0, 0x4443) * by.by23);
    const uint32_t at = w * (B == 0 ? by.by23 : B == 1 ? by.by15 : by.by7);
    return __uint_as_float(at & 0x7f800000u);
}

template <int BITS, int D, int HPC, int NT>
__global__ void __launch_bounds__(StreamCfg<BITS, D, HPC, NT>::kThreads, 1)
    stream_decode_kernel(const __grid_constant__ StreamParams sp)
{
    using C = StreamCfg<BITS, D, HPC, NT>;
    constexpr int kWarps = C::kWarps;
    constexpr int NST = C::kStages;
    constexpr int U = C::kTiles;
    constexpr int G32 = D / kQ4Group;             // scales of a head vector
    const FusedParams &p = sp.f;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    uint64_t *empty = full + NST * C::kFulls;
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kAbortOffset);
    int *prefix = reinterpret_cast<int *>(smem + C::kPrefixOffset);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const int Bv = p.Bv;
    // byte b of token t's row, 16-byte units permuted within 128 bytes so
    // that the units of eight tokens at one column are in different banks
    constexpr int kKeyShift = C::kRowBytes >= 128 ? 0 : C::kRowBytes == 64 ? 1 : 2;
    auto line_addr = [](int t, int b) {
        return C::kBulk ? (uint32_t)(t * C::kPitch + b)
                        : (uint32_t)(t * C::kRowBytes + b) ^
                              (uint32_t)((t >> kKeyShift) & 7) << 4;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            // a producer warp's lanes, or kSplit warps once and their lanes' copies
            for (int j = 0; j < C::kFulls; ++j)
                mbar_init(&full[i * C::kFulls + j], C::kBulk ? 32 : 33 * C::kSplit);
            mbar_init(&empty[i], kWarps);
        }
        fence_mbar_init();
        *abort = 0;
    }
    grid_dependency_wait();

    // the partition of the seen tokens; or whole rows, of which this block takes
    // every gridDim.x-th: its row r (of n_rows) is virtual row row_of(r)
    const int n_rows = p.whole_rows ? (Bv - cta + (int)gridDim.x - 1) / (int)gridDim.x : Bv;
    auto row_of = [&](int r) { return p.whole_rows ? cta + r * (int)gridDim.x : r; };
    row_prefix(p, prefix, n_rows, row_of, [&](int L) { return min(L, sp.most_seen); },
               p.whole_rows || cta == 0);

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
            if (threadIdx.x == 0 && !p.whole_rows) {
                p.row_info[2 * r] = 0;
                p.row_info[2 * r + 1] = 0;
            }
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
        // A warp has the tokens first .. first + kShare - 1 of every kTurn-th stage.  Lane l
        // looks up its tokens l, 32 + l, ... and copies their scales; the copies of the
        // rows take the tokens' slots from it.
        const int pw = warp - kWarps;
        const int first = pw % C::kSplit * C::kShare;
        const uint64_t policy = policy_evict_first();
        constexpr int IDS = (C::kShare + 31) / 32;    // page ids a lane holds
        auto page_of_tok = [&](int t) {
            return p.ps_shift >= 0 ? (t >> p.ps_shift) : (t / p.page_size);
        };
        // A stage: seen tokens [tok, t1) of a row as far as they fit; hg < 0: none.
        struct Stage {
            int r, tok, t1, hg, pg0, npg, skip;
        };
        // the first stage of the rows from r on
        auto row_stage = [&](Stage &s, int r) {
            while (r < n_rows && prefix[r + 1] == prefix[r])
                ++r;
            // [lo, hi): the positions of the row's seen tokens
            const int lo = r < n_rows ? prefix[r] + p.row_cost : end;
            s.hg = -1;
            if (lo >= end)
                return;
            const int hi = prefix[r + 1], v = row_of(r), b = v % p.B;
            s.r = r;
            s.tok = max(start, lo) - lo;
            s.t1 = min(end, hi) - lo;
            s.hg = v / p.B;
            s.pg0 = p.kv_indptr[b];
            s.npg = p.kv_indptr[b + 1] - s.pg0;
            if (s.pg0 < 0 || s.npg < 0 || s.pg0 > p.num_indices - s.npg)
                s.npg = 0;
            // tokens that a row of the window's length skips behind its sinks
            s.skip = 0;
            if (hi - lo == sp.most_seen) {
                unsigned bad = 0;
                s.skip = checked_row_len(p, b, bad) - sp.most_seen;
            }
        };
        auto step = [&](Stage &s, int n) {
            for (int k = 0; k < n && s.hg >= 0; ++k) {
                s.tok += C::kTok;
                if (s.tok >= s.t1)
                    row_stage(s, s.r + 1);
            }
        };
        auto token = [&](const Stage &s, int i) { return i < sp.sinks ? i : i + s.skip; };
        // the table's entry for this lane's k-th token of a stage
        auto load_id = [&](const Stage &s, int k) {
            const int at = k * 32 + lane;
            const bool there = s.hg >= 0 && at < C::kShare && s.tok + first + at < s.t1;
            const int pi = page_of_tok(there ? token(s, s.tok + first + at) : 0);
            return there && pi < s.npg ? p.kv_indices[s.pg0 + pi] : 0;
        };
        int it = pw / C::kSplit;
        Stage cur;
        row_stage(cur, r0);
        step(cur, it);
        int ids[IDS];
#pragma unroll
        for (int k = 0; k < IDS; ++k)
            ids[k] = load_id(cur, k);
        for (; cur.hg >= 0; it += C::kTurn) {
            const int st = it % NST;
            // the ids of this warp's next stage, of another row too, are on their way
            Stage after = cur;
            step(after, C::kTurn);
            int next[IDS];
#pragma unroll
            for (int k = 0; k < IDS; ++k)
                next[k] = load_id(after, k);
            if (it >= NST) {
                // (a consumer that gave up releases its stages without having
                // waited for them, after it has set the abort word)
                const bool ok =
                    mbar_wait_or_abort(&empty[st], (uint32_t)(((it / NST) - 1) & 1),
                                       p.handoff_wait_ns, abort) &&
                    !*abort;
                if (!__all_sync(kFull, ok)) {
                    if (lane == 0) {
                        *abort = 1;
                        atomicOr(p.status, kFlagTimeout);
                    }
                    break;
                }
            }
            unsigned char *stage = smem + st * C::kStageBytes;
            unsigned char *sc0 = smem + C::kScaleOffset + st * C::kScaleBytes;
            // (of this warp's share)
            const int tok0 = cur.tok + first;
            const int nvalid = max(0, min(C::kShare, cur.t1 - tok0));
            // a page id of a token that is there, checked
            auto checked = [&](int page, bool there) {
                if (page < 0 || page >= p.num_pages) {
                    if (there)
                        atomicOr(p.status, kFlagBadPage);
                    page = 0;
                }
                return page;
            };
            // a token's scale bytes of one pool, from byte `at` of it
            auto copy_scales = [&](const uint8_t *scales, int row, size_t at) {
                unsigned char *sc = sc0 + row * C::kScalePitch;
                if constexpr (C::kScaleRow >= 16) {
#pragma unroll
                    for (int j = 0; j < C::kScaleRow; j += 16)
                        cp_async16(smem_addr(sc + j), scales + at + j, policy);
                } else if constexpr (C::kScaleRow == 8) {
                    cp_async<8>(sc, scales + at, 8);
                } else if constexpr (C::kScaleRow == 4) {
                    cp_async<4>(sc, scales + at, 4);
                } else {
                    // the aligned word around the two bytes (the pool's last may be
                    // half a word), and where they are in it
                    const size_t word = at & ~(size_t)3;
                    const size_t left =
                        (size_t)p.num_pages * p.page_size * p.Hkv * G32 - word;
                    cp_async<4>(sc, scales + word, left < 4 ? (int)left : 4);
                    sc[4] = (unsigned char)(at & 3);
                }
            };
            if constexpr (C::kBulk) {
                // Lane l: token first + l % kShare, K, or from lane kShare on V.  The rows
                // of V that end the piece's last tile are zeroed: their weights are 0,
                // and what a stage held may be NaN.
                const int at = lane % C::kShare;
                const bool mine = lane < 2 * C::kShare, of_v = lane >= C::kShare;
                const bool there = mine && at < nvalid;
                const int t = there ? token(cur, tok0 + at) : 0;
                const int page = checked(__shfl_sync(kFull, ids[0], at), there);
                uint64_t *bar = &full[st * C::kFulls + pw];
                fence_proxy_async_smem();          // the slot's last reads, before the copies
                unsigned char *to = stage + ((of_v ? C::kTok : 0) + first + at) * C::kPitch;
                if (mine && of_v && !there)
                    for (int j = 0; j < C::kRowBytes / 16; ++j)
                        reinterpret_cast<uint4 *>(to)[j] = make_uint4(0u, 0u, 0u, 0u);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, (uint32_t)(nvalid * 2 * C::kRowBytes));
                else
                    mbar_arrive(bar);
                if (there) {
                    const size_t slot = (size_t)page * p.page_size + t - page_of_tok(t) * p.page_size;
                    const uint8_t *from = (of_v ? p.v_codes : p.k_codes) +
                                          slot * ((size_t)p.Hkv * C::kHeadBytes) +
                                          (size_t)cur.hg * C::kRowBytes;
                    bulk_copy_g2s_hint(to, from, C::kRowBytes, bar, policy);
                }
            } else {
                // bf16: the rows of V that end the piece's last tile are zeroed (their
                // weights are 0, and what a stage held may be NaN)
                const int tiles_end = (min(C::kTok, cur.t1 - cur.tok) + 15) & ~15;
                const int filled = BITS == 16 ? min(C::kShare, tiles_end - first) : nvalid;
                constexpr int CH = C::kRowBytes / 16;      // 16-byte lines of a token
                const size_t line0 = (size_t)cur.hg * C::kRowBytes;
                const unsigned tok_bytes = (unsigned)(p.Hkv * C::kHeadBytes);
#pragma unroll
                for (int k = 0; k < IDS; ++k) {
                    if (k * 32 >= filled)
                        break;
                    const int row = k * 32 + lane;
                    const bool there = row < nvalid;
                    const int t = there ? token(cur, tok0 + row) : 0;
                    const int page = checked(ids[k], there);
                    const int slot = page * p.page_size + t - page_of_tok(t) * p.page_size;
                    if constexpr (C::kCodes) {
                        if (there) {
                            const size_t at = ((size_t)slot * p.Hkv + (size_t)cur.hg * HPC) * G32;
                            copy_scales(p.k_scale, first + row, at);
                            copy_scales(p.v_scale, C::kTok + first + row, at);
                        }
                    }
                    // 32 lines at a time, 32 / CH tokens' (or part of one): line
                    // 32 j + lane lies at byte 16 (32 j + lane) of these tokens'
                    // rows, its swizzle that of the lane, of j and of the share, which
                    // starts at a multiple of its size (no carry)
                    constexpr int ROUNDS = (C::kShare < 32 ? C::kShare : 32) * CH / 32;
                    const uint32_t lane_key =
                        (uint32_t)(((lane / CH) >> kKeyShift ^ first >> kKeyShift) & 7) << 4;
                    const uint32_t to = smem_addr(stage) + (first + k * 32) * C::kRowBytes;
#pragma unroll 8
                    for (int j = 0; j < ROUNDS; ++j) {
                        const int from = (j * 32 + lane) / CH, ch = (j * 32 + lane) % CH;
                        const unsigned s_ = (unsigned)__shfl_sync(kFull, slot, from);
                        const bool in = k * 32 + from < nvalid;
                        const size_t off = (size_t)s_ * tok_bytes + (line0 + ch * 16);
                        const uint32_t dst =
                            to + j * 512 +
                            ((lane * 16u) ^ lane_key ^
                             (uint32_t)((j * 32 / CH) >> kKeyShift & 7) << 4);
                        if (in)
                            cp_async16(dst, p.k_codes + off, policy);
                        if (in)
                            cp_async16(dst + C::kTok * C::kRowBytes, p.v_codes + off, policy);
                        else if (BITS == 16 && k * 32 + from < filled)
                            cp_async16_part(dst + C::kTok * C::kRowBytes, p.v_codes, 0, policy);
                    }
                }
                cp_async_arrive(&full[st]);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[st]);
            }
#pragma unroll
            for (int k = 0; k < IDS; ++k)
                ids[k] = next[k];
            cur = after;
        }
        // Let this warp's copies land, and their arrivals, before it exits, with the full
        // time limit: a consumer that gave up skips its stages, and the block must not
        // exit while a copy into its shared memory is in flight.
        if constexpr (C::kBulk || C::kSplit == 1) {
            const int f = C::kBulk ? pw : 0;
            for (int k = it - C::kTurn, n = 0; k >= 0 && n < NST; k -= C::kTurn, n += C::kTurn)
                (void)mbar_wait_bounded(&full[k % NST * C::kFulls + f], (uint32_t)((k / NST) & 1));
        } else {
            // A stage's barrier is kSplit warps', which filled the same stages unless
            // somebody gave up.  (A barrier for each would be complete whatever the others
            // did, but costs the consumers more waits: 49.4 us in place of 47.7 on the
            // serving batch, 48.2 with a lane a barrier.)
            cp_async_wait_all();
            for (int k = it - C::kTurn, n = 0; k >= 0 && n < NST && !*abort;
                 k -= C::kTurn, n += C::kTurn)
                (void)mbar_wait_or_abort(&full[k % NST], (uint32_t)((k / NST) & 1),
                                         kWaitLimitNs, abort);
            volatile int *ends = abort + 4;
            if (lane == 0)
                ends[pw] = it;
            named_bar_sync(2, C::kProducers * 32);
            if (*abort) {
                // Then a warp arrives in the stages that the others filled without it, so
                // that each completes, and waits for them all.  (Who fills a slot again has
                // seen its last filling complete: the arrivals go to the stages meant.)
                int last = it;
                for (int i = 0; i < C::kSplit; ++i)
                    last = max(last, ends[pw / C::kSplit * C::kSplit + i]);
                if (lane == 0)
                    for (int k = it; k < last; k += C::kTurn)
                        mbar_arrive(&full[k % NST], 33);
                for (int k = last - C::kTurn, n = 0; k >= 0 && n < NST;
                     k -= C::kTurn, n += C::kTurn)
                    (void)mbar_wait_bounded(&full[k % NST], (uint32_t)((k / NST) & 1));
            }
        }
        grid_launch_dependents();
        return;
    }

    // ========================= consumer warps ===============================
    const int hw = warp % HPC, tg = warp / HPC;   // kv head, its part
    const int g = lane >> 2, c = lane & 3;
    const uint32_t smem_s = smem_addr(smem);
    // Matrix loads: lane l addresses token l % 16 of a tile and the 16-byte
    // column l / 16 of each two; the 32-byte column i of a row whose first is at
    // `addr` is at addr ^ 32 i: the swizzle is in the same bits.
    auto column = [](uint32_t addr, int i) {
        return C::kBulk ? addr + i * 32u : addr ^ (i * 32u);
    };
    const int tile0 = tg * 16 * U;                // this warp's first token of a stage
    const uint32_t k_off =
        smem_s + line_addr(tile0 + (lane & 15), hw * C::kHeadBytes + (lane >> 4) * 16);
    const uint32_t v_off = k_off + C::kTok * C::kPitch;
    // a tile further: 16 rows, and their bits of the swizzle
    auto tile = [](uint32_t addr, int u) {
        return (addr + u * 16 * C::kRowBytes) ^ (uint32_t)((u * 16 >> kKeyShift) & 7) << 4;
    };
    // bf16 weights need no room under the largest; f16's end 2^-24 under 1
    constexpr float kUnder = BITS == 16 ? 0.f : 7.f;
    const Shifts by = shifts();
    int st = 0;                        // the next stage's slot, and the phase of its filling
    uint32_t phase = 0;
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

        // q as the products' B operand, of head g.  bf16: lane (g, c) holds elements
        // 2c, 2c + 1, 2c + 8, 2c + 9 of each 16.  4 bits: elements 8c .. 8c + 7 of each
        // 32, the codes of a word of K, two products' depth.  (Plain loads: the
        // grid before may have written q while this one was already on the GPU.)
        uint32_t qf[NT][D / 16][2];
        float cq[NT][2];                   // factors of heads 2c, 2c + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + g;
            const bool live = h < p.n_rep;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q + (qrow0 + h) * D);
            if constexpr (BITS == 16) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    qf[nt][j][0] = live ? src[8 * j + c] : 0u;
                    qf[nt][j][1] = live ? src[8 * j + 4 + c] : 0u;
                }
                cq[nt][0] = cq[nt][1] = p.scale_log2;
            } else {
                uint4 raw[G32];
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < G32; ++j) {
                    raw[j] = live ? reinterpret_cast<const uint4 *>(src)[4 * j + c]
                                  : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                // 2^(15 - n), n the exponent of amax, both powers kept in the normal range
                // (the largest, 2^16 less a bf16 step, is within f16; infinity stays)
                const int n = min(max((int)(__float_as_uint(amax) >> 23) - 127, -111), 127);
                const float down = __uint_as_float((unsigned)(127 + 15 - n) << 23);
#pragma unroll
                for (int j = 0; j < G32; ++j) {
                    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        qf[nt][2 * j + k / 2][k % 2] =
                            pack_f16x2(bf16_lo(w[k]) * down, bf16_hi(w[k]) * down);
                }
                const float up = __uint_as_float((unsigned)(127 - 15 + n) << 23) * p.scale_log2;
                cq[nt][0] = __shfl_sync(kFull, up, (2 * c) * 4);
                cq[nt][1] = __shfl_sync(kFull, up, (2 * c + 1) * 4);
            }
        }

        // the sums carry 2^-m_run; base: m_run, 0 before the first finite score; a
        // score past `limit` raises it
        float m_run[NT][2], l_run[NT][2], base[NT][2], limit[NT][2];
        float oacc[NT][D / 16][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m_run[nt][0] = m_run[nt][1] = limit[nt][0] = limit[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = base[nt][0] = base[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                oacc[nt][j][0] = oacc[nt][j][1] = oacc[nt][j][2] = oacc[nt][j][3] = 0.f;
        }

        for (int tok = t0; tok < t1; tok += C::kTok) {
            if (!aborted) {
                bool ok = true;
#pragma unroll
                for (int f = 0; f < C::kFulls; ++f)
                    ok = ok && mbar_wait_or_abort(&full[st * C::kFulls + f], phase,
                                                  p.handoff_wait_ns, abort);
                if (!__all_sync(kFull, ok)) {
                    aborted = true;
                    if (lane == 0) {
                        *abort = 1;
                        atomicOr(p.status, kFlagTimeout);
                    }
                }
            }
            const int left = t1 - tok - tile0;          // of the warp's 16 U tokens
            if (!aborted && left > 0) {
                const uint32_t stage = (uint32_t)st * C::kStageBytes;
                const unsigned char *sc =
                    smem + C::kScaleOffset + st * C::kScaleBytes + tile0 * C::kScalePitch;
                const bool cut = left < 16 * U;
                auto in = [&](int t) { return t < left; };
                // scores (log2 domain) of rows g, g + 8 (x >> 1) and heads 2c, 2c + 1 (x & 1)
                float y[NT][U][4];
                // 4 bits: the tokens' scale words of V, and the scores y - ev without them
                uint32_t wv[U][2];
                float x_[NT][U][4];
                if constexpr (BITS == 16) {
                    float sacc[NT][4] = {};
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t a[4];
                        ldmatrix_x4(a[0], a[1], a[2], a[3], column(stage + k_off, i));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_bf16_16816(sacc[nt], a, qf[nt][i][0], qf[nt][i][1]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            y[nt][0][x] = sacc[nt][x] * cq[nt][x & 1];
                    if (cut) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (!in(g + (x >> 1) * 8))
                                    y[nt][0][x] = -INFINITY;
                    }
                } else {
                    // the scale words of the tokens at rows g and g + 8 of each tile
                    uint32_t wk[U][2];
                    auto scale_word = [&](int row) {
                        const unsigned char *at = sc + row * C::kScalePitch;
                        if constexpr (C::kScaleRow == 2)
                            return (uint32_t)*reinterpret_cast<const uint16_t *>(at + (at[4] & 2));
                        else if constexpr (G32 == 2)
                            return (uint32_t)reinterpret_cast<const uint16_t *>(at)[hw];
                        else
                            return reinterpret_cast<const uint32_t *>(at)[hw];
                    };
                    float s[NT][U][4];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            wk[u][k] = scale_word(u * 16 + k * 8 + g);
                            wv[u][k] = scale_word(C::kTok + u * 16 + k * 8 + g);
                        }
                    // (the scale bytes of a token that is not there may be any: none)
                    if (cut) {
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                if (!in(u * 16 + k * 8 + g))
                                    wv[u][k] = 0;
                    }
                    auto unit = [&](auto at, int u, uint32_t lo_, uint32_t hi_) {
                        constexpr int i = decltype(at)::value;
                        const uint32_t a0[4] = {f16x2_of_e2m1x2<0>(lo_), f16x2_of_e2m1x2<0>(hi_),
                                                f16x2_of_e2m1x2<1>(lo_), f16x2_of_e2m1x2<1>(hi_)};
                        const uint32_t a1[4] = {f16x2_of_e2m1x2<2>(lo_), f16x2_of_e2m1x2<2>(hi_),
                                                f16x2_of_e2m1x2<3>(lo_), f16x2_of_e2m1x2<3>(hi_)};
                        const float f[2] = {scale_of<i>(wk[u][0], by), scale_of<i>(wk[u][1], by)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float acc[4];
                            mma_f16_from_zero(acc, a0, qf[nt][2 * i][0], qf[nt][2 * i][1]);
                            mma_f16(acc, a1, qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[nt][u][x] = i == 0 ? acc[x] * f[x >> 1]
                                                     : fmaf(acc[x], f[x >> 1], s[nt][u][x]);
                        }
                    };
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        uint32_t w[4];
                        const uint32_t at = tile(stage + k_off, u);
                        ldmatrix_x4(w[0], w[1], w[2], w[3], at);
                        unit(Const<0>(), u, w[0], w[1]);
                        unit(Const<1>(), u, w[2], w[3]);
                        if constexpr (G32 == 4) {
                            ldmatrix_x4(w[0], w[1], w[2], w[3], column(at, 1));
                            unit(Const<2>(), u, w[0], w[1]);
                            unit(Const<3>(), u, w[2], w[3]);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float top = fmaxf(scale_of<0>(wv[u][k], by), scale_of<1>(wv[u][k], by));
                            if constexpr (G32 == 4)
                                top = fmax3(top, scale_of<2>(wv[u][k], by),
                                            scale_of<3>(wv[u][k], by));
                            // 2^23 + 128 times its byte, as a float: the upper half of its
                            // bits, and from there the exponent ev = byte - 127
                            const float up = __uint_as_float(
                                __byte_perm(__float_as_uint(top), 0x4b000000u, 0x7632));
                            const float ev = fmaf(up, 0x1p-7f, -(65536.f + 127.f));
                            const float nan = top - top;      // of scale 255, else 0
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    x_[nt][u][2 * k + e] = fmaf(s[nt][u][2 * k + e], cq[nt][e], nan);
                                    y[nt][u][2 * k + e] = x_[nt][u][2 * k + e] + ev;
                                }
                        }
                    if (cut) {
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                if (!in(u * 16 + k * 8 + g)) {
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                        for (int e = 0; e < 2; ++e)
                                            x_[nt][u][2 * k + e] = y[nt][u][2 * k + e] = -INFINITY;
                                }
                    }
                }
                // (a score past its limit: the sign of a difference, as the
                // comparison would be on the pipe that is short)
                unsigned raise = 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            raise |= __float_as_uint(limit[nt][x & 1] - y[nt][u][x]);
                if (__any_sync(kFull, (int)raise < 0)) {
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
                            base[nt][e] = mn == -INFINITY ? 0.f : mn;
                            limit[nt][e] = mn + kRaise;
                            l_run[nt][e] *= a;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                oacc[nt][j][e] *= a;
                                oacc[nt][j][e + 2] *= a;
                            }
                        }
                }
                // the weights: 4 bits: without the values' scales
                float w[NT][U][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if constexpr (BITS == 4) {
                                w[nt][u][x] = exp2_ftz(x_[nt][u][x] - base[nt][x & 1]);
                                l_run[nt][x & 1] += w[nt][u][x];
                            } else {
                                w[nt][u][x] = exp2_ftz(y[nt][u][x] - base[nt][x & 1]);
                            }
                        }
                }
                // O^T += V^T P^T.  S^T's layout has a token's heads in a lane, P^T's B
                // operand a head's tokens: transpose the two 8 x 8 halves.
                if constexpr (BITS == 16) {
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t v = pack_bf16x2(w[nt][0][2 * k], w[nt][0][2 * k + 1]);
                            l_run[nt][0] += bf16_lo(v);
                            l_run[nt][1] += bf16_hi(v);
                            pb[nt][k] = movmatrix_trans(v);
                        }
                    // a transposed 8-token x 8-element matrix gives lane (g, c) elements
                    // g of tokens 2c and 2c + 1
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t a[4];
                        ldmatrix_x4_trans(a[0], a[2], a[1], a[3], column(stage + v_off, i));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_bf16_16816(oacc[nt][i], a, pb[nt][0], pb[nt][1]);
                    }
                } else {
                    // a transposed 8-token x 16-byte matrix gives lane (g, c) the codes
                    // 4g .. 4g + 3 of a unit, of tokens 2c and 2c + 1: products 2i and
                    // 2i + 1 take codes 4g, 4g + 1 and 4g + 2, 4g + 3 as rows g, g + 8
                    auto unit = [&](auto at, int u, uint32_t lo_, uint32_t hi_) {
                        constexpr int i = decltype(at)::value;
                        const float f[2] = {scale_of<i>(wv[u][0], by), scale_of<i>(wv[u][1], by)};
                        uint32_t pb[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                pb[nt][k] = movmatrix_trans(pack_f16x2(
                                    w[nt][u][2 * k] * f[k], w[nt][u][2 * k + 1] * f[k]));
                        uint32_t le, lo, he, ho;
                        two_tokens(lo_, by, le, lo);
                        two_tokens(hi_, by, he, ho);
                        const uint32_t a0[4] = {f16x2_of_e2m1x2<2>(le), f16x2_of_e2m1x2<2>(lo),
                                                f16x2_of_e2m1x2<2>(he), f16x2_of_e2m1x2<2>(ho)};
                        const uint32_t a1[4] = {f16x2_of_e2m1x2<3>(le), f16x2_of_e2m1x2<3>(lo),
                                                f16x2_of_e2m1x2<3>(he), f16x2_of_e2m1x2<3>(ho)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(oacc[nt][2 * i], a0, pb[nt][0], pb[nt][1]);
                            mma_f16(oacc[nt][2 * i + 1], a1, pb[nt][0], pb[nt][1]);
                        }
                    };
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        uint32_t v[4];
                        const uint32_t at = tile(stage + v_off, u);
                        ldmatrix_x4_trans(v[0], v[1], v[2], v[3], at);
                        unit(Const<0>(), u, v[0], v[1]);
                        unit(Const<1>(), u, v[2], v[3]);
                        if constexpr (G32 == 4) {
                            ldmatrix_x4_trans(v[0], v[1], v[2], v[3], column(at, 1));
                            unit(Const<2>(), u, v[0], v[1]);
                            unit(Const<3>(), u, v[2], v[3]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[st]);
            if (++st == NST) {
                st = 0;
                phase ^= 1u;
            }
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
        const bool whole = t0 == 0 && t1 == hi - lo;
        if (t0 == 0 && warp == 0 && lane == 0 && !p.whole_rows) {
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
                float inv = l > 0.f ? 1.f / l : 0.f;
                if (!(l >= 0.f))             // NaN (or a NaN scale): kept through the combine
                    l = 1.f, m = 0.f, inv = __uint_as_float(0x7fffffffu);
                // oacc[nt][j][e], [e + 2]: 4 bits: columns 32 (j / 2) + 4g + 2 (j % 2) and the
                // next; bf16: 16 j + g and 8 on: lanes of two g trade one of them to have
                // two in a row (every lane, as the shuffle needs the warp)
                float2 o[D / 16];
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    float a = oacc[nt][j][e] * inv, d = oacc[nt][j][e + 2] * inv;
                    if constexpr (BITS == 16) {
                        const float got = __shfl_xor_sync(kFull, g & 1 ? a : d, 4);
                        if (g & 1)
                            a = got;
                        else
                            d = got;
                    }
                    o[j] = make_float2(a, d);
                }
                if (h >= p.n_rep)
                    continue;
                const int col = BITS == 16 ? (g & 1 ? 8 + g - 1 : g) : 4 * g;
                auto at = [&](int j) { return BITS == 16 ? 16 * j : 32 * (j / 2) + 2 * (j % 2); };
                if (whole) {
                    __nv_bfloat16 *to = p.out + (qrow0 + h) * D + col;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        *reinterpret_cast<uint32_t *>(to + at(j)) = pack_bf16x2(o[j].x, o[j].y);
                } else {
                    float *to = p.o_part + (slot0 + h) * D + col;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        *reinterpret_cast<float2 *>(to + at(j)) = o[j];
                    if (g == 0)
                        reinterpret_cast<float2 *>(p.ml_part)[slot0 + h] =
                            l > 0.f ? make_float2(m * kLn2f, l) : make_float2(-INFINITY, 0.f);
                }
            }
    }
    grid_launch_dependents();
}

template <int BITS, int D, int HPC, int NT>
cudaError_t launch(const StreamParams &p, int grid, cudaStream_t stream)
{
    using C = StreamCfg<BITS, D, HPC, NT>;
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        cudaError_t r = cudaFuncSetAttribute(stream_decode_kernel<BITS, D, HPC, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmemBytes);
        if (r != cudaSuccess)
            return r;
        return cudaFuncSetAttribute(stream_decode_kernel<BITS, D, HPC, NT>,
                                    cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess)
        return e;
    return launch_pdl(stream_decode_kernel<BITS, D, HPC, NT>, dim3(grid), dim3(C::kThreads),
                      C::kSmemBytes, stream, p);
}

template <int BITS, int D, int HPC>
cudaError_t launch_nt(const StreamParams &p, int grid, cudaStream_t stream)
{
    return p.f.n_rep <= 8 ? launch<BITS, D, HPC, 1>(p, grid, stream)
                          : launch<BITS, D, HPC, 2>(p, grid, stream);
}

template <int BITS, int D>
cudaError_t launch_d(const StreamParams &p, int grid, cudaStream_t stream)
{
    switch (p.f.hpc) {
    case 8:
        return launch_nt<BITS, D, 8>(p, grid, stream);
    case 4:
        return launch_nt<BITS, D, 4>(p, grid, stream);
    case 2:
        return launch_nt<BITS, D, 2>(p, grid, stream);
    default:
        return launch_nt<BITS, D, 1>(p, grid, stream);
    }
}

} // namespace

cudaError_t launch_stream_decode(const StreamParams &params, int D, int grid, cudaStream_t stream)
{
    StreamParams p = params;
    p.f.handoff_wait_ns = handoff_wait_ns();
    if (p.bits == 4)
        return D == 64 ? launch_d<4, 64>(p, grid, stream) : launch_d<4, 128>(p, grid, stream);
    return D == 64 ? launch_d<16, 64>(p, grid, stream) : launch_d<16, 128>(p, grid, stream);
}

} // namespace pkv
