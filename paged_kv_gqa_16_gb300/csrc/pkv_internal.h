// pkv_internal.h -- parameter blocks and launchers shared by the .cu files of
// libpkv (not part of the public ABI; see include/pkv.h for that).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <mutex>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pkv.h"

namespace pkv {

// Largest split count any entry point accepts.
constexpr int kMaxSplits = 65536;

// Shape checks common to every entry point (pkv_api.cu).
pkv_status check_dims(const pkv_dims *d);

// One-time set-up of a kernel's function attributes (the opt-in shared
// memory size, the carveout).  Those attributes belong to the current
// device's context, so a process that launches on several devices sets them
// once on each; host threads may launch concurrently, hence the lock.
constexpr int kMaxDevices = 64;

class DeviceOnce {
public:
    template <typename F>
    cudaError_t run(F &&setup)
    {
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return e;
        if (dev < 0 || dev >= kMaxDevices)
            return cudaErrorInvalidDevice;
        if (done_[dev].load(std::memory_order_acquire))
            return cudaSuccess;
        std::lock_guard<std::mutex> lock(mu_);
        if (done_[dev].load(std::memory_order_relaxed))
            return cudaSuccess;
        e = setup();
        if (e == cudaSuccess)
            done_[dev].store(true, std::memory_order_release);
        return e;
    }

private:
    std::mutex mu_;
    std::atomic<bool> done_[kMaxDevices]{};
};

// Launch with programmatic stream serialisation: the kernel may start while
// the one before it drains, and waits for it (griddepcontrol.wait) itself.
template <typename Kernel, typename... Params>
inline cudaError_t launch_pdl(Kernel k, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       const Params &...p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p...);
}

struct AppendParams {
    __nv_bfloat16 *q;
    const __nv_bfloat16 *k_new;
    const __nv_bfloat16 *v_new;
    __nv_bfloat16 *k_pool;
    __nv_bfloat16 *v_pool;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *seq_lens;
    const float *rope;     // [rope_max_pos, D/2, 2] or nullptr
    uint32_t *status;      // nullable
    int B, Hq, Hkv, D, page_size, num_pages, num_indices, max_seq_len;
    int rope_max_pos, rope_q;
    const int32_t *qo_indptr;  // extend: [B+1] chunk offsets (append: unused)
    int total_q;               // extend: tokens in all chunks
};

// New tokens written to the cache (pkv_tokens.cu); bits 16: bf16 pools, 8 and 4:
// codes and e8m0 scales.
struct TokenWriteParams {
    const __nv_bfloat16 *q;        // nullable: no query work
    const __nv_bfloat16 *k;
    const __nv_bfloat16 *v;
    long long q_stride, k_stride, v_stride;
    __nv_bfloat16 *q_out;
    const __nv_bfloat16 *q_norm;   // [D] or nullptr
    const __nv_bfloat16 *k_norm;
    const float *rope;             // [rope_max_pos, D/2, 2] or nullptr
    void *k_pool;                  // bf16 pools or codes
    void *v_pool;
    uint8_t *k_scale;
    uint8_t *v_scale;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *seq_lens;
    const int32_t *qo_indptr;      // extend: [B+1]; append: nullptr
    uint32_t *status;              // nullable
    float norm_eps;
    int T, B, Hq, Hkv, page_size, num_pages, num_indices, max_seq_len, rope_max_pos;
    int bits;                      // 16, 8 or 4
    int width_shift;               // log2 of the lane groups a token takes (set by the launcher)
};

// An 8-bit or 4-bit cache read back as bf16 (pkv_q8_read.cu).
struct ReadCodesParams {
    const uint8_t *k_codes;
    const uint8_t *v_codes;
    const uint8_t *k_scale;
    const uint8_t *v_scale;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *seq_lens;
    __nv_bfloat16 *k_out;
    __nv_bfloat16 *v_out;
    uint32_t *status;              // nullable
    int B, Hkv, page_size, num_pages, num_indices, max_seq_len;
    int ps_shift;                  // log2 of page_size, or -1
    int bits;                      // 8 or 4
    int per_warp;                  // token slots a warp takes at a time (set by the launcher)
};

struct DecodeParams {
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *k_pool;
    const __nv_bfloat16 *v_pool;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *seq_lens;
    float *o_part;         // [B, Hq, S, D]
    float *ml_part;        // [B, Hq, S, 2]
    __nv_bfloat16 *out;    // [B, Hq, D], used when direct != 0
    uint32_t *status;
    int B, Hq, Hkv, n_rep, page_size, ps_shift, num_pages, num_indices;
    int max_seq_len, num_splits, chunk, direct;
    float scale_log2;      // scale * log2(e)
};

// Device-side metadata advance (pkv_advance.cu).
struct AdvanceParams {
    int32_t *seq_lens;
    const int32_t *kv_indptr;
    int32_t *kv_indices;
    const int32_t *free_pages;
    int32_t *free_head;
    uint32_t *status;      // nullable
    int B, page_size, max_seq_len, num_indices, num_free;
};

// Paged ragged prefill / extend (pkv_prefill.cu).
struct PrefillParams {
    const __nv_bfloat16 *q;        // [total_q, Hq, D]
    const int32_t *qo_indptr;      // [B+1]
    const __nv_bfloat16 *k_pool;
    const __nv_bfloat16 *v_pool;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *seq_lens;
    __nv_bfloat16 *out;            // [total_q, Hq, D]
    uint32_t *status;              // nullable
    int B, Hq, Hkv, n_rep, page_size, ps_shift, num_pages, num_indices, max_seq_len, total_q;
    int tq;                        // query tokens per block: 128 / n_rep
    float scale_log2;
    // a query sees the last `window` keys up to its own and the first `sinks`
    // (window 0: all keys up to its own)
    int window;
    int sinks;
    // the pools as 3-D tiled tensors {D, Hkv, pages x page_size} with a box of
    // {64, 1, tma_rows} and 128-byte swizzle (use_tma != 0; set by
    // launch_prefill when the page size is a multiple of 8)
    CUtensorMap tmap_k;
    CUtensorMap tmap_v;
    int use_tma;
    unsigned ps_magic;             // token / page_size by a product (set by launch_prefill)
    int ps_magic_shift;
    int tma_rows;                  // the power of two dividing page_size, at most 128
    // q as {D, Hq, total_q} with a box of {64, n_rep, tq}: one query tile's
    // rows (token-major, head-minor), 128-byte swizzled (q_tma != 0)
    CUtensorMap tmap_q;
    int q_tma;
    // the units of work (set by launch_prefill): pairs of query tiles per
    // chunk (from max_q_len) and pairs x B x Hkv
    int pairs;
    int n_units;                   // entries of the list: units, then split parts
    int group_rows;                // rows per group of the unit list
    // the key split (split > 1): entries [split_base, n_units) are the parts
    // of the list's last units, split to a unit; entry e's tile x leaves its
    // normalised rows at ws_o [(2 e + x) x 128 + row][D] and each row's
    // (base, l) at ws_ml [(2 e + x) x 128 + row] for the merge kernel
    int split;
    int split_base;
    __nv_bfloat16 *ws_o;
    float2 *ws_ml;
    // out is 32-byte aligned: rows are stored with 32-byte stores (set by
    // launch_prefill; otherwise 16-byte stores, each lane its own row)
    int out_align32;
};

// The prefill's key split.  When the unit list's last round would leave at
// least half the SMs idle, its units are cut along their key blocks into
// parts on separate SMs (at most kPrefillMaxParts, each of at least
// kPrefillMinPartBlocks blocks).
constexpr int kPrefillMaxParts = 16;
constexpr int kPrefillMinPartBlocks = 2;
// Workspace: per entry of the split round, two tiles of 128 bf16 rows of D
// (all entries' rows first) and two tiles of 128 fp32 (base, l) pairs; for
// up to kPrefillMaxSms SMs.
constexpr int kPrefillMaxSms = 1024;
inline size_t prefill_slot_o_bytes(int D) { return (size_t)2 * 128 * D * 2; }
inline size_t prefill_slot_bytes(int D) { return prefill_slot_o_bytes(D) + (size_t)2 * 128 * 8; }

// Persistent token-balanced decode (pkv_fused.cu).
constexpr int kFusedMaxRows = 4096;     // virtual rows whose prefix sums fit in smem
constexpr int kFusedMinTokens = 64;     // fewest tokens a block is given
// Partition weight of a row beyond its tokens: a block pays a fixed cost at
// each row it starts (page-table window, q block, partial write), measured
// at about 1.8 us per extra row, the time of ~20 streamed tokens.  Charging
// it in the partition gives blocks that cross more row boundaries fewer
// tokens; 32 measured best of {0, 16, 32, 48} on the serving mixes.
constexpr int kFusedRowCost = 32;

struct FusedParams {
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *k_pool;
    const __nv_bfloat16 *v_pool;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *seq_lens;
    __nv_bfloat16 *out;
    float *o_part;         // [(grid + Bv) * HQV, D]  piece partials
    float *ml_part;        // [(grid + Bv) * HQV, 2]
    int32_t *row_info;     // [Bv, 2]: first block, piece count
    uint32_t *status;
    int B, Hq, Hkv, n_rep, page_size, ps_shift, num_pages, num_indices, max_seq_len;
    int Bv;                // virtual rows: (Hkv / hpc) head groups x B
    int row_cost;          // partition weight of a non-empty row beyond its tokens
    int hpc;               // kv heads per block (1, 2, 4 or 8)
    float scale_log2;
    // fused step: the new token (k_new, v_new at position seq_len - 1) is
    // rotated, written to its pool slot and attended from shared memory; q
    // is rotated in registers.  step == 0: plain decode over the pool.
    int step;
    __nv_bfloat16 *k_pool_w;          // the pools, writable (step only)
    __nv_bfloat16 *v_pool_w;
    const __nv_bfloat16 *k_new;       // [B, Hkv, D]
    const __nv_bfloat16 *v_new;
    const float *rope;                // [rope_max_pos, D/2, 2] or nullptr
    int rope_max_pos;
    // limit of the waits that hand a stage or the q block between the
    // producer and the consumers (normally the full ~2 s; shortened only by
    // the testing call).  Waits for copies already issued keep the full limit.
    unsigned long long handoff_wait_ns;
    // the 8-bit cache (pkv_q8_decode.cu), in place of k_pool and v_pool
    const uint8_t *k_codes;
    const uint8_t *v_codes;
    const uint8_t *k_scale;
    const uint8_t *v_scale;
    int whole_rows;        // each block takes whole rows: cta, cta + grid, ...
    // the step's plan (paged_decode_plan) or nullptr: the partition computed
    // at the kernel's start instead
    const int32_t *plan;
    // unplanned calls: where to leave the partition as the step's plan
    // (nullptr: nowhere)
    int32_t *plan_out;
};

// The same over the 8-bit cache, whose tokens stream in half the time: of {16,
// 32, 48, 64, 96, 128, 192}, 64 measured best on the serving batch of 128 (59.1,
// 58.1, 58.4, 57.4, 57.9, 58.7, 59.0 us) and 8 rows of 513 to 1,025 tokens (10.6,
// 10.0, 9.9, 9.2, 9.2, 9.2, 9.2 us).
constexpr int kQ8RowCost = 64;
// Over the 8-bit cache a row of at most this many bytes of K and V of a block's
// kv heads (by max_seq_len) is not split, and twice as many where there are rows
// x kv-head groups for half the SMs: no combine, and no block with dozens of
// rows because the split count counts tokens alone.  Unsplit against split, us:
//   8 heads of 128, 128 tokens (256 KB): 1 row 8.9, 9.7; 76 rows 9.2, 11.9; 512
//   rows 28.5, 33.0.  192 (384 KB): 11.0, 9.9; 11.6, 13.8; 36.9, 39.3.  256
//   (512 KB): 13.4, 9.9; 14.0, 14.7; 46.0, 46.1.  512: 22.2, 10.1; 23.4, 19.0;
//   82.4, 74.9.  2 heads of 64, 32 rows of 512 (128 KB): 8.0, 10.3.  1 head of
//   64, 76 rows of 512 (64 KB): 7.4, 12.0.
constexpr long long kQ8WholeBytes = 256 << 10;
// Rows x kv-head groups of one launch over the 8-bit cache (pkv_q8_decode.cu),
// whose ring of stages needs the room of more prefix sums.
constexpr int kQ8MaxRows = 1024;

// Decode over the 4-bit cache or through a window (pkv_stream_decode.cu).  A row's
// last token sees its first `sinks` tokens and the last most_seen - sinks (a row of
// at most most_seen: all); no window: most_seen is max_seq_len's bound and no row's
// tokens are skipped.  f.k_codes and f.v_codes are the pools of either kind.
constexpr int kQ4RowCost = 64;
constexpr int kWindowRowCost = 32;
// Rows of which at most so many bytes (K and V of a block's kv heads) are seen are not
// split, and twice as many (by lines 1.5 times) where there are `many`: rows x kv-head
// groups for half the SMs.  4 bits: 56 KB and 8 for each head of the block; bf16 by
// 16-byte lines 128 KB and 16, by bulk copies 512 KB.  (With fewer heads a block, more
// warps join their parts at a row's end.)  Unsplit against split, us:
//   4 bits, 8 heads of 128, 128 tokens (136 KB): 1 row 8.1, 9.0; 76 rows 8.2, 10.9; 512
//   rows 26.0, 33.0.  192 (204 KB): 10.1, 9.4; 10.4, 11.8; 34.4, 40.1.  256: 12.2, 9.0;
//   12.6, 13.0; 43.2, 47.3.  8 heads of 64, 192 (102 KB): 7.7, 7.8; 7.9, 9.7.  384 (204
//   KB): 11.8, 7.7; 12.0, 12.2; 40.9, 44.2.  1 head of 128, 384 (51 KB): 8.9, 9.0.  512
//   (68 KB): 9.9, 9.1; 10.2, 12.1.  1,024 (136 KB): 13.9, 9.4; 14.1, 14.1; 47.8, 52.6.
//   bf16, 8 heads of 64, 96 (192 KB): 6.8, 7.3; 128: 8.2, 8.1; 8 rows 8.2, 8.4; 76 rows
//   8.7, 9.9.  192 (384 KB): 10.9, 8.4; 76 rows 11.8, 11.3; 512 rows 39.3, 41.4.  4 of 64,
//   192 (192 KB): 7.0, 7.2.  256: 8.4, 7.3; 8.8, 9.4; 28.7, 29.8.  1 of 128, 256 (128
//   KB): 7.2, 7.3.  512: 10.3, 7.7; 11.0, 11.4; 34.7, 35.9.
//   By bulk copies, 8 heads of 128, 128 tokens (512 KB): 1 row 9.6, 9.4; 76 rows 12.4,
//   14.7; 512 rows 46.1, 51.1.  256: 15.0, 9.6; 20.0, 20.0; 85.5, 88.7.
inline long long stream_whole_bytes(int bits, int hpc, bool bulk, bool many)
{
    const long long kb = bits == 4 ? 56 + 8 * hpc : bulk ? 512 : 128 + 16 * hpc;
    return (bits == 4 || bulk ? many ? 2 * kb : kb : many ? kb * 3 / 2 : kb) << 10;
}
// Rows of K (or V) that are copied by one bulk copy each: a token's kv heads of a block.
constexpr int kBulkRowBytes = 2048;
struct StreamParams {
    FusedParams f;
    int bits;              // 16 (bf16 pools) or 4 (codes and scales)
    int most_seen;
    int sinks;
};

// Threads of a plan block.
constexpr int kPlanThreads = 256;
// int32 words of the plan for Bv virtual rows and a grid of `grid` blocks.
inline size_t plan_words(int Bv, int grid)
{
    return 16 + (((size_t)Bv + 1 + 3) & ~(size_t)3) + (size_t)72 * grid;
}

// The hand-off wait limit launches use (pkv_testing_set_handoff_wait_ns).
unsigned long long handoff_wait_ns();

struct PieceCombineParams {
    const float *o_part;
    const float *ml_part;
    const int32_t *row_info;
    __nv_bfloat16 *out;
    int B, Bv, Hq, HQV;
    // a planned call's plan: if it is of this grid and shape, row_info is the
    // plan's and may be read before the decode grid has completed
    const int32_t *plan;
    int grid, page_size, row_cost;
    // paged_decode_step_advance: one extra block runs the metadata advance
    // (adv.seq_lens == nullptr: none)
    AdvanceParams adv;
};

struct CombineParams {
    const float *o_part;
    const float *ml_part;
    __nv_bfloat16 *out;
    int B, Hq, D, num_splits;
};

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_extend(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_token_write(const TokenWriteParams &p, int D, cudaStream_t stream);
cudaError_t launch_read_codes(const ReadCodesParams &p, int D, cudaStream_t stream);
// the decode over an 8-bit cache; p.k_codes ... p.v_scale in place of the pools
cudaError_t launch_decode_q8(const FusedParams &p, int D, int grid, cudaStream_t stream);
cudaError_t launch_stream_decode(const StreamParams &p, int D, int grid, cudaStream_t stream);
cudaError_t launch_advance(const AdvanceParams &p, cudaStream_t stream);
// one persistent block per SM over the units (pairs of query tiles x B x Hkv)
// The prefill's list for a launch (host only): units of tile pairs, their
// grouping, and the key split of the last round.
struct PrefillPlan {
    int pairs;       // tile pairs a chunk of max_q_len has
    int units;       // pairs x B x Hkv (0: nothing to run)
    int group_rows;  // rows per group of the list
    int entries;     // units, or with a split units - last + last x split
    int split;       // parts per unit of the last round (1: no split)
    int split_base;  // the last round's first entry
    int grid;        // blocks: min(entries, sms)
};
// false when the list would exceed 2^31 - 1 units.  ws_bytes: the key
// split's workspace (0: none).
bool prefill_plan(int B, int Hkv, int tq, int max_q_len, int sms, int D, size_t ws_bytes,
                  PrefillPlan *pl);

// workspace (nullable, 256-byte aligned, ws_bytes long) enables the key
// split with as many part slots as it holds.
cudaError_t launch_prefill(const PrefillParams &p, int D, int max_q_len, void *workspace,
                           size_t ws_bytes, cudaStream_t stream);
// table[0..B] = 0..B (kv_indptr), table[B+1+b] = idx ? idx[b] : b (kv_indices)
cudaError_t launch_contig_table(const int32_t *idx, int B, int32_t *table, cudaStream_t stream);
cudaError_t launch_rope_table(float *cos_sin, int max_pos, int D, double base,
                              cudaStream_t stream);
cudaError_t launch_split_decode(const DecodeParams &p, int D, cudaStream_t stream);
cudaError_t launch_combine(const CombineParams &p, cudaStream_t stream);
cudaError_t launch_fused_decode(const FusedParams &p, int D, int grid, cudaStream_t stream);
cudaError_t launch_piece_combine(const PieceCombineParams &p, int D, int grid_blocks,
                                 cudaStream_t stream);
// The per-step plan for the decode kernel's grid of `grid` blocks; p carries
// the shape, the tables, row_info and the status word.  entries: with the
// blocks' own entries, which the bf16 decode reads.
cudaError_t launch_decode_plan(const FusedParams &p, int grid, int32_t *plan, bool entries,
                               cudaStream_t stream);
int fused_heads_per_block(int Hkv);

// Resident split-decode blocks per SM for head dim D (shared-memory bound).
int split_decode_blocks_per_sm(int D);

} // namespace pkv
