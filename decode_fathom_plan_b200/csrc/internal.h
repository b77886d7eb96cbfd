// Host-side interfaces between the C-ABI layer and the kernel launchers
// (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <nvtx3/nvToolsExt.h>

#include "fathom.h"

namespace fathom {

// Named NVTX range for the lifetime of a scope: marks each C-ABI call and
// each scan phase on a profiler's timeline (Nsight Systems); without a
// profiler attached the calls return at once.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// Address of this device's status word (a __device__ int).
int *device_status_ptr();
// Count one kernel launch (for fathom_launch_count).
void note_launch(int n = 1);
// Limit of a kernel's wait in nanoseconds (fathom_set_wait_limit).
unsigned long long wait_limit_ns();
// Record the CUDA error of a failed step (reported on stderr once per site
// by the C-ABI layer) and return it.
cudaError_t note_error(cudaError_t e, const char *site);

// Code width b of an index: 4, or 8 for the 8-plane variant (the C ABI
// reads 0 as 4 and rejects anything else before a launcher runs).
inline int index_bits(const fathom_index &ix) { return ix.bits == 8 ? 8 : 4; }
// Statistics rows per KV head: 1, or the blocks the planes can hold when the
// index has grouped per-token-block scales (block_keys > 0).
inline int index_blocks(const fathom_index &ix)
{
    return ix.block_keys ? (int)(((long long)ix.n_words * 32 + ix.block_keys - 1) / ix.block_keys)
                         : 1;
}

// ---- pack.cu
cudaError_t launch_pack(const float *keys, const fathom_index &ix, uint32_t *ws_minmax,
                        cudaStream_t stream);
// sigma^2 of every (head, channel) from its exact sums and the key count n
// (combined over the blocks of a block-scaled index).
cudaError_t launch_channel_stats(const fathom_index &ix, int n, cudaStream_t stream);
// Appends m keys (device float32 [H][m][d]) to a block-scaled index whose
// ix.n_keys is a whole number of blocks: the new blocks are packed on their
// own, sigma^2 is recomputed for ix.n_keys + m keys.
cudaError_t launch_append_blocks(const float *keys, const fathom_index &ix, int m,
                                 cudaStream_t stream);

// ---- append.cu
// Appends m keys (device float32 [H][m][d]) at positions ix.n_keys.. and
// recomputes sigma^2 for ix.n_keys + m keys; clamped may be null.
cudaError_t launch_append(const float *keys, const fathom_index &ix, int m, uint32_t *clamped,
                          cudaStream_t stream);

// ---- plan.cu
cudaError_t launch_plan(const fathom_index &ix, const uint16_t *q, const int32_t *budget,
                        int32_t fixed_r, bool fixed, uint8_t *t, uint8_t *t_union,
                        uint64_t *bytes, cudaStream_t stream);
cudaError_t launch_plan_marginal(const fathom_index &ix, const uint16_t *q, const int32_t *budget,
                                 uint8_t *t, uint8_t *t_union, uint64_t *bytes,
                                 cudaStream_t stream);

// ---- lift.cu
// An 8-plane index's scan arguments rewritten for the 4-plane scan over 2d
// nibble channels (the planes themselves need no change).
struct LiftArgs {
    const float *mn, *scale;     // [stat_rows][d]: one row per (head, scale block)
    const uint16_t *q;           // [Q][d]
    const uint8_t *t, *tu;       // [Q][d], [H][d]
    float *mn2, *scale2;         // [stat_rows][2d]
    uint16_t *q2;                // [Q][2d]
    uint8_t *t2, *tu2;           // [Q][2d], [H][2d]
    int H, Q, d, stat_rows;
};
// Workspace bytes of the primed arrays (each rounded up to 16 bytes).
size_t lift_bytes(int H, int Q, int d, int stat_rows);
// Points the primed arrays of *a into ws (lift_bytes(...) bytes, 16-byte
// aligned) and sets its sizes; the caller sets the inputs.
void lift_carve(void *ws, int H, int Q, int d, int stat_rows, LiftArgs *a);
cudaError_t launch_lift(const LiftArgs &a, cudaStream_t stream);

// ---- fetch.cu
// One host-resident index to fetch: for each of its n_channels = H*d
// (head, channel) pairs, the first t_union[hc] slots of n_words words.
struct FetchJob {
    const uint32_t *src;       // device-mapped host planes [H][d][4][n_words]
    uint32_t *dst;             // device ring slot, same layout
    const uint8_t *t_union;    // [H][d]
    int n_channels;
    int n_words;
};
// CTAs per multiprocessor of a fetch that shares the GPU with the scoring
// kernels of the previous unit (the link needs few SMs to stay busy).
constexpr int kFetchCtasPerSmShared = 2;
cudaError_t launch_fetch(const FetchJob *jobs, int n_jobs, cudaStream_t stream, int ctas_per_sm);

// ---- attention.cu
// Split-K runs per query for k selected keys.
int attention_splits(int k);
// Attention of Q = H*G queries over their k selected keys; part: workspace
// of Q * attention_splits(k) * (d + 2) floats.
cudaError_t launch_attention(const float *keys, const float *values, int H, int G, int d, int n,
                             const uint16_t *q_bf16, const int32_t *idx, int k, float scale,
                             float *out, float *part, cudaStream_t stream);

// ---- merge.cu
constexpr int kMaxMergeShards = 64;
constexpr int kMaxMergeCandidates = 16384;   // S * k_s per query (shared memory)
struct MergeOffsets {
    long long offset[kMaxMergeShards];       // first global key of each shard
};
size_t merge_smem_bytes(int S, int k_s);
cudaError_t launch_merge(const int32_t *idx, const float *score, const MergeOffsets &off, int S,
                         int Q, int k_s, int k, int32_t *out_idx, float *out_score,
                         cudaStream_t stream);

// ---- rotary.cu
// One kind of head rows (queries, keys or values) on its way through
// launch_rows: input view, output view (out_ts unused when paged), norm weight
// or null, and whether its pairs are rotated.
struct RowSet {
    const void *in;
    void *out;
    const void *weight;
    long long in_ts, in_hs, out_ts, out_hs;
    int heads;
    int out_dtype;
    int turn;
    // set by the launcher: whether rows only move, tokens and heads of a CTA,
    // CTAs per token tile
    int copy, tile, heads_per_cta, chunks;
};
struct RowsArgs {
    RowSet set[2];               // heads 0 where there is none
    const int32_t *pos;          // [n_tokens]
    const double *turns;         // [rotary_dim / 2]
    float magnitude, eps;
    int n_tokens, head_dim;
    int rotary_dim, interleaved; // rotary_dim 0: no rotation
    // rows that go to the pages of a cache: out is its k or v, out_hs its
    // head stride
    int paged;
    const int32_t *seq, *table;
    int n_seqs, table_stride, n_pages, page_shift;
    long long page_stride, slot_stride;
    // set by the launcher
    int lanes;                   // that hold a row
    int blocks0;                 // CTAs of set 0
    float inv_dim;
    int *status;
};
// dtype: type of every input row and weight.  vector: all bases and strides
// allow 16-byte accesses of 8 elements and rotary_dim is a multiple of 16.
cudaError_t launch_rows(RowsArgs a, int dtype, bool vector, cudaStream_t stream);

// ---- paged_attention.cu, paged_sparse.cu
struct PagedView {               // a paged cache and its table, device addresses
    const void *k, *v;
    long long page_stride, head_stride, slot_stride;
    int n_pages, page_shift, n_kv_heads, head_dim, dtype;
    const int32_t *table;
    int table_stride;
};
struct PagedQuery {              // the query rows, the scores and the output rows
    const void *q;
    void *out;
    long long q_ts, q_hs, out_ts, out_hs;
    const int32_t *seq_lens;
    const float *slopes;
    float softmax_scale, softcap;
    int n_seqs, group;
};
// What a call uses, and the most that any call of up to these sizes does.
size_t paged_attention_bytes(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len,
                             int prefix_len);
size_t paged_attention_most_bytes(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len,
                                  int prefix_len);
cudaError_t launch_paged_attention(const PagedView &kv, const PagedQuery &q, int max_len,
                                   int prefix_len, void *ws, cudaStream_t stream);
size_t paged_sparse_bytes(int n_rows, int head_dim, int k);
size_t paged_sparse_most_bytes(int n_rows, int head_dim, int k);
cudaError_t launch_paged_sparse(const PagedView &kv, const PagedQuery &q, const int32_t *idx, int k,
                                void *ws, cudaStream_t stream);

// ---- paged_merge.cu
// Parts of attention rows that were computed apart.  The part at place p has
// the sum sum_j 2^(s_j - max) V_j [d] at o + p*d and (max, sum_j 2^(s_j - max))
// at ml[p], s in powers of two.
struct PartsView {
    float *o;
    float2 *ml;
};
size_t round16(size_t b);
size_t parts_bytes(size_t places, int head_dim);
// Points the parts into ws (parts_bytes(...) bytes, 16-byte aligned).
PartsView parts_carve(void *ws, size_t places, int head_dim);
struct MergeArgs {
    PartsView pv;
    PagedQuery q;
    int n_heads, head_dim;
    int fixed;            // parts that every row has, at row*fixed
    // Keys past the first lens_from of a sequence were split evenly over CTAs
    // (lens_from < 0: the fixed parts are all).  info[b*H + h] is the first
    // and the last CTA of a KV head's rows.  One CTA: the row is finished, or
    // with fixed parts beside it one part at full_at + row.  Several: the
    // first CTA's part at cta_at + (2*cta + 1)*G + g, the others' at
    // cta_at + 2*cta*G + g.
    int lens_from;
    const int2 *info;
    size_t full_at, cta_at;
    int shared, max_len;  // lengths outside {0} and [shared, max_len] are refused
    int *status;          // set by the launcher
};
// out[row] = sum of the row's parts over the sum of their weights, zeros where
// that is 0.
cudaError_t launch_merge_parts(const MergeArgs &a, int dtype, cudaStream_t stream);

// ---- paged_prefix.cu
// How the products over a shared prefix are split: sequences of a block of up
// to 128 rows, CTAs of one or two blocks, runs of key tiles, places per row.
struct PrefixPlan {
    int slot_seqs, two_blocks, row_groups, n_tiles, splits, parts;
};
PrefixPlan plan_prefix(int n_kv_heads, int head_dim, int n_seqs, int group, int prefix_len);
// Writes the first p.parts places of every row.
cudaError_t launch_paged_prefix(const PagedView &kv, const PagedQuery &q, const PrefixPlan &p,
                                const PartsView &pv, int prefix_len, int max_len, cudaStream_t stream);

// ---- scan.cu
struct ScanSessionArgs {
    const fathom_index *ix;
    const uint16_t *q;
    const uint8_t *t;
    const uint8_t *t_union;
    int32_t *out_idx;
    float *out_score;
};

// Workspace bytes for a batch of sessions (single call = batch of one).
size_t scan_workspace_bytes(const fathom_index *sessions, int n_sessions, int k);

// Profiling events around the dominant kernel of a scan call
// (FATHOM_SCAN_PROFILE): the fetch sequence when any index is host-resident, else
// the main scan.
struct ScanProfileHook {
    bool enabled;
    cudaEvent_t begin, end;
    bool recorded;   // set when that kernel was launched and timed
};

cudaError_t launch_scan(const ScanSessionArgs *sessions, int n_sessions, int k,
                        void *ws, size_t ws_bytes, uint32_t flags, cudaStream_t stream,
                        ScanProfileHook *hook);

}  // namespace fathom
