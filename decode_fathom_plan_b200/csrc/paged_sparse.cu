// Attention of each query head over the keys its top-k selected, gathered from
// a paged cache: the paged, batched form of the attention after the scan
// (Fathom explainer, papers.ananclaw.com, arXiv 2609.17652, section
// 解决什么真问题: the decode step attends over the selected rows of the cache).
//
// Every list is its query's own, so a key row serves one query: 4*d flops for
// 4*d bytes of K and V, and only the reads count.  Four lanes share a key,
// lane t holding channels [64j + 16t, +16), so a 32-byte load of each brings a
// line of the row (16-byte loads: 10.9 us for 10.6 in the second case below),
// a warp has eight keys at once, a dot product costs two shuffles, and the sums over V need none: each group of four lanes keeps its
// own running maximum, sum and output, which are joined once at the end.
// A query's list is split into runs, one CTA each.  Registers (the output and
// the query: 48 of some 126 at d = 128) leave 16 warps of 4 KB in flight a
// multiprocessor; a second step's rows on their way at 12 warps was slower.
// Measured on B200: 512 rows of 1024 keys of 128 channels, lists of 16
// sequences, 55 us (4.3 TB/s, 67% of a plain copy, of single 256-byte rows); 32 rows of
// 2048 keys 10.6 us.
#include <math.h>

#include <algorithm>

#include "paged.cuh"

namespace fathom {
namespace {

constexpr int kSparseThreads = 128;
constexpr int kSparseWarps = kSparseThreads / 32;

struct SparseArgs {
    PagedView kv;
    PagedQuery q;
    PartsView pv;
    ScoreArgs score;
    const int32_t *idx;
    int k, run_keys, direct;
    int *status;
};

// grid (runs, query heads, sequences)
template <typename T, int E>
__global__ void __launch_bounds__(kSparseThreads)
paged_sparse_kernel(const SparseArgs a)
{
    constexpr int d = 32 * E;
    wait_for_earlier_kernels();
    let_next_kernel_start();
    __shared__ float s_m[kSparseWarps], s_l[kSparseWarps];
    __shared__ alignas(16) float s_o[kSparseWarps][d];
    const int b = blockIdx.z, head = blockIdx.y, run = blockIdx.x, n_heads = gridDim.y;
    const int h = head / a.q.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    const int n = a.q.seq_lens[b];
    const int32_t *table = a.kv.table + (size_t)b * a.kv.table_stride;
    const int32_t *idx = a.idx + ((size_t)b * n_heads + head) * a.k;
    const int shift = a.kv.page_shift, mask = (1 << shift) - 1;
    const uint16_t *K = static_cast<const uint16_t *>(a.kv.k) + h * a.kv.head_stride;
    const uint16_t *V = static_cast<const uint16_t *>(a.kv.v) + h * a.kv.head_stride;
    const float slope = a.q.slopes ? a.q.slopes[head] * kLog2e : 0.0f;

    // Offset of the listed key i, -1 where there is none.  A warp looks its keys up 32 at a time, a
    // lane each, one group ahead of the rows: a list entry, its page and its row are three
    // dependent loads.
    const int i1 = min(a.k, (run + 1) * a.run_keys);
    const auto entry = [&](int i) { return i < i1 ? idx[i] : -1; };
    bool bad = false;
    const auto look_up = [&](int key) -> long long {
        if (key == -1) return -1;
        int page = -1;
        if (key >= 0 && key < n && (key >> shift) < a.kv.table_stride) page = table[key >> shift];
        if (page >= 0 && page < a.kv.n_pages)
            return page * a.kv.page_stride + (key & mask) * a.kv.slot_stride;
        bad = true;
        return -1;
    };
    int i0 = run * a.run_keys + warp * 32;
    int key_next = entry(i0 + lane), key_then = entry(i0 + kSparseWarps * 32 + lane);
    uint4 qr[E];
    {
        const T *q = static_cast<const T *>(a.q.q) + b * a.q.q_ts + head * a.q.q_hs;
#pragma unroll
        for (int j = 0; j < E; ++j) qr[j] = *reinterpret_cast<const uint4 *>(q + group_channel<E>(j, t));
    }
    long long at_next = look_up(key_next);
    float m = -INFINITY, l = 0.0f, o[E][8];
#pragma unroll
    for (int j = 0; j < E; ++j)
#pragma unroll
        for (int x = 0; x < 8; ++x) o[j][x] = 0.0f;

    for (; i0 < i1; i0 += kSparseWarps * 32) {
        const int key_of = key_next;
        const long long at_of = at_next;
        key_next = key_then;
        key_then = entry(i0 + 2 * kSparseWarps * 32 + lane);
        at_next = look_up(key_next);
#pragma unroll 2
        for (int it = 0; it < 4; ++it) {
            const int from = it * 8 + (lane >> 2);
            const int key = __shfl_sync(0xFFFFFFFFu, key_of, from);
            const long long at = __shfl_sync(0xFFFFFFFFu, at_of, from);
            uint4 kr[E], vr[E];
            load_groups<E>(K + at, t, at >= 0, kr);
            load_groups<E>(V + at, t, at >= 0, vr);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const uint32_t ku[4] = {kr[j].x, kr[j].y, kr[j].z, kr[j].w};
                const uint32_t qu[4] = {qr[j].x, qr[j].y, qr[j].z, qr[j].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 kf = widen2<T>(ku[x]), qf = widen2<T>(qu[x]);
                    dot = fmaf(kf.x, qf.x, fmaf(kf.y, qf.y, dot));
                }
            }
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, 1);
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, 2);
            const float s = at >= 0 ? score_logit(dot, a.score) - slope * (float)(n - 1 - key) : -INFINITY;
            if (__any_sync(0xFFFFFFFFu, s > m + kRescale)) {
                const float next = fmaxf(m, s);
                const float w = m == next ? 1.0f : exp2_fast(m - next);
                m = next;
                l *= w;
#pragma unroll
                for (int j = 0; j < E; ++j)
#pragma unroll
                    for (int x = 0; x < 8; ++x) o[j][x] *= w;
            }
            const float p = exp2_fast(s - (m == -INFINITY ? 0.0f : m));
            l += p;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const uint32_t vu[4] = {vr[j].x, vr[j].y, vr[j].z, vr[j].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 vf = widen2<T>(vu[x]);
                    o[j][2 * x] = fmaf(p, vf.x, o[j][2 * x]);
                    o[j][2 * x + 1] = fmaf(p, vf.y, o[j][2 * x + 1]);
                }
            }
        }
    }
    if (bad) set_status(a.status, FATHOM_ERR_INVALID_ARG);

    // join the warp's eight key groups, then the warps
    float top = m;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    const float w = top == -INFINITY ? 0.0f : exp2_fast(m - top);
    l *= w;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
#pragma unroll
    for (int j = 0; j < E; ++j)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            o[j][x] *= w;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) o[j][x] += __shfl_xor_sync(0xFFFFFFFFu, o[j][x], off);
        }
    if (lane < 4) {
#pragma unroll
        for (int j = 0; j < E; ++j)
#pragma unroll
            for (int x = 0; x < 8; x += 4)
                *reinterpret_cast<float4 *>(&s_o[warp][group_channel<E>(j, t) + x]) =
                    make_float4(o[j][x], o[j][x + 1], o[j][x + 2], o[j][x + 3]);
        if (lane == 0) {
            s_m[warp] = top;
            s_l[warp] = l;
        }
    }
    __syncthreads();
    const int c0 = threadIdx.x * 4;
    if (c0 >= d) return;
    top = -INFINITY;
#pragma unroll
    for (int x = 0; x < kSparseWarps; ++x) top = fmaxf(top, s_m[x]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < kSparseWarps; ++x) {
        const float f = exp2_fast(s_m[x] - ref);
        const float4 v = *reinterpret_cast<const float4 *>(&s_o[x][c0]);
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
        sum += f * s_l[x];
    }
    if (a.direct) {
        store_row<T>(a.q, b, head, c0, acc, sum);
    } else {
        const size_t place = ((size_t)b * n_heads + head) * gridDim.x + run;
        *reinterpret_cast<float4 *>(a.pv.o + place * d + c0) = acc;
        if (c0 == 0) a.pv.ml[place] = make_float2(top, sum);
    }
}

template <typename T>
cudaError_t launch_sparse(const SparseArgs &a, dim3 grid, cudaStream_t stream)
{
    const auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, kSparseThreads, 0, stream, a); };
    switch (a.kv.head_dim / 32) {
    case 1: return go(paged_sparse_kernel<T, 1>);
    case 2: return go(paged_sparse_kernel<T, 2>);
    case 3: return go(paged_sparse_kernel<T, 3>);
    case 4: return go(paged_sparse_kernel<T, 4>);
    case 5: return go(paged_sparse_kernel<T, 5>);
    case 6: return go(paged_sparse_kernel<T, 6>);
    case 7: return go(paged_sparse_kernel<T, 7>);
    default: return go(paged_sparse_kernel<T, 8>);
    }
}

// Keys of a CTA: a group of 32 for each warp, or several (whose look-ups then overlap) where
// there are rows enough.
constexpr int kLeastRun = 128, kMostRun = 512;
constexpr long long kFullGpu = 148 * 8;
int sparse_run_keys(int n_rows, int k)
{
    const long long groups = (long long)n_rows * k / kFullGpu;
    return (int)std::min<long long>(std::max<long long>(groups / kLeastRun * kLeastRun, kLeastRun), kMostRun);
}
int sparse_runs(int n_rows, int k) { return (k - 1) / sparse_run_keys(n_rows, k) + 1; }

}  // namespace

size_t paged_sparse_bytes(int n_rows, int head_dim, int k)
{
    const int runs = sparse_runs(n_rows, k);
    return runs == 1 ? 0 : parts_bytes((size_t)n_rows * runs, head_dim);
}

// Fewer rows or keys may have more runs.  Runs of r keys (but the longest) are taken while
// rows * k < kFullGpu * (r + kLeastRun) = p, and rows have several only where k > r: then there are
// at most p / r rows, with rows * ceil(k / r) <= p / r + rows parts.
size_t paged_sparse_most_bytes(int n_rows, int head_dim, int k)
{
    long long most = 0;
    for (int r = kLeastRun; r <= kMostRun; r += kLeastRun) {
        if (k <= r) break;
        long long parts = (long long)n_rows * ((k - 1) / r + 1);
        if (r < kMostRun) {
            const long long p = kFullGpu * (r + kLeastRun);
            parts = std::min(parts, p / r + std::min<long long>(n_rows, p / r));
        }
        most = std::max(most, parts);
    }
    return most ? parts_bytes((size_t)most, head_dim) : 16;
}

cudaError_t launch_paged_sparse(const PagedView &kv, const PagedQuery &q, const int32_t *idx, int k,
                                void *ws, cudaStream_t stream)
{
    const int n_heads = kv.n_kv_heads * q.group, rows = q.n_seqs * n_heads;
    const int runs = sparse_runs(rows, k);
    SparseArgs a{};
    a.kv = kv;
    a.q = q;
    a.score = score_args(q.softmax_scale, q.softcap);
    a.idx = idx;
    a.k = k;
    a.run_keys = sparse_run_keys(rows, k);
    a.direct = runs == 1;
    if (!a.direct) a.pv = parts_carve(ws, (size_t)rows * runs, kv.head_dim);
    a.status = device_status_ptr();
    const dim3 grid(runs, n_heads, q.n_seqs);
    note_launch();
    const cudaError_t e = kv.dtype == FATHOM_BF16 ? launch_sparse<__nv_bfloat16>(a, grid, stream)
                                                  : launch_sparse<__half>(a, grid, stream);
    if (e != cudaSuccess || a.direct) return e;
    MergeArgs m{};
    m.pv = a.pv;
    m.q = q;
    m.n_heads = n_heads;
    m.head_dim = kv.head_dim;
    m.fixed = runs;
    m.lens_from = -1;
    return launch_merge_parts(m, kv.dtype, stream);
}

}  // namespace fathom
