// Attention of one query token per sequence over its pages.
//
// Every key of a sequence is read once per KV head and multiplied with the G
// <= 8 queries that share it, 4*G*d flops for 4*d bytes: memory bounds it, if
// the products cost next to nothing.  They go to the matrix instructions
// m16n8k16 in the transposed form, whose N = 8 is the group:
//   S^T [16 keys x 8] = K [16 x d] Q^T [d x 8],
//   O^T [d x 8]      += V^T [d x 16 keys] P^T [16 keys x 8].
// Both products contract or list the channels in an order that is free as
// long as both operands, or the output, follow it.  It is chosen so that the
// fragments of K and V are what 32-byte loads of the cached rows bring:
//  - K: lane (g, t) = (lane/4, lane%4) loads channels [64j + 16t, +16) of keys
//    g and g + 8; each four words are the A fragments of two k-steps whose
//    contraction index (2t, 2t+1, 2t+8, 2t+9) stands for four neighbours of
//    those channels.  Q's fragments are loaded with the same indexes.
//  - V: lane (g, t) loads channels [128j + 16g, +16) of keys 2t, 2t+1, 2t+8,
//    2t+9; a byte permute pairs two keys' values of one channel, and the eight
//    m-tiles of the block take the channel pairs (16g + 2i, 16g + 2i + 1).
//    What is left of a row whose length is no multiple of 64 or 128 takes shorter
//    loads.  Against 16 bytes a lane: 64 agents' own keys 134.2 -> 131.8 us
//    with the prefix, 16 sessions 76.5 -> 76.3, 4 x 8192 keys 29.1 -> 28.7.
//  - P: the accumulator of S^T holds (key g; queries 2t, 2t+1), the B fragment
//    wants (keys 2t, 2t+1; query g): an 8x8 transpose (movmatrix).
// So nothing passes through shared memory before the end, every warp runs on
// its own keys without a barrier, and the loads in flight are its registers.
//
// The softmax is a running one in powers of two, with one reference maximum
// per query and warp: a vote of the warp finds out whether any score passed it
// by more than 2^8, and only then is it renewed and the sums rescaled.
// P is rounded to the cache's type for its product.  For bfloat16 it is split
// into two terms (its rounding and what that left): 8 bits of P would add as
// much error again as the rounding of the output itself, and the second
// product is free under the loads.  A float16 P is relative to a reference 2^7
// lower, so that small probabilities keep their bits.
//
// The keys of all sequences and KV heads are one list of blocks of 64, dealt
// out evenly: CTA i of N takes blocks [i*total/N, (i+1)*total/N), so one wave of
// CTAs ends together whatever the lengths are (which only the device knows).
// Each CTA works the list out for itself from the lengths.  A KV head that one
// CTA has to itself is finished there; the others' parts go to merge_parts_kernel.
//
// Measured on B200, a call among others, on several GPUs: 16 sessions of up to
// 16385 keys, 8 queries of 64 channels a KV head, 75 to 80 us (77 to 81% of a
// plain copy); one of 131072 keys 90 us (92%); one of 2047 keys 8.3 us with the
// joining, in nine dependent loads.  The kernel alone on 64 sequences of up to
// 2048 keys of 128: 73.5 us (5.5 TB/s).  Memory bounds it; it has 4 KB or more in
// flight for each of 16 to 20 warps a multiprocessor.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"

namespace fathom {
namespace {

constexpr int kSplitThreads = 128;
constexpr int kSplitWarps = kSplitThreads / 32;
constexpr int kBlockKeys = 16;

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                        uint32_t a2, uint32_t a3, uint32_t b0,
                                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                 uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit values: row lane/4, columns 2*(lane%4) and the next.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

constexpr int kUnitKeys = kSplitWarps * kBlockKeys;

// First of the channel pair that lane group g has of m-tile i of O^T: 16
// neighbours of every 128, then 8 of a 64 and 4 of a 32 left over.
template <int E>
__device__ __forceinline__ constexpr int tile_channel(int i, int g)
{
    if (i < 8 * (E / 4)) return 128 * (i >> 3) + 16 * g + 2 * (i & 7);
    i -= 8 * (E / 4);
    if ((E & 2) && i < 4) return 128 * (E / 4) + 8 * g + 2 * i;
    return 32 * (E - 1) + 4 * g + 2 * (i & 3);
}

// A 16-byte load from shared memory that stays where it is written.
__device__ __forceinline__ uint4 load_shared(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
    return v;
}

struct SplitArgs {
    PagedView kv;
    PagedQuery q;
    PartsView pv;
    ScoreArgs score;
    int shared;       // keys that every sequence has at least (or none)
    int first;        // first key that this kernel reads (those before are another's)
    int max_len;
    int others;       // whether rows have parts of another kernel
    size_t full_at, cta_at;
    int2 *info;
    int *status;
};

// Registers allow this many CTAs per multiprocessor.
template <int E>
constexpr int split_residency()
{
    return E <= 2 ? 5 : E <= 4 ? 4 : E <= 6 ? 3 : 2;
}

// Blocks of 64 keys that sequence b has in this kernel's list for each KV head.
__device__ __forceinline__ int unit_count(const SplitArgs &a, int b)
{
    const int n = a.q.seq_lens[b];
    return refused_length(n, a.shared, a.max_len) || n <= a.first ? 0 : (n - a.first - 1) / kUnitKeys + 1;
}

template <typename T, int E>
__global__ void __launch_bounds__(kSplitThreads, split_residency<E>())
paged_split_kernel(const SplitArgs a)
{
    constexpr int d = 32 * E;
    constexpr int kTilesM = d / 16;                 // m-tiles of O^T
    constexpr bool kSplitP = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kWordsV = 2 * E;
    // What a warp loads at a time, 4 KB or more, must fit the registers with the accumulators: wide
    // heads keep Q's fragments (the same for every warp) in shared memory, narrow ones take
    // several blocks of keys.
    constexpr bool kSharedQ = E >= 3;
    constexpr int KB = E == 1 ? 2 : 1;
    __shared__ long long s_sum[kSplitWarps];
    __shared__ long long s_before;
    __shared__ int s_seq;
    __shared__ float s_m[kSplitWarps][8], s_l[kSplitWarps][8];
    __shared__ alignas(16) float s_o[kSplitWarps][8][d];
    __shared__ uint4 s_q[kSharedQ ? E : 1][32];
    // beside the kernel of the prefix nothing is read that an earlier one of this call writes
    if (!a.others) wait_for_earlier_kernels();
    let_next_kernel_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int H = a.kv.n_kv_heads, G = a.q.group, n_heads = G * H;

    // this CTA's run of the list: units [w, w_end), the first in sequence b,
    // before which lie `before` units of each KV head
    const int slice = (a.q.n_seqs + kSplitThreads - 1) / kSplitThreads;
    const int b0 = threadIdx.x * slice, b1 = min(a.q.n_seqs, b0 + slice);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += unit_count(a, b);
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, upto, off);
        if (lane >= off) upto += x;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int x = 0; x < kSplitWarps; ++x) {
        if (x < warp) upto += s_sum[x];
        total += s_sum[x];
    }
    total *= H;
    // at least a unit a CTA, so that none between two that share a row has none
    const long long sharers = min((long long)gridDim.x, total);
    long long w = sharers ? total * blockIdx.x / sharers : 0;
    const long long w_end = sharers ? min(total, total * (blockIdx.x + 1) / sharers) : 0;
    if (w >= w_end) {
        if (a.others) wait_for_earlier_kernels();
        return;
    }
    if ((upto - mine) * H <= w && w < upto * H) {
        long long before = upto - mine;
        int b = b0, n = unit_count(a, b);
        while (w >= (before + n) * H) {
            before += n;
            n = unit_count(a, ++b);
        }
        s_before = before;
        s_seq = b;
    }
    __syncthreads();
    int b = s_seq;
    long long before = s_before;
    bool bad = false;

    while (w < w_end) {
        int units = unit_count(a, b);
        while (w >= (before + units) * H) {         // the next sequence that has keys
            before += units;
            units = unit_count(a, ++b);
        }
        const int at_unit = (int)(w - before * H);
        const int h = at_unit / units, u0 = at_unit - h * units;
        const int u1 = (int)min((long long)units, u0 + (w_end - w));
        w += u1 - u0;
        const int n = a.q.seq_lens[b];
        const int lo = a.first + u0 * kUnitKeys, hi = (int)min((long long)n, a.first + (long long)u1 * kUnitKeys);

        // fragments of Q: query g of the group, zeros past it
        uint4 qr[kSharedQ ? 1 : E];
        __syncthreads();                            // the last run's, and its outputs, are read
        if (!kSharedQ || warp == 0) {
            const T *q = static_cast<const T *>(a.q.q) + b * a.q.q_ts + (h * G + g) * a.q.q_hs;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint4 w4 = g < G ? *reinterpret_cast<const uint4 *>(q + group_channel<E>(e, t))
                                       : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (kSharedQ)
                    s_q[e][lane] = w4;
                else
                    qr[e] = w4;
            }
        }
        if (kSharedQ) __syncthreads();
        float slope[2] = {0.0f, 0.0f};
        if (a.q.slopes) {
            if (2 * t < G) slope[0] = a.q.slopes[h * G + 2 * t] * kLog2e;
            if (2 * t + 1 < G) slope[1] = a.q.slopes[h * G + 2 * t + 1] * kLog2e;
        }
        const int32_t *table = a.kv.table + (size_t)b * a.kv.table_stride;
        const int shift = a.kv.page_shift, mask = (1 << shift) - 1;
        const uint16_t *K = static_cast<const uint16_t *>(a.kv.k) + h * a.kv.head_stride;
        const uint16_t *V = static_cast<const uint16_t *>(a.kv.v) + h * a.kv.head_stride;

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        float o[kTilesM][4];
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.0f;

        // pages of the blocks' halves, read one step ahead: eight keys from a
        // multiple of eight lie in one page
        int next[KB][2];
        const auto look_up = [&](int base) {
#pragma unroll
            for (int u = 0; u < KB; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = base + u * kUnitKeys + 8 * x;
                    next[u][x] = j < hi ? table[j >> shift] : -1;
                }
        };
        look_up(lo + warp * kBlockKeys);
        for (int base = lo + warp * kBlockKeys; base < hi; base += KB * kUnitKeys) {
            bool key[KB][2];
            uint4 kr[KB][2][E];
            uint32_t vr[KB][4][kWordsV];
#pragma unroll
            for (int u = 0; u < KB; ++u) {
                const int j0 = base + u * kUnitKeys;
                long long at[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = j0 + 8 * x;
                    const bool ok = next[u][x] >= 0 && next[u][x] < a.kv.n_pages;
                    bad |= j < hi && !ok;
                    at[x] = ok ? next[u][x] * a.kv.page_stride + (j & mask) * a.kv.slot_stride : -1;
                    key[u][x] = ok && j + g < hi;
                    load_groups<E>(K + at[x] + g * a.kv.slot_stride, t, key[u][x], kr[u][x]);
                }
                // keys past the end are not read: what their slots hold may be anything, NaN too
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int s = 2 * t + (x & 1);
                    const bool live = at[x >> 1] >= 0 && j0 + 8 * (x >> 1) + s < hi;
                    const uint16_t *p = V + at[x >> 1] + s * a.kv.slot_stride;
                    uint32_t *to = vr[u][x];
#pragma unroll
                    for (int e = 0; e < E / 4; ++e, to += 8) {
                        uint4 v0, v1;
                        load32(p + 128 * e + 16 * g, live, v0, v1);
                        to[0] = v0.x; to[1] = v0.y; to[2] = v0.z; to[3] = v0.w;
                        to[4] = v1.x; to[5] = v1.y; to[6] = v1.z; to[7] = v1.w;
                    }
                    if constexpr (E & 2) {
                        const uint4 w4 = live ? __ldg(reinterpret_cast<const uint4 *>(p + 128 * (E / 4) + 8 * g))
                                              : make_uint4(0u, 0u, 0u, 0u);
                        to[0] = w4.x; to[1] = w4.y; to[2] = w4.z; to[3] = w4.w;
                        to += 4;
                    }
                    if constexpr (E & 1) {
                        const uint2 w2 = live ? __ldg(reinterpret_cast<const uint2 *>(p + 32 * (E - 1) + 4 * g))
                                              : make_uint2(0u, 0u);
                        to[0] = w2.x; to[1] = w2.y;
                    }
                }
            }
            look_up(base + KB * kUnitKeys);
            // c: (key g; queries 2t, 2t+1), (key g + 8; the same)
            float c[KB][4];
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int u = 0; u < KB; ++u) {
#pragma unroll
                for (int x = 0; x < 4; ++x) c[u][x] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint4 q4 = kSharedQ ? load_shared(&s_q[kSharedQ ? e : 0][lane]) : qr[kSharedQ ? 0 : e];
                    mma16816<T>(c[u], kr[u][0][e].x, kr[u][1][e].x, kr[u][0][e].y, kr[u][1][e].y, q4.x, q4.y);
                    mma16816<T>(c[u], kr[u][0][e].z, kr[u][1][e].z, kr[u][0][e].w, kr[u][1][e].w, q4.z, q4.w);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float s = score_logit(c[u][x], a.score) -
                                    slope[x & 1] * (float)(n - 1 - (base + u * kUnitKeys + 8 * (x >> 1) + g));
                    c[u][x] = key[u][x >> 1] ? s : -INFINITY;
                    top[x & 1] = fmaxf(top[x & 1], c[u][x]);
                }
            }
            if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kRescale || top[1] > m[1] + kRescale)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], off));
                    const float renew = fmaxf(m[x], top[x]);
                    const float f = m[x] == renew ? 1.0f : exp2_fast(m[x] - renew);
                    m[x] = renew;
                    l[x] *= f;
#pragma unroll
                    for (int i = 0; i < kTilesM; ++i) {
                        o[i][x] *= f;
                        o[i][x + 2] *= f;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < KB; ++u) {
                float p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float ref = m[x & 1] == -INFINITY ? 0.0f : prob_reference<T>(m[x & 1]);
                    p[x] = exp2_fast(c[u][x] - ref);
                    if (kSplitP) l[x & 1] += p[x];
                }
                const uint32_t p0 = narrow2<T>(p[0], p[1]), p1 = narrow2<T>(p[2], p[3]);
                if constexpr (!kSplitP) {
                    // the sum of the rounded ones, those that V is weighted with
                    const float2 w0 = widen2<T>(p0), w1 = widen2<T>(p1);
                    l[0] += w0.x + w1.x;
                    l[1] += w0.y + w1.y;
                }
                const uint32_t f0 = transpose8x8(p0), f1 = transpose8x8(p1);
                uint32_t r0 = 0u, r1 = 0u;
                if constexpr (kSplitP) {
                    const float2 w0 = widen2<T>(p0), w1 = widen2<T>(p1);
                    r0 = transpose8x8(narrow2<T>(p[0] - w0.x, p[1] - w0.y));
                    r1 = transpose8x8(narrow2<T>(p[2] - w1.x, p[3] - w1.y));
                }
#pragma unroll
                for (int i = 0; i < kTilesM; ++i) {
                    const uint32_t a0 = __byte_perm(vr[u][0][i], vr[u][1][i], 0x5410);
                    const uint32_t a1 = __byte_perm(vr[u][0][i], vr[u][1][i], 0x7632);
                    const uint32_t a2 = __byte_perm(vr[u][2][i], vr[u][3][i], 0x5410);
                    const uint32_t a3 = __byte_perm(vr[u][2][i], vr[u][3][i], 0x7632);
                    mma16816<T>(o[i], a0, a1, a2, a3, f0, f1);
                    if constexpr (kSplitP) mma16816<T>(o[i], a0, a1, a2, a3, r0, r1);
                }
            }
        }

        // join the warps: maxima and sums of the 8 queries, then the outputs
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], off);
            if (g == 0) {
                s_m[warp][2 * t + x] = prob_reference<T>(m[x]);
                s_l[warp][2 * t + x] = l[x];
            }
#pragma unroll
            for (int i = 0; i < kTilesM; ++i) {
                const int c0 = tile_channel<E>(i, g);
                *reinterpret_cast<float2 *>(&s_o[warp][2 * t + x][c0]) = make_float2(o[i][x], o[i][x + 2]);
            }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == units;
        if (threadIdx.x == 0) {
            int2 *info = a.info + (size_t)b * H + h;
            if (u0 == 0) info->x = blockIdx.x;
            if (u1 == units) info->y = blockIdx.x;
        }
        for (int i = threadIdx.x; i < G * (d / 4); i += kSplitThreads) {
            const int qi = i / (d / 4), c0 = (i - qi * (d / 4)) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < kSplitWarps; ++x) top = fmaxf(top, s_m[x][qi]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kSplitWarps; ++x) {
                const float f = exp2_fast(s_m[x][qi] - ref);
                const float4 v = *reinterpret_cast<const float4 *>(&s_o[x][qi][c0]);
                acc.x += f * v.x;
                acc.y += f * v.y;
                acc.z += f * v.z;
                acc.w += f * v.w;
                sum += f * s_l[x][qi];
            }
            const int head = h * G + qi;
            if (whole && !a.others) {
                store_row<T>(a.q, b, head, c0, acc, sum);
            } else {
                const size_t place = whole ? a.full_at + (size_t)b * n_heads + head
                                           : a.cta_at + (2 * blockIdx.x + (u0 == 0 ? 1 : 0)) * (size_t)G + qi;
                *reinterpret_cast<float4 *>(a.pv.o + place * d + c0) = acc;
                if (c0 == 0) a.pv.ml[place] = make_float2(top, sum);
            }
        }
    }
    if (bad) set_status(a.status, FATHOM_ERR_INVALID_ARG);
    if (a.others) wait_for_earlier_kernels();       // so that whoever waits for this waits for those too
}

template <typename T, int E>
cudaError_t launch_one(const SplitArgs &a, int ctas, cudaStream_t stream)
{
    return launch_overlapped(paged_split_kernel<T, E>, dim3(ctas), kSplitThreads, 0, stream, a);
}

template <typename T>
cudaError_t launch_split(const SplitArgs &a, int ctas, cudaStream_t stream)
{
    switch (a.kv.head_dim / 32) {
    case 1: return launch_one<T, 1>(a, ctas, stream);
    case 2: return launch_one<T, 2>(a, ctas, stream);
    case 3: return launch_one<T, 3>(a, ctas, stream);
    case 4: return launch_one<T, 4>(a, ctas, stream);
    case 5: return launch_one<T, 5>(a, ctas, stream);
    case 6: return launch_one<T, 6>(a, ctas, stream);
    case 7: return launch_one<T, 7>(a, ctas, stream);
    default: return launch_one<T, 8>(a, ctas, stream);
    }
}

// One wave of CTAs, or one for every 64 keys where the batch may have fewer.
int split_ctas(int n_kv_heads, int head_dim, int n_seqs, int own)
{
    constexpr int residency[8] = {split_residency<1>(), split_residency<2>(), split_residency<3>(),
                                  split_residency<4>(), split_residency<5>(), split_residency<6>(),
                                  split_residency<7>(), split_residency<8>()};
    const long long units = ((long long)own + kUnitKeys - 1) / kUnitKeys * n_kv_heads * n_seqs;
    return (int)std::min<long long>(148 * residency[head_dim / 32 - 1], units);
}

struct Plan {
    PrefixPlan prefix;
    int first, ctas;
    size_t full_at, cta_at, places;
};
Plan plan_parts(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len, int prefix_len)
{
    Plan p{};
    const size_t rows = (size_t)n_seqs * n_kv_heads * group;
    p.prefix = plan_prefix(n_kv_heads, head_dim, n_seqs, group, prefix_len);
    p.first = p.prefix.parts ? prefix_len : 0;
    p.ctas = split_ctas(n_kv_heads, head_dim, n_seqs, max_len - p.first);
    p.full_at = rows * p.prefix.parts;
    p.cta_at = p.full_at + (p.prefix.parts ? rows : 0);
    p.places = p.cta_at + (size_t)p.ctas * 2 * group;
    return p;
}

}  // namespace

size_t paged_attention_bytes(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len,
                             int prefix_len)
{
    const Plan p = plan_parts(n_kv_heads, head_dim, n_seqs, group, max_len, prefix_len);
    return parts_bytes(p.places, head_dim) + round16((size_t)n_seqs * n_kv_heads * sizeof(int2));
}

// A smaller batch may have more parts: fewer blocks of rows are split into more runs.  Between two
// multiples of the sequences of a slot the runs are the same, so the most rows have the most places;
// from 148 blocks on there is one run.  Runs grow with the prefix and CTAs with the own keys, which
// are all of them where the prefix is left out.
size_t paged_attention_most_bytes(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len,
                                  int prefix_len)
{
    size_t most = 0;
    const auto consider = [&](long long seqs) {
        const size_t parts = plan_prefix(n_kv_heads, head_dim, (int)seqs, group, prefix_len).parts;
        if (parts) most = std::max(most, (size_t)seqs * n_kv_heads * group * (parts + 1));
    };
    const int slot = plan_prefix(n_kv_heads, head_dim, n_seqs, group, prefix_len).slot_seqs;
    consider(n_seqs);
    if (slot)
        for (int i = 1; i <= 2 * 149 && (long long)i * slot < n_seqs; ++i) consider((long long)i * slot);
    const size_t places = most + (size_t)split_ctas(n_kv_heads, head_dim, n_seqs, max_len) * 2 * group;
    return parts_bytes(places, head_dim) + round16((size_t)n_seqs * n_kv_heads * sizeof(int2));
}

cudaError_t launch_paged_attention(const PagedView &kv, const PagedQuery &q, int max_len,
                                   int prefix_len, void *ws, cudaStream_t stream)
{
    const Plan p = plan_parts(kv.n_kv_heads, kv.head_dim, q.n_seqs, q.group, max_len, prefix_len);
    SplitArgs a{};
    a.kv = kv;
    a.q = q;
    a.pv = parts_carve(ws, p.places, kv.head_dim);
    a.score = score_args(q.softmax_scale, q.softcap);
    a.shared = prefix_len;
    a.first = p.first;
    a.max_len = max_len;
    a.others = p.prefix.parts > 0;
    a.full_at = p.full_at;
    a.cta_at = p.cta_at;
    a.info = reinterpret_cast<int2 *>(static_cast<unsigned char *>(ws) + parts_bytes(p.places, kv.head_dim));
    a.status = device_status_ptr();
    cudaError_t e = cudaSuccess;
    if (p.prefix.parts) e = launch_paged_prefix(kv, q, p.prefix, a.pv, prefix_len, max_len, stream);
    if (e == cudaSuccess && p.ctas) {
        e = kv.dtype == FATHOM_BF16 ? launch_split<__nv_bfloat16>(a, p.ctas, stream)
                                    : launch_split<__half>(a, p.ctas, stream);
        note_launch();
    }
    if (e != cudaSuccess) return e;
    MergeArgs m{};
    m.pv = a.pv;
    m.q = q;
    m.n_heads = kv.n_kv_heads * q.group;
    m.head_dim = kv.head_dim;
    m.fixed = p.prefix.parts;
    m.lens_from = p.first;
    m.info = a.info;
    m.full_at = p.full_at;
    m.cta_at = p.cta_at;
    m.shared = prefix_len;
    m.max_len = max_len;
    return launch_merge_parts(m, kv.dtype, stream);
}

}  // namespace fathom
