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
// fragments of K and V are what 16-byte loads of the cached rows bring:
//  - K: lane (g, t) = (lane/4, lane%4) loads channels [32j + 8t, +8) of keys g
//    and g + 8; the four words are the A fragments of two k-steps whose
//    contraction index (2t, 2t+1, 2t+8, 2t+9) stands for channels 32j + 8t +
//    (4s..4s+3).  Q's fragments are loaded with the same indexes.
//  - V: lane (g, t) loads channels [64j + 8g, +8) of keys 2t, 2t+1, 2t+8,
//    2t+9; a byte permute pairs two keys' values of one channel, and the four
//    m-tiles of the block take the channel pairs (8g + 2i, 8g + 2i + 1).
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
// product is free under the loads.
//
// The keys of a sequence are split into chunks, one CTA each, joined by
// merge_parts_kernel; a batch whose longest sequence is one chunk writes its
// outputs itself.
#include <math.h>

#include <algorithm>

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

struct SplitArgs {
    PagedView kv;
    PagedQuery q;
    PartsView pv;
    ScoreArgs score;
    int shared;       // keys that every sequence has at least (or none)
    int first;        // first key that this kernel reads (those before are another's)
    int fixed;        // places of a row before those of its own part
    int chunk;        // keys of a CTA, a multiple of kBlockKeys
    int max_len;
    int direct;       // one part per row: write the output itself
    int *status;
};

// grid (chunks, KV heads, sequences)
template <typename T, int E>
__global__ void __launch_bounds__(kSplitThreads)
paged_split_kernel(const SplitArgs a)
{
    constexpr int d = 32 * E;
    constexpr int kTilesM = d / 16;                 // m-tiles of O^T
    constexpr bool kSplitP = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
    __shared__ float s_m[kSplitWarps][8], s_l[kSplitWarps][8];
    __shared__ alignas(16) float s_o[kSplitWarps][8][d];
    const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
    const int G = a.q.group, n_heads = G * a.kv.n_kv_heads;
    const int n = a.q.seq_lens[b];
    const bool refused = n < 0 || n > a.max_len || (n > 0 && n < a.shared);
    if (refused && threadIdx.x == 0) set_status(a.status, FATHOM_ERR_INVALID_ARG);
    const int lo = a.first + split * a.chunk;
    const int hi = refused ? 0 : min(n, lo + a.chunk);
    if (lo >= hi && !(a.direct && split == 0)) return;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    // fragments of Q: query g of the group, zeros past it
    uint32_t qf[E][4];
    {
        const T *q = static_cast<const T *>(a.q.q) + b * a.q.q_ts + (h * G + g) * a.q.q_hs + 8 * t;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (g < G) u = *reinterpret_cast<const uint4 *>(q + 32 * j);
            qf[j][0] = u.x; qf[j][1] = u.y; qf[j][2] = u.z; qf[j][3] = u.w;
        }
    }
    float slope[2] = {0.0f, 0.0f};
    if (a.q.slopes) {
        if (2 * t < G) slope[0] = a.q.slopes[h * G + 2 * t] * kLog2e;
        if (2 * t + 1 < G) slope[1] = a.q.slopes[h * G + 2 * t + 1] * kLog2e;
    }
    const int32_t *table = a.kv.table + (size_t)b * a.kv.table_stride;
    const int shift = a.kv.page_shift, mask = (1 << shift) - 1;
    const T *K = static_cast<const T *>(a.kv.k) + h * a.kv.head_stride;
    const T *V = static_cast<const T *>(a.kv.v) + h * a.kv.head_stride;

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float o[kTilesM][4];
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] = 0.0f;
    bool bad = false;

    for (int base = lo + warp * kBlockKeys; base < hi; base += kSplitWarps * kBlockKeys) {
        // eight keys from a multiple of eight lie in one page
        long long at[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = base + 8 * x;
            const int page = j < hi ? table[j >> shift] : -1;
            const bool ok = page >= 0 && page < a.kv.n_pages;
            bad |= j < hi && !ok;
            at[x] = ok ? page * a.kv.page_stride + (j & mask) * a.kv.slot_stride : -1;
        }
        const bool key[2] = {at[0] >= 0 && base + g < hi, at[1] >= 0 && base + 8 + g < hi};
        uint4 kr[2][E];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const T *p = K + at[x] + g * a.kv.slot_stride + 8 * t;
#pragma unroll
            for (int j = 0; j < E; ++j)
                kr[x][j] = key[x] ? __ldg(reinterpret_cast<const uint4 *>(p + 32 * j))
                                  : make_uint4(0u, 0u, 0u, 0u);
        }
        // keys past the end are not read: what their slots hold may be anything, NaN too
        uint32_t vr[4][(E / 2) * 4 + (E & 1) * 2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int s = 2 * t + (x & 1);
            const bool live = at[x >> 1] >= 0 && base + 8 * (x >> 1) + s < hi;
            const T *p = V + at[x >> 1] + s * a.kv.slot_stride;
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const uint4 u = live ? __ldg(reinterpret_cast<const uint4 *>(p + 64 * j + 8 * g))
                                     : make_uint4(0u, 0u, 0u, 0u);
                vr[x][4 * j] = u.x; vr[x][4 * j + 1] = u.y; vr[x][4 * j + 2] = u.z; vr[x][4 * j + 3] = u.w;
            }
            if constexpr (E & 1) {
                const uint2 u = live ? __ldg(reinterpret_cast<const uint2 *>(p + 32 * (E - 1) + 4 * g))
                                     : make_uint2(0u, 0u);
                vr[x][(E / 2) * 4] = u.x; vr[x][(E / 2) * 4 + 1] = u.y;
            }
        }
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < E; ++j) {
            mma16816<T>(c, kr[0][j].x, kr[1][j].x, kr[0][j].y, kr[1][j].y, qf[j][0], qf[j][1]);
            mma16816<T>(c, kr[0][j].z, kr[1][j].z, kr[0][j].w, kr[1][j].w, qf[j][2], qf[j][3]);
        }
        // c: (key g; queries 2t, 2t+1), (key g + 8; the same)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float s = score_logit(c[x], a.score) -
                            slope[x & 1] * (float)(n - 1 - (base + 8 * (x >> 1) + g));
            c[x] = key[x >> 1] ? s : -INFINITY;
        }
        float top[2] = {fmaxf(c[0], c[2]), fmaxf(c[1], c[3])};
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kRescale || top[1] > m[1] + kRescale)) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], off));
                const float next = fmaxf(m[x], top[x]);
                const float w = m[x] == next ? 1.0f : exp2_fast(m[x] - next);
                m[x] = next;
                l[x] *= w;
#pragma unroll
                for (int i = 0; i < kTilesM; ++i) {
                    o[i][x] *= w;
                    o[i][x + 2] *= w;
                }
            }
        }
        float p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float ref = m[x & 1] == -INFINITY ? 0.0f : m[x & 1];
            p[x] = exp2_fast(c[x] - ref);
            l[x & 1] += p[x];
        }
        const uint32_t hi0 = narrow2<T>(p[0], p[1]), hi1 = narrow2<T>(p[2], p[3]);
        const uint32_t b0 = transpose8x8(hi0), b1 = transpose8x8(hi1);
        uint32_t r0 = 0u, r1 = 0u;
        if constexpr (kSplitP) {
            const float2 f0 = widen2<T>(hi0), f1 = widen2<T>(hi1);
            r0 = transpose8x8(narrow2<T>(p[0] - f0.x, p[1] - f0.y));
            r1 = transpose8x8(narrow2<T>(p[2] - f1.x, p[3] - f1.y));
        }
#pragma unroll
        for (int i = 0; i < kTilesM; ++i) {
            const uint32_t a0 = __byte_perm(vr[0][i], vr[1][i], 0x5410);
            const uint32_t a1 = __byte_perm(vr[0][i], vr[1][i], 0x7632);
            const uint32_t a2 = __byte_perm(vr[2][i], vr[3][i], 0x5410);
            const uint32_t a3 = __byte_perm(vr[2][i], vr[3][i], 0x7632);
            mma16816<T>(o[i], a0, a1, a2, a3, b0, b1);
            if constexpr (kSplitP) mma16816<T>(o[i], a0, a1, a2, a3, r0, r1);
        }
    }
    if (bad) set_status(a.status, FATHOM_ERR_INVALID_ARG);

    // join the warps: maxima and sums of the 8 queries, then the outputs
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], off);
        if (g == 0) {
            s_m[warp][2 * t + x] = m[x];
            s_l[warp][2 * t + x] = l[x];
        }
#pragma unroll
        for (int i = 0; i < kTilesM; ++i) {
            const int c0 = i < 4 * (E / 2) ? 64 * (i >> 2) + 8 * g + 2 * (i & 3)
                                           : 32 * (E - 1) + 4 * g + 2 * (i & 3);
            *reinterpret_cast<float2 *>(&s_o[warp][2 * t + x][c0]) = make_float2(o[i][x], o[i][x + 2]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * (d / 4); i += kSplitThreads) {
        const int qi = i / (d / 4), c0 = (i - qi * (d / 4)) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) top = fmaxf(top, s_m[w][qi]);
        const float ref = top == -INFINITY ? 0.0f : top;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) {
            const float f = exp2_fast(s_m[w][qi] - ref);
            const float4 v = *reinterpret_cast<const float4 *>(&s_o[w][qi][c0]);
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
            sum += f * s_l[w][qi];
        }
        const int head = h * G + qi;
        if (a.direct) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint16_t *out = static_cast<uint16_t *>(a.q.out) + b * a.q.out_ts + head * a.q.out_hs + c0;
            *reinterpret_cast<uint2 *>(out) = make_uint2(narrow2<T>(acc.x * inv, acc.y * inv),
                                                         narrow2<T>(acc.z * inv, acc.w * inv));
        } else {
            const size_t place = (size_t)(b * n_heads + head) * a.pv.parts + a.fixed + split;
            *reinterpret_cast<float4 *>(a.pv.o + place * d + c0) = acc;
            if (c0 == 0) a.pv.ml[place] = make_float2(top, sum);
        }
    }
}

template <typename T>
void launch_split(const SplitArgs &a, dim3 grid, cudaStream_t stream)
{
    switch (a.kv.head_dim / 32) {
    case 1: paged_split_kernel<T, 1><<<grid, kSplitThreads, 0, stream>>>(a); break;
    case 2: paged_split_kernel<T, 2><<<grid, kSplitThreads, 0, stream>>>(a); break;
    case 3: paged_split_kernel<T, 3><<<grid, kSplitThreads, 0, stream>>>(a); break;
    case 4: paged_split_kernel<T, 4><<<grid, kSplitThreads, 0, stream>>>(a); break;
    case 5: paged_split_kernel<T, 5><<<grid, kSplitThreads, 0, stream>>>(a); break;
    case 6: paged_split_kernel<T, 6><<<grid, kSplitThreads, 0, stream>>>(a); break;
    case 7: paged_split_kernel<T, 7><<<grid, kSplitThreads, 0, stream>>>(a); break;
    default: paged_split_kernel<T, 8><<<grid, kSplitThreads, 0, stream>>>(a); break;
    }
}

// Keys of one CTA: enough CTAs for the GPU where the batch allows it, at least
// one block for each warp and at most 1024 keys, so that uneven lengths even out.
int chunk_keys(int n_kv_heads, int n_seqs, int own)
{
    const long long want = (long long)own * n_kv_heads * n_seqs / (148 * 8);
    const long long chunk = (want + 63) / 64 * 64;
    return (int)std::min<long long>(std::max<long long>(chunk, 64), 1024);
}

struct Plan {
    PrefixPlan prefix;
    int first, chunk, chunks, parts, direct;
};
Plan plan_parts(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len, int prefix_len)
{
    Plan p{};
    p.prefix = plan_prefix(n_kv_heads, head_dim, n_seqs, group, prefix_len);
    p.first = p.prefix.parts ? prefix_len : 0;
    const int own = max_len - p.first;
    p.chunk = chunk_keys(n_kv_heads, n_seqs, own);
    p.chunks = (own + p.chunk - 1) / p.chunk;
    p.parts = p.prefix.parts + p.chunks;
    p.direct = p.parts == 1 && p.chunks == 1;
    return p;
}

}  // namespace

size_t paged_attention_bytes(int n_kv_heads, int head_dim, int n_seqs, int group, int max_len,
                             int prefix_len)
{
    const Plan p = plan_parts(n_kv_heads, head_dim, n_seqs, group, max_len, prefix_len);
    return p.direct ? 0 : parts_bytes(n_seqs * n_kv_heads * group, head_dim, p.parts);
}

cudaError_t launch_paged_attention(const PagedView &kv, const PagedQuery &q, int max_len,
                                   int prefix_len, void *ws, cudaStream_t stream)
{
    const Plan p = plan_parts(kv.n_kv_heads, kv.head_dim, q.n_seqs, q.group, max_len, prefix_len);
    const int n_heads = kv.n_kv_heads * q.group;
    SplitArgs a{};
    a.kv = kv;
    a.q = q;
    if (!p.direct) a.pv = parts_carve(ws, q.n_seqs * n_heads, kv.head_dim, p.parts);
    a.score = score_args(q.softmax_scale, q.softcap);
    a.shared = prefix_len;
    a.first = p.first;
    a.fixed = p.prefix.parts;
    a.chunk = p.chunk;
    a.max_len = max_len;
    a.direct = p.direct;
    a.status = device_status_ptr();
    if (p.prefix.parts) {
        const cudaError_t e = launch_paged_prefix(kv, q, p.prefix, a.pv, prefix_len, stream);
        if (e != cudaSuccess) return e;
    }
    if (p.chunks) {
        const dim3 grid(p.chunks, kv.n_kv_heads, q.n_seqs);
        if (kv.dtype == FATHOM_BF16)
            launch_split<__nv_bfloat16>(a, grid, stream);
        else
            launch_split<__half>(a, grid, stream);
        note_launch();
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || p.direct) return e;
    }
    return launch_merge_parts(a.pv, q, n_heads, kv.head_dim, kv.dtype, a.fixed, prefix_len, a.first,
                              p.chunk, max_len, stream);
}

}  // namespace fathom
