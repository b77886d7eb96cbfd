// Joining the parts of attention rows whose keys were split over CTAs.
//
// Part p of a row holds a_p = sum_j 2^(s_j - m_p) V_j and l_p = sum_j
// 2^(s_j - m_p); the row is sum_p 2^(m_p - M) a_p / sum_p 2^(m_p - M) l_p with
// M = max m_p.  One CTA per row: d/4 lanes of 16-byte loads by as many part
// groups as fit, summed through shared memory in a fixed order.
#include <math.h>

#include "paged.cuh"

namespace fathom {
namespace {

constexpr int kMergeThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kMergeThreads)
merge_parts_kernel(const PartsView pv, const PagedQuery q, int n_heads, int d, int fixed, int shared,
                   int first, int chunk, int max_len, int *status)
{
    __shared__ float s_m[kMergeThreads / 32];
    __shared__ float4 s_o[kMergeThreads];
    __shared__ float s_l[kMergeThreads];
    const int row = blockIdx.x, b = row / n_heads, head = row - b * n_heads;
    int parts = pv.parts;
    if (chunk) {
        const int n = q.seq_lens[b];
        const bool refused = n < 0 || n > max_len || (n > 0 && n < shared);
        if (refused && threadIdx.x == 0) set_status(status, FATHOM_ERR_INVALID_ARG);
        parts = (n == 0 || refused) ? 0 : fixed + (n - first + chunk - 1) / chunk;
    }
    const float2 *ml = pv.ml + (size_t)row * pv.parts;
    float m = -INFINITY;
    for (int p = threadIdx.x; p < parts; p += kMergeThreads) m = fmaxf(m, ml[p].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
    __syncthreads();
    m = s_m[0];
#pragma unroll
    for (int w = 1; w < kMergeThreads / 32; ++w) m = fmaxf(m, s_m[w]);
    const float ref = m == -INFINITY ? 0.0f : m;

    const int lanes = d / 4, groups = kMergeThreads / lanes;
    const int grp = threadIdx.x / lanes, lane = threadIdx.x - grp * lanes;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    if (grp < groups) {
        const float4 *o = reinterpret_cast<const float4 *>(pv.o + (size_t)row * pv.parts * d);
#pragma unroll 4
        for (int p = grp; p < parts; p += groups) {
            const float2 x = ml[p];
            if (x.x == -INFINITY && x.y == 0.0f) continue;   // no key, and no sum written
            const float4 v = o[(size_t)p * lanes + lane];
            const float w = exp2_fast(x.x - ref);
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
            l += w * x.y;
        }
    }
    s_o[threadIdx.x] = acc;
    s_l[threadIdx.x] = l;
    __syncthreads();
    if (grp != 0) return;
    for (int g = 1; g < groups; ++g) {
        const float4 v = s_o[g * lanes + lane];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        l += s_l[g * lanes + lane];
    }
    // l is 0 only where no key took part (the key that set a part's maximum weighs 1 in it),
    // NaN if a score was
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = static_cast<uint16_t *>(q.out) + b * q.out_ts + head * q.out_hs;
    *reinterpret_cast<uint2 *>(out + lane * 4) =
        l == 0.0f ? make_uint2(0u, 0u)
                  : make_uint2(narrow2<T>(acc.x * inv, acc.y * inv), narrow2<T>(acc.z * inv, acc.w * inv));
}

size_t round16(size_t b) { return (b + 15) & ~(size_t)15; }

}  // namespace

size_t parts_bytes(int rows, int head_dim, int parts)
{
    return round16((size_t)rows * parts * head_dim * sizeof(float)) +
           round16((size_t)rows * parts * sizeof(float2));
}

PartsView parts_carve(void *ws, int rows, int head_dim, int parts)
{
    PartsView pv{};
    pv.o = static_cast<float *>(ws);
    pv.ml = reinterpret_cast<float2 *>(static_cast<unsigned char *>(ws) +
                                       round16((size_t)rows * parts * head_dim * sizeof(float)));
    pv.parts = parts;
    return pv;
}

cudaError_t launch_merge_parts(const PartsView &pv, const PagedQuery &q, int n_heads, int head_dim,
                               int dtype, int fixed, int shared, int first, int chunk,
                               int max_len, cudaStream_t stream)
{
    const int rows = q.n_seqs * n_heads;
    if (dtype == FATHOM_BF16)
        merge_parts_kernel<__nv_bfloat16><<<rows, kMergeThreads, 0, stream>>>(
            pv, q, n_heads, head_dim, fixed, shared, first, chunk, max_len, device_status_ptr());
    else
        merge_parts_kernel<__half><<<rows, kMergeThreads, 0, stream>>>(
            pv, q, n_heads, head_dim, fixed, shared, first, chunk, max_len, device_status_ptr());
    note_launch();
    return cudaGetLastError();
}

}  // namespace fathom
