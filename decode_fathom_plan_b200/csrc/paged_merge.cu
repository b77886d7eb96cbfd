// Joining the parts of attention rows whose keys were split over CTAs.
//
// Part p of a row holds a_p = sum_j 2^(s_j - m_p) V_j and l_p = sum_j
// 2^(s_j - m_p); the row is sum_p 2^(m_p - M) a_p / sum_p 2^(m_p - M) l_p with
// M = max m_p.  One CTA per row: d/4 lanes of 16-byte loads by as many part
// groups as fit, each with a running maximum over several parts at a time, so
// that a row of 32 parts costs one round of loads; the groups are summed
// through shared memory in a fixed order.
// It is launched while the kernels before it run (programmatic dependent
// launch) and waits for them: back to back 2 us a call less.
#include <math.h>

#include "paged.cuh"

namespace fathom {
namespace {

// Few rows: threads for their parts.  Many: small CTAs, which wait beside the kernel before them
// without taking its room (16 sessions 76.4 us a call, with 256 threads 78.3), but 92 places of 460
// rows cost 24.0 us a call with 128 threads and 23.0 with 256.
constexpr int kFewRows = 148 * 4, kFewThreads = 256, kManyThreads = 128;

template <typename T, int kMergeThreads>
__global__ void __launch_bounds__(kMergeThreads)
merge_parts_kernel(const MergeArgs a)
{
    constexpr int kAtOnce = kMergeThreads == kManyThreads ? 8 : 6;
    __shared__ float4 s_o[kMergeThreads];
    __shared__ float s_m[kMergeThreads], s_l[kMergeThreads];
    const int row = blockIdx.x, b = row / a.n_heads, head = row - b * a.n_heads;
    const int d = a.head_dim;
    wait_for_earlier_kernels();
    int own = 0;                       // parts behind the fixed ones
    size_t own_at = 0;                 // place of the first
    bool joined = false;               // the row's own keys are one part
    int fixed = a.fixed;
    if (a.lens_from >= 0) {
        const int h = head / a.q.group, g = head - h * a.q.group;
        const int n = a.q.seq_lens[b];
        const int2 ctas = a.info[(size_t)b * (a.n_heads / a.q.group) + h];   // not written where no keys are
        if (refused_length(n, a.shared, a.max_len)) {
            if (threadIdx.x == 0) set_status(a.status, FATHOM_ERR_INVALID_ARG);
            fixed = 0;
        } else if (n == 0) {
            fixed = 0;
        } else if (n > a.lens_from) {
            if (ctas.x == ctas.y) {
                if (!a.fixed) return;  // written by the CTA that had it all
                joined = true;
                own = 1;
                own_at = a.full_at + row;
            } else {
                own = ctas.y - ctas.x + 1;
                own_at = a.cta_at + (size_t)ctas.x * 2 * a.q.group + g;
            }
        }
    }
    const int parts = fixed + own;
    // of the CTAs that share a row the first keeps its part in its second
    // place (the row begins there), the others in their first
    const auto place = [&](int p) -> size_t {
        if (p < fixed) return (size_t)row * a.fixed + p;
        if (joined) return own_at;
        p -= fixed;
        return own_at + (size_t)(2 * p + (p == 0 ? 1 : 0)) * a.q.group;
    };

    const int lanes = d / 4, groups = kMergeThreads / lanes;
    const int grp = threadIdx.x / lanes, lane = threadIdx.x - grp * lanes;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = -INFINITY, l = 0.0f;
    if (grp < groups) {
        for (int p0 = grp; p0 < parts; p0 += kAtOnce * groups) {
            float2 x[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int p = p0 + u * groups;
                x[u] = make_float2(-INFINITY, 0.0f);
                if (p < parts) {
                    const size_t at = place(p);
                    x[u] = a.pv.ml[at];
                    v[u] = reinterpret_cast<const float4 *>(a.pv.o)[at * lanes + lane];
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) top = fmaxf(top, x[u].x);
            const float ref = top == -INFINITY ? 0.0f : top;
            float w = exp2_fast(m - ref);
            acc.x *= w;
            acc.y *= w;
            acc.z *= w;
            acc.w *= w;
            l *= w;
            m = top;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                if (x[u].x == -INFINITY && x[u].y == 0.0f) continue;   // no key, and no sum written
                w = exp2_fast(x[u].x - ref);
                acc.x += w * v[u].x;
                acc.y += w * v[u].y;
                acc.z += w * v[u].z;
                acc.w += w * v[u].w;
                l += w * x[u].y;
            }
        }
    }
    s_o[threadIdx.x] = acc;
    s_m[threadIdx.x] = m;
    s_l[threadIdx.x] = l;
    __syncthreads();
    if (grp != 0) return;
    float top = m;
    for (int g = 1; g < groups; ++g) top = fmaxf(top, s_m[g * lanes + lane]);
    const float ref = top == -INFINITY ? 0.0f : top;
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    l = 0.0f;
    for (int g = 0; g < groups; ++g) {
        const float w = exp2_fast(s_m[g * lanes + lane] - ref);
        const float4 v = s_o[g * lanes + lane];
        acc.x += w * v.x;
        acc.y += w * v.y;
        acc.z += w * v.z;
        acc.w += w * v.w;
        l += w * s_l[g * lanes + lane];
    }
    store_row<T>(a.q, b, head, lane * 4, acc, l);
}

}  // namespace

size_t round16(size_t b) { return (b + 15) & ~(size_t)15; }

size_t parts_bytes(size_t places, int head_dim)
{
    return places * head_dim * sizeof(float) + round16(places * sizeof(float2));
}

PartsView parts_carve(void *ws, size_t places, int head_dim)
{
    float *o = static_cast<float *>(ws);
    return PartsView{o, reinterpret_cast<float2 *>(o + places * head_dim)};
}

cudaError_t launch_merge_parts(const MergeArgs &args, int dtype, cudaStream_t stream)
{
    MergeArgs a = args;
    a.status = device_status_ptr();
    note_launch();
    const int rows = a.q.n_seqs * a.n_heads;
    const auto go = [&](auto kernel, int threads) {
        return launch_overlapped(kernel, dim3(rows), threads, 0, stream, a);
    };
    if (dtype == FATHOM_BF16)
        return rows <= kFewRows ? go(merge_parts_kernel<__nv_bfloat16, kFewThreads>, kFewThreads)
                                : go(merge_parts_kernel<__nv_bfloat16, kManyThreads>, kManyThreads);
    return rows <= kFewRows ? go(merge_parts_kernel<__half, kFewThreads>, kFewThreads)
                            : go(merge_parts_kernel<__half, kManyThreads>, kManyThreads);
}

}  // namespace fathom
