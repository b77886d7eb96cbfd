// Norm and rotation of query and key heads, and their way into a paged cache.
//
// A head row x of d channels becomes y = x * w * rsqrt(mean(x^2) + eps), and
// its first rotary_dim channels are rotated in pairs,
//   (a, b) -> m (a cos f - b sin f, b cos f + a sin f),  f = 2 pi pos turns_i.
// fathom_qk_norm_rope does this to query and key rows, fathom_append_kv to the
// key rows while it writes them, and the value rows beside them, into pages.
//
// The angle: pos * turns_i is a number of turns, whose whole part a float32
// product would leave too few bits for the fraction (at position 2^20 an
// eighth of a turn in float32 is good to 0.06 turns).  It is taken in float64,
// reduced to [-1/2, 1/2] there, and only the fraction goes to sincospi.  A
// token's angles serve all its heads: a CTA computes the (cos, sin) of its
// tokens once into shared memory, one float64 product each.
//
// What bounds it: memory (6 flops an element against 4 bytes or more).  Eight
// elements of each half of a pair are one 16-byte load, a head row is held by
// d/16 neighbouring lanes between its load and its store, and its norm is a
// few shuffles among them, so every element moves once in and once out.
#include <algorithm>

#include "paged.cuh"

namespace fathom {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxTile = 4;                       // tokens of a CTA
constexpr int kMaxPairs = kMaxHeadDim / 2;

template <typename T>
__device__ __forceinline__ void load_chunk(const T *p, float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen2<T>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ void load_chunk(const T *p, float (&x)[1])
{
    x[0] = static_cast<float>(*p);
}

__device__ __forceinline__ void store_chunk(void *base, long long off, int dtype, const float (&x)[8])
{
    if (dtype == FATHOM_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + off);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = dtype == FATHOM_BF16 ? narrow2<__nv_bfloat16>(x[2 * i], x[2 * i + 1])
                                    : narrow2<__half>(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_chunk(void *base, long long off, int dtype, const float (&x)[1])
{
    if (dtype == FATHOM_F32)
        static_cast<float *>(base)[off] = x[0];
    else if (dtype == FATHOM_BF16)
        static_cast<__nv_bfloat16 *>(base)[off] = __float2bfloat16_rn(x[0]);
    else
        static_cast<__half *>(base)[off] = __float2half_rn(x[0]);
}

__device__ __forceinline__ void rotate(float &x, float &y, float2 cs)
{
    const float rx = x * cs.x - y * cs.y;
    y = y * cs.x + x * cs.y;
    x = rx;
}

// Shared-memory place of the (cos, sin) of pair u*VEC + j: lane u's pairs of
// equal j lie side by side, so the lanes of a row read consecutive words.
template <int VEC>
__device__ __forceinline__ int pair_slot(int u, int j, int units)
{
    return VEC == 8 ? ((j >> 1) * units + u) * 2 + (j & 1) : u;
}

// VEC elements of each half of a pair run per lane and step: 8 where all rows
// allow 16-byte accesses and rotary_dim is a multiple of 16, else 1.
// LANES lanes hold a row; UNITS = d / (2*VEC) units of 2*VEC channels.
template <int VEC, typename T>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const RowsArgs a)
{
    constexpr int kIter = VEC == 8 ? 1 : kMaxPairs / 32;
    __shared__ alignas(16) float2 s_cs[kMaxTile][kMaxPairs];
    __shared__ long long s_dst[kMaxTile];
    const int t0 = blockIdx.x * a.tile, tile = min(a.tile, a.n_tokens - t0);
    const int half = a.rotary_dim >> 1;
    const int units = a.head_dim / (2 * VEC), rot_units = a.rotary_dim / (2 * VEC);

    for (int i = threadIdx.x; i < tile * half; i += kRowThreads) {
        const int t = i / half, p = i - t * half;
        double turn = (double)a.pos[t0 + t] * a.turns[p];
        turn -= rint(turn);
        float s, c;
        sincospif((float)(2.0 * turn), &s, &c);
        s_cs[t][pair_slot<VEC>(p / VEC, p % VEC, rot_units)] = make_float2(c * a.magnitude, s * a.magnitude);
    }
    if (a.paged && (int)threadIdx.x < tile) {
        const int t = t0 + threadIdx.x;
        const int b = a.seq[t], p = a.pos[t];
        long long dst = -1;
        if (b >= 0) {
            int page = -1;
            if (b < a.n_seqs && p >= 0 && (p >> a.page_shift) < a.table_stride)
                page = a.table[(size_t)b * a.table_stride + (p >> a.page_shift)];
            if (page >= 0 && page < a.n_pages)
                dst = page * a.page_stride + (p & ((1 << a.page_shift) - 1)) * a.slot_stride;
            else
                set_status(a.status, FATHOM_ERR_INVALID_ARG);
        }
        s_dst[threadIdx.x] = dst;
    }
    __syncthreads();

    const int lane = threadIdx.x & (a.lanes - 1), grp = threadIdx.x / a.lanes;
    const int groups = kRowThreads / a.lanes;
    const int h0 = blockIdx.y * a.heads_per_cta;
    const int heads = min(a.heads_per_cta, a.set[0].heads + a.set[1].heads - h0);
    // every lane of a warp makes the same number of steps: the shuffles of a row are warp-wide
    const int steps = (tile * heads + groups - 1) / groups;
    for (int step = 0; step < steps; ++step) {
        const int item = step * groups + grp;
        bool live = item < tile * heads;
        const int t = live ? item / heads : 0;
        int h = live ? h0 + item - t * heads : 0;
        const bool second = h >= a.set[0].heads;
        const RowSet &r = a.set[second ? 1 : 0];
        if (second) h -= a.set[0].heads;
        if (a.paged && s_dst[t] < 0) live = false;
        const T *in = static_cast<const T *>(r.in) + (long long)(t0 + t) * r.in_ts + h * r.in_hs;
        const long long out = (a.paged ? s_dst[t] : (long long)(t0 + t) * r.out_ts) + h * r.out_hs;
        float lo[kIter][VEC], hi[kIter][VEC];
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int u = lane + 32 * i;
            if (!live || u >= units) continue;
            const bool apart = u < rot_units && !a.interleaved;
            const int at = apart ? u * VEC : u * 2 * VEC;
            load_chunk(in + at, lo[i]);
            load_chunk(in + (apart ? at + half : at + VEC), hi[i]);
            if (r.weight)
#pragma unroll
                for (int j = 0; j < VEC; ++j) sq = fmaf(lo[i][j], lo[i][j], fmaf(hi[i][j], hi[i][j], sq));
        }
        for (int off = a.lanes >> 1; off > 0; off >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, off);
        if (!live) continue;
        const float norm = rsqrtf(sq / a.head_dim + a.eps);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int u = lane + 32 * i;
            if (u >= units) continue;
            const bool apart = u < rot_units && !a.interleaved;
            const int at = apart ? u * VEC : u * 2 * VEC, at2 = apart ? at + half : at + VEC;
            if (r.weight) {
                float w[VEC];
                load_chunk(static_cast<const T *>(r.weight) + at, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) lo[i][j] *= norm * w[j];
                load_chunk(static_cast<const T *>(r.weight) + at2, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) hi[i][j] *= norm * w[j];
            }
            if (r.turn && u < rot_units) {
                if (apart || VEC == 1) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        rotate(lo[i][j], hi[i][j], s_cs[t][pair_slot<VEC>(u, j, rot_units)]);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j)
                        rotate(lo[i][2 * j], lo[i][2 * j + 1], s_cs[t][pair_slot<VEC>(u, j, rot_units)]);
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j)
                        rotate(hi[i][2 * j], hi[i][2 * j + 1],
                               s_cs[t][pair_slot<VEC>(u, VEC / 2 + j, rot_units)]);
                }
            }
            store_chunk(r.out, out + at, r.out_dtype, lo[i]);
            store_chunk(r.out, out + at2, r.out_dtype, hi[i]);
        }
    }
}

template <int VEC>
void launch_rows_vec(const RowsArgs &a, int dtype, dim3 grid, cudaStream_t stream)
{
    if (dtype == FATHOM_F32)
        rows_kernel<VEC, float><<<grid, kRowThreads, 0, stream>>>(a);
    else if (dtype == FATHOM_BF16)
        rows_kernel<VEC, __nv_bfloat16><<<grid, kRowThreads, 0, stream>>>(a);
    else
        rows_kernel<VEC, __half><<<grid, kRowThreads, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_rows(RowsArgs a, int dtype, bool vector, cudaStream_t stream)
{
    a.status = device_status_ptr();
    const int units = a.head_dim / (vector ? 16 : 2);
    a.lanes = 1;
    while (a.lanes < units && a.lanes < 32) a.lanes *= 2;
    const int groups = kRowThreads / a.lanes, heads = a.set[0].heads + a.set[1].heads;
    // Few tokens: the heads of a token go to several CTAs, one step each.
    a.tile = a.n_tokens >= 1024 ? kMaxTile : 1;
    a.heads_per_cta = a.n_tokens >= 1024 ? heads : std::min(heads, groups);
    const dim3 grid((a.n_tokens + a.tile - 1) / a.tile, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
    if (vector)
        launch_rows_vec<8>(a, dtype, grid, stream);
    else
        launch_rows_vec<1>(a, dtype, grid, stream);
    note_launch();
    return cudaGetLastError();
}

}  // namespace fathom
