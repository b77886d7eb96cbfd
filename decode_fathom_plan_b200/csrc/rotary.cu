// Norm and rotation of query and key heads, and their way into a paged cache.
//
// A head row x of d channels becomes y = x * w * rsqrt(mean(x^2) + eps), and
// its first rotary_dim channels are rotated in pairs,
//   (a, b) -> m (a cos f - b sin f, b cos f + a sin f),  f = 2 pi pos turns_i.
// fathom_qk_norm_rope does this to query and key rows, fathom_append_kv to the
// key rows while it writes them, and the value rows beside them, into pages.
//
// The angle: pos * turns_i is a number of turns, of which only the fraction
// counts; a float32 product would leave it too few bits (at position 2^20 an
// eighth of a turn in float32 is good to 0.06 turns).  As pos is whole, the
// fraction is the low 64 bits of pos * T_i with T_i the fraction of turns_i in
// units of 2^-64: one 64-bit integer product, exact but for T's own rounding
// (2^-34 turns at position 2^31).  Its top bits are the quadrant and an angle
// of at most an eighth of a turn either way, whose sine and cosine are Taylor
// polynomials to the 9th and 8th power (within 2^-25).  A token's angles serve
// all its heads: a CTA computes those of its tokens once into shared memory.
//
// What bounds it: memory (6 flops an element against 4 bytes or more).  Eight
// elements of each half of a pair are one 16-byte load, a head row is held by
// d/16 neighbouring lanes between its load and its store, and its norm is a
// few shuffles among them, so every element moves once in and once out.  The
// next rows load while the current ones are worked on; 16 warps of 64
// registers a multiprocessor in CTAs of 128 threads keep enough in flight
// (CTAs of 256 threads: 4 to 10% slower; a register more per thread and a
// quarter fewer warps: 8% slower).  A CTA's rows are all queries, all keys or
// all values, so that what describes them is uniform (mixed: 20% slower).
// Measured on B200, a call among others, on several GPUs: a 32768-token prompt
// of 32 + 8 heads of 128, bf16 to bf16 and float32, 134 to 142 us (80 to 85% of
// a plain copy), float32 throughout 207 us; its keys and values into pages of
// 32, 52 us (80%); one token 3.4 us.  An element at a time (rows off their 16
// bytes, rotated widths that are no multiple of 16) the prompt takes 420 us.
#include <algorithm>

#include "paged.cuh"

namespace fathom {
namespace {

constexpr int kRowThreads = 128;
constexpr int kMaxPairs = kMaxHeadDim / 2;
constexpr int kMaxTile = 32;                      // tokens of a CTA
constexpr int kTilePairs = 1024;                  // and their pairs (8 KB of shared memory)

// VEC elements as they are loaded, widened only when they are used.
template <int VEC, typename T>
struct Chunk {                                    // one element
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void widen(float (&x)[VEC]) const { x[0] = static_cast<float>(v); }
};
template <typename T>
struct Chunk<8, T> {                              // 16 bytes of eight 16-bit elements
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    __device__ __forceinline__ void widen(float (&x)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen2<T>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Chunk<8, float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const
    {
        *reinterpret_cast<float4 *>(p) = a;
        *reinterpret_cast<float4 *>(p + 4) = b;
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

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

// Rotates pairs of channels (x[j], y[j]), or two of them at once.
__device__ __forceinline__ void rotate(float &x, float &y, float c, float s)
{
    const float rx = x * c - y * s;
    y = y * c + x * s;
    x = rx;
}
__device__ __forceinline__ void rotate(float *x, float *y, const float *c, const float *s)
{
    const Pair xx(x[0], x[1]), yy(y[0], y[1]), cc(c[0], c[1]), ss(s[0], s[1]);
    (xx * cc - yy * ss).split(x[0], x[1]);
    fma2(xx, ss, yy * cc).split(y[0], y[1]);
}
// x * w * f element by element.
template <int VEC>
__device__ __forceinline__ void scale(float (&x)[VEC], const float (&w)[VEC], float f)
{
    if constexpr (VEC == 1) {
        x[0] *= w[0] * f;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) (Pair(x[j], x[j + 1]) * Pair(w[j], w[j + 1]) * Pair(f, f)).split(x[j], x[j + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ float sum_squares(const float (&x)[VEC], const float (&y)[VEC])
{
    if constexpr (VEC == 1) {
        return fmaf(x[0], x[0], y[0] * y[0]);
    } else {
        Pair s(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const Pair a(x[j], x[j + 1]), b(y[j], y[j + 1]);
            s = fma2(a, a, fma2(b, b, s));
        }
        float u, v;
        s.split(u, v);
        return u + v;
    }
}

// Cosine (which 0) or sine (1) of pair u*VEC + j in a token's part of the
// table: four of a unit are one 16-byte word, the units' words side by side.
template <int VEC>
__device__ __forceinline__ int angle_slot(int which, int u, int j, int units)
{
    return VEC == 8 ? ((which * 2 + (j >> 2)) * units + u) * 4 + (j & 3) : which * units + u;
}
// The four of a 16-byte word, or one.
template <int VEC>
__device__ __forceinline__ void angles(const float *from, float *to)
{
    if constexpr (VEC == 8) {
        const float4 v = *reinterpret_cast<const float4 *>(from);
        to[0] = v.x; to[1] = v.y; to[2] = v.z; to[3] = v.w;
    } else {
        to[0] = from[0];
    }
}
// Fraction of a turn in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_fraction(double turns)
{
    return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}
// (cos, sin) of a phase in units of 2^-64 turns.
__device__ __forceinline__ float2 cos_sin(unsigned long long phase)
{
    const int hi = (int)(phase >> 32);
    const int quadrant = (int)((unsigned)hi + 0x20000000u) >> 30;       // nearest quarter turn
    const int rest = (int)((unsigned)hi - ((unsigned)quadrant << 30));  // in +-2^29 of 2^-32 turns
    const float x = (float)rest * (6.2831853071795865f / 4294967296.0f), y = x * x;
    const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f),
                                     -1.0f / 6.0f), x);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 40320.0f, -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
    const float a = quadrant & 1 ? s : c, b = quadrant & 1 ? c : s;
    return make_float2((quadrant + 1) & 2 ? -a : a, quadrant & 2 ? -b : b);
}

// What a lane holds of a row: kIter units of VEC elements of each half.
template <int VEC, typename T>
struct Piece {
    static constexpr int kIter = VEC == 8 ? 1 : kMaxPairs / 32;
    Chunk<VEC, T> lo[kIter], hi[kIter];
};

// VEC elements of each half of a pair run per lane and step: 8 where all rows
// allow 16-byte accesses and rotary_dim is a multiple of 16, else 1.  A unit
// is 2*VEC channels of a row: with pairs apart the VEC at u*VEC and those half
// the rotated channels further, else 2*VEC neighbours.
template <int VEC, typename T>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 4 ? 5 : 8)
rows_kernel(const RowsArgs a)
{
    using P = Piece<VEC, T>;
    __shared__ alignas(16) float s_cs[2 * kTilePairs];
    __shared__ long long s_dst[kMaxTile];
    // a CTA's rows are of one kind, so all that describes them is uniform
    const bool second = blockIdx.x >= a.blocks0;
    const RowSet r = second ? a.set[1] : a.set[0];
    const int block = blockIdx.x - (second ? a.blocks0 : 0);
    const int t0 = block / r.chunks * r.tile, h0 = block % r.chunks * r.heads_per_cta;
    const int tile = min(r.tile, a.n_tokens - t0), heads = min(r.heads_per_cta, r.heads - h0);
    const int half = r.turn ? a.rotary_dim >> 1 : 0;
    const int units = a.head_dim / (2 * VEC), rot_units = half / VEC;
    const int lane = threadIdx.x & (a.lanes - 1), grp = threadIdx.x / a.lanes;
    const int groups = kRowThreads / a.lanes;
    const int step_t = groups / heads, step_h = groups - step_t * heads;
    wait_for_earlier_kernels();
    let_next_kernel_start();

    // offsets of the lane's units in a row
    int at[P::kIter], at2[P::kIter];
#pragma unroll
    for (int i = 0; i < P::kIter; ++i) {
        const int u = lane + 32 * i;
        const bool apart = u < rot_units && !a.interleaved;
        at[i] = apart ? u * VEC : u * 2 * VEC;
        at2[i] = apart ? at[i] + half : at[i] + VEC;
    }
    const auto load = [&](const T *in, P &p) {
#pragma unroll
        for (int i = 0; i < P::kIter; ++i)
            if (lane + 32 * i < units) {
                p.lo[i].load(in + at[i]);
                p.hi[i].load(in + at2[i]);
            }
    };
    const auto row = [&](int t, int h) {
        return static_cast<const T *>(r.in) + (long long)(t0 + t) * r.in_ts + (h0 + h) * r.in_hs;
    };

    // the first rows are on their way while the angles and places are worked out
    P next;
    int t = grp / heads, h = grp - t * heads;
    if (t < tile) load(row(t, h), next);
    const int last = kRowThreads - 1 - threadIdx.x;      // the last warp looks up the places
    if (a.paged && last < tile) {
        const int b = a.seq[t0 + last], p = a.pos[t0 + last];
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
        s_dst[last] = dst;
    }
    P w;
    if (r.weight) load(static_cast<const T *>(r.weight), w);
    if (half) {
        const int per = kRowThreads / half;              // tokens at a time
        const int x0 = threadIdx.x / half, p = threadIdx.x - x0 * half;
        const unsigned long long turn = turn_fraction(a.turns[p]);
        float *const c = s_cs + angle_slot<VEC>(0, p / VEC, p % VEC, rot_units);
        float *const s = s_cs + angle_slot<VEC>(1, p / VEC, p % VEC, rot_units);
        if (x0 < per)
#pragma unroll 4
            for (int x = x0; x < tile; x += per) {
                const float2 cs = cos_sin((unsigned long long)(long long)a.pos[t0 + x] * turn);
                c[x * 2 * half] = cs.x * a.magnitude;
                s[x * 2 * half] = cs.y * a.magnitude;
            }
    }
    __syncthreads();

    if (r.copy) {                                         // rows that only move
        for (; t < tile;) {
            const P cur = next;
            const long long dst = a.paged ? s_dst[t] : (long long)(t0 + t) * r.out_ts;
            T *out = static_cast<T *>(r.out) + dst + (h0 + h) * r.out_hs;
            t += step_t;
            h += step_h;
            if (h >= heads) {
                h -= heads;
                ++t;
            }
            if (t < tile) load(row(t, h), next);
            if (a.paged && dst < 0) continue;
#pragma unroll
            for (int i = 0; i < P::kIter; ++i)
                if (lane + 32 * i < units) {
                    cur.lo[i].store(out + at[i]);
                    cur.hi[i].store(out + at2[i]);
                }
        }
        return;
    }
    // every lane of a warp makes the same number of steps: the shuffles of a row are warp-wide
    for (int step = (tile * heads + groups - 1) / groups; step > 0; --step) {
        const P cur = next;
        const int cur_t = t, cur_h = h;
        t += step_t;
        h += step_h;
        if (h >= heads) {
            h -= heads;
            ++t;
        }
        if (t < tile) load(row(t, h), next);
        bool live = cur_t < tile;
        long long out = 0;
        if (live) {
            out = a.paged ? s_dst[cur_t] : (long long)(t0 + cur_t) * r.out_ts;
            live = !a.paged || out >= 0;
            out += (h0 + cur_h) * r.out_hs;
        }
        float lo[P::kIter][VEC], hi[P::kIter][VEC];
#pragma unroll
        for (int i = 0; i < P::kIter; ++i) {
            cur.lo[i].widen(lo[i]);
            cur.hi[i].widen(hi[i]);
        }
        if (r.weight) {
            float sq = 0.0f;
#pragma unroll
            for (int i = 0; i < P::kIter; ++i)
                if (lane + 32 * i < units) sq += sum_squares(lo[i], hi[i]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                if (off < a.lanes) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, off);
            const float norm = rsqrtf(sq * a.inv_dim + a.eps);
#pragma unroll
            for (int i = 0; i < P::kIter; ++i) {
                float x[VEC];
                w.lo[i].widen(x);
                scale(lo[i], x, norm);
                w.hi[i].widen(x);
                scale(hi[i], x, norm);
            }
        }
        if (!live) continue;
        const float *cs = s_cs + cur_t * 2 * half;
#pragma unroll
        for (int i = 0; i < P::kIter; ++i) {
            const int u = lane + 32 * i;
            if (u >= units) continue;
            if (u < rot_units) {
                float c[VEC], s[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j += VEC == 8 ? 4 : 1) {
                    angles<VEC>(cs + angle_slot<VEC>(0, u, j, rot_units), c + j);
                    angles<VEC>(cs + angle_slot<VEC>(1, u, j, rot_units), s + j);
                }
                if constexpr (VEC == 1) {
                    rotate(lo[i][0], hi[i][0], c[0], s[0]);
                } else if (!a.interleaved) {
#pragma unroll
                    for (int j = 0; j < VEC; j += 2) rotate(lo[i] + j, hi[i] + j, c + j, s + j);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        rotate(lo[i][2 * j], lo[i][2 * j + 1], c[j], s[j]);
                        rotate(hi[i][2 * j], hi[i][2 * j + 1], c[VEC / 2 + j], s[VEC / 2 + j]);
                    }
                }
            }
            store_chunk(r.out, out + at[i], r.out_dtype, lo[i]);
            store_chunk(r.out, out + at2[i], r.out_dtype, hi[i]);
        }
    }
}

template <int VEC>
cudaError_t launch_rows_vec(const RowsArgs &a, int dtype, int blocks, cudaStream_t stream)
{
    if (dtype == FATHOM_F32)
        return launch_overlapped(rows_kernel<VEC, float>, dim3(blocks), kRowThreads, 0, stream, a);
    if (dtype == FATHOM_BF16)
        return launch_overlapped(rows_kernel<VEC, __nv_bfloat16>, dim3(blocks), kRowThreads, 0, stream, a);
    return launch_overlapped(rows_kernel<VEC, __half>, dim3(blocks), kRowThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_rows(RowsArgs a, int dtype, bool vector, cudaStream_t stream)
{
    a.status = device_status_ptr();
    a.inv_dim = 1.0f / a.head_dim;
    const int units = a.head_dim / (vector ? 16 : 2);
    a.lanes = 1;
    while (a.lanes < units && a.lanes < 32) a.lanes *= 2;
    const int groups = kRowThreads / a.lanes;
    // A CTA takes one step of rows where there are few, and up to kSteps of them, so that all but
    // the first load while others are worked on and many rows share the angles.
    constexpr int kFill = 148 * 4, kSteps = 8;
    long long blocks[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        RowSet &r = a.set[i];
        if (!r.heads) continue;
        r.turn = r.turn && a.rotary_dim;
        r.copy = !r.turn && !r.weight && r.out_dtype == dtype;
        const long long even = (long long)a.n_tokens * r.heads / kFill;
        const int rows = (int)std::min<long long>(std::max<long long>(even, groups), kSteps * groups);
        r.heads_per_cta = std::min(r.heads, rows);
        r.tile = std::min({rows / r.heads_per_cta, kMaxTile,
                           r.turn ? kTilePairs / (a.rotary_dim / 2) : kMaxTile});
        r.chunks = (r.heads + r.heads_per_cta - 1) / r.heads_per_cta;
        blocks[i] = ((long long)a.n_tokens + r.tile - 1) / r.tile * r.chunks;
    }
    if (blocks[0] + blocks[1] > INT32_MAX) return cudaErrorInvalidValue;
    a.blocks0 = (int)blocks[0];
    note_launch();
    return vector ? launch_rows_vec<8>(a, dtype, (int)(blocks[0] + blocks[1]), stream)
                  : launch_rows_vec<1>(a, dtype, (int)(blocks[0] + blocks[1]), stream);
}

}  // namespace fathom
