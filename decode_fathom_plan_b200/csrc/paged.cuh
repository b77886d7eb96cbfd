// Shared by the kernels of the paged cache: element types, addresses of
// cached rows, and the scores of the attention kernels (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace fathom {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------ element types
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t u);
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t u)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t u)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
// Two floats rounded to nearest even, a in the low half.
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float a, float b);
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// --------------------------------------------------- two floats an instruction
struct Pair {
    unsigned long long v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void split(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Pair operator*(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b)
{
    Pair r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// --------------------------------------------------------------- cached rows
// 32 bytes of a cached row: four lanes bring a whole line of 128 bytes with one instruction, where
// 16 bytes a lane took two.
__device__ __forceinline__ void load32(const void *p, bool there, uint4 &a, uint4 &b)
{
    a = b = make_uint4(0u, 0u, 0u, 0u);
    if (there)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                     : "l"(p));
}
// First of the eight channels that lane t of the four that share a key holds as its m-th group, of
// E: 16 neighbours of every 64, and of a 32 left over 8.
template <int E>
__host__ __device__ __forceinline__ constexpr int group_channel(int m, int t)
{
    return m < (E & ~1) ? 64 * (m >> 1) + 16 * t + 8 * (m & 1) : 32 * (E - 1) + 8 * t;
}
// All of them of one row, from its first channel.
template <int E>
__device__ __forceinline__ void load_groups(const uint16_t *row, int t, bool there, uint4 (&to)[E])
{
#pragma unroll
    for (int m = 0; m + 1 < E; m += 2) load32(row + group_channel<E>(m, t), there, to[m], to[m + 1]);
    if constexpr (E & 1)
        to[E - 1] = there ? __ldg(reinterpret_cast<const uint4 *>(row + group_channel<E>(E - 1, t)))
                          : make_uint4(0u, 0u, 0u, 0u);
}

// -------------------------------------------------------------------- scores
// 2^x, within 2^-22 of the value; 2^-inf = 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A dot product as a logit times log2(e), so that the softmax is a power of
// two.  The cap is cap * tanh(x / cap) with tanh(y) = 1 - 2 / (1 + e^2y), off by
// at most 2^-20 of the cap, an absolute error of a logit: in units of 2^-23 the
// power's 2^-22 counts 1 (the quotient q <= 2 moves by q (1 - q/2) <= 1/2 of
// it), four roundings of its argument 0.9, that of 1 + e^2y 1, the quotient's
// two last places 2, the product and the constant's rounding 1: 5.9 in all
// (worst measured over 2^24 scores 2.5, 2^-21.6 of the cap).  The hardware's own
// tanh is 2^-11 off, 0.02 of a logit at a cap of 50.  Caps larger than
// kMaxSoftcap, at which that bound is 2^-6 of a logit, are refused.
constexpr float kMaxSoftcap = 16384.0f;
struct ScoreArgs {
    float scale;      // softmax_scale * log2(e); with a cap 2 * log2(e) * softmax_scale / cap
    float cap;        // cap * log2(e), or 0 without a cap
};
__device__ __forceinline__ float score_logit(float dot, const ScoreArgs &s)
{
    const float x = dot * s.scale;
    if (s.cap == 0.0f) return x;
    return s.cap * (1.0f - __fdividef(2.0f, 1.0f + exp2_fast(x)));
}

inline ScoreArgs score_args(float softmax_scale, float softcap)
{
    return softcap > 0.0f ? ScoreArgs{2.0f * kLog2e * softmax_scale / softcap, softcap * kLog2e}
                          : ScoreArgs{kLog2e * softmax_scale, 0.0f};
}

// ------------------------------------------------------------------- lengths
__host__ __device__ __forceinline__ bool refused_length(int n, int shared, int max_len)
{
    return n < 0 || n > max_len || (n > 0 && n < shared);
}

// ------------------------------------------------------------------- outputs
// Four channels of an output row: sum over weight, zeros where no key took
// part.  (The key that set a part's maximum weighs at least 2^-8 in it, so the
// weight is 0 only then; it is NaN if a score was.)
template <typename T>
__device__ __forceinline__ void store_row(const PagedQuery &q, int b, int head, int c, float4 sum, float weight)
{
    const float inv = weight == 0.0f ? 0.0f : 1.0f / weight;
    uint16_t *out = static_cast<uint16_t *>(q.out) + b * q.out_ts + head * q.out_hs + c;
    *reinterpret_cast<uint2 *>(out) =
        weight == 0.0f ? make_uint2(0u, 0u)
                       : make_uint2(narrow2<T>(sum.x * inv, sum.y * inv), narrow2<T>(sum.z * inv, sum.w * inv));
}

// ------------------------------------------------- kernels that follow closely
// A kernel launched by launch_overlapped may start once every CTA of the one
// before it in the stream has called let_next_kernel_start() or ended; what it
// reads or overwrites of that kernel it touches after wait_for_earlier_kernels(),
// which waits for it to end.  A kernel lets the next one start after its own
// wait: then all that was in the stream before the kernel has ended.  On that
// rests the one exception, the kernel of the own keys behind a prefix: it takes
// nothing from the kernel of the prefix and runs beside it, without a wait but
// at its end, so that whoever waits for it waits for both.  All that is gained is
// the launch: a microsecond or two from one small kernel to the next.
__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Scores may pass the reference maximum by this many powers of two before
// the sums are rescaled to a new one: 2^8 more in a float32 sum costs no
// accuracy, fits float16, and most tiles then rescale nothing.
constexpr float kRescale = 8.0f;

// The reference that probabilities of type T are relative to for their product
// with V, from the reference maximum m.  A float16 is a multiple of 2^-24, so
// far below 1 a probability has few bits and then none; relative to 2^7 below m
// it is at most 2^15, which float16 holds, and its half step at most 2^-32 of
// the largest weight.  (Relative to m itself, keys 17.2 and 17.4 nats below
// another had 1.4 times and half their weight.)  A bfloat16 has the range of a
// float.  Parts keep this reference beside their sums.
template <typename T>
__device__ __forceinline__ float prob_reference(float m);
template <>
__device__ __forceinline__ float prob_reference<__nv_bfloat16>(float m) { return m; }
template <>
__device__ __forceinline__ float prob_reference<__half>(float m) { return m - 7.0f; }

}  // namespace fathom
