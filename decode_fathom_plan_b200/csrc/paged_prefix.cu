// Attention of all queries of a batch over the prefix that its sequences share.
//
// The rows of KV head h are the G query heads of every sequence: R = n_seqs*G
// rows over the same keys, 4*R*d flops for 4*d bytes.  From some 250 rows on
// the tensor cores bound it, below that memory, so the products run on the
// 5th-generation tensor cores (tcgen05, accumulators in TMEM):
//   S [128 rows x 128 keys] = Q K^T   both operands K-major in shared memory,
//   O [128 rows x d]       += P V     P from TMEM, V as it is stored (N-major).
// A CTA per SM takes one KV head, up to 256 rows and a run of key tiles:
//   warp 0      copies K and V tiles by TMA, one box per page, through a ring
//               of stages; a page past the prefix, or a bad one, becomes an
//               out-of-range coordinate, which TMA fills with zeros;
//   warp 1      issues the products;
//   warp 2      allocates TMEM;
//   warps 4-7   softmax of slot 0, thread = row: S from TMEM, running maximum
//   warps 8-11  and sum in registers, P back to TMEM over S; slot 1 likewise.
// Two slots keep the tensor cores busy while a slot's softmax runs.  With more
// than 128 rows the slots are two row blocks over the same tiles; with fewer
// they are the even and the odd tiles of the same rows.  Head dims over 128
// leave TMEM for one slot.
// O is rescaled (in TMEM, by the softmax warps) only when a row's maximum grew
// by more than 2^8.  The parts of all runs are joined with the sequences' own
// keys by merge_parts_kernel.
//
// Every wait has a time limit; where one runs out the CTA records
// FATHOM_ERR_TIMEOUT, waits for its copies and products and leaves.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "paged.cuh"

namespace fathom {
namespace {

constexpr int kRows = 128;                       // rows of a slot
constexpr int kTile = 128;                       // keys of a tile
constexpr int kBlockBytes = kTile * 128;         // 128 rows of 64 channels (128 bytes, swizzled)
constexpr unsigned long long kWaitNs = 500000000ull;
constexpr int kTmemCols = 512;

template <int NB>
struct PrefixShape {                             // NB = 64-channel blocks of a row
    static constexpr int kSlots = NB <= 2 ? 2 : 1;
    static constexpr int kStages = NB == 1 ? 8 : NB == 2 ? 5 : NB == 3 ? 3 : 2;
    static constexpr int kTileBytes = NB * kBlockBytes;
    static constexpr int kThreads = 128 + 128 * kSlots;
    static constexpr int kSmem = (kSlots + kStages) * kTileBytes + 1024;
};

struct PrefixArgs {
    PagedQuery q;
    PartsView pv;
    ScoreArgs score;
    const int32_t *table;                        // the first row of the page table
    int n_heads, n_pages, page_shift, head_dim;
    int prefix_len, rows, n_tiles, splits, row_groups, two_blocks, parts;
    int *status;
};

// ------------------------------------------------------------- PTX wrappers
__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long global_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits for the phase of the given parity, the whole warp together; false once
// *stop is set or the limit is over (which sets it).  Inlined: the warps that
// issue products and copies make no calls.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *stop)
{
    bool ok = mbar_try(bar, parity);
    if (!ok) {
        const unsigned long long start = global_ns();
        do {
            ok = mbar_try(bar, parity);
            if (!ok && (*stop || global_ns() - start > kWaitNs)) {
                *stop = 1;
                break;
            }
        } while (!ok);
    }
    return __all_sync(0xFFFFFFFFu, ok);
}
// The same after a stop, for what is still under way; gives up after the limit.
__device__ __forceinline__ void wait_anyway(uint32_t bar, uint32_t parity)
{
    const unsigned long long start = global_ns();
    while (!mbar_try(bar, parity) && global_ns() - start < kWaitNs) {
    }
    __syncwarp();
}
// One lane of a warp that is together; the same one every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c,
                                         int slot, int head, int page)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(c), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
// Matrix descriptor of a 128-byte-swizzled tile: lbo between 64-element blocks
// of an N-major operand (unused for K-major), 1024 bytes between groups of
// eight 128-byte rows.
__device__ __forceinline__ uint64_t umma_desc(uint32_t addr, uint32_t lbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *x)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float *x)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float *x)
{
    const uint32_t *r = reinterpret_cast<const uint32_t *>(x);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Whole 32-byte sectors: each lane writes another row.
__device__ __forceinline__ void store8(float *p, const float *x)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]),
                 "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// Walks the steps (iteration, slot) of a CTA in the order in which their
// tiles are consumed; the copying and the issuing warp follow the same walk.
// At each step comes first V of the slot's previous tile, then K of its next.
struct Walk {
    int tiles;        // of this CTA
    int slots;
    bool shared;      // the slots take the same tiles (else tile 2i + s)
    __device__ int iterations() const { return shared ? tiles : (tiles + slots - 1) / slots; }
    __device__ int tile(int i, int s) const { return shared ? i : i * slots + s; }
    __device__ bool has(int i, int s) const { return i >= 0 && tile(i, s) < tiles; }
    __device__ int count(int s) const { return shared ? tiles : (tiles - s + slots - 1) / slots; }
};

// grid: (row group, KV head) fastest, then the run of tiles
template <typename T, int NB>
__global__ void __launch_bounds__(PrefixShape<NB>::kThreads, 1)
paged_prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const PrefixArgs a)
{
    using Shape = PrefixShape<NB>;
    constexpr int kSlots = Shape::kSlots, kStages = Shape::kStages, kTileBytes = Shape::kTileBytes;
    let_next_kernel_start();
    extern __shared__ unsigned char s_raw[];
    __shared__ alignas(8) uint64_t s_bar[2 * kStages + 3 * kSlots + 2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
    const uint32_t q_addr = base, ring = base + kSlots * kTileBytes;
    const uint32_t full = smem_u32(s_bar), empty = full + 8 * kStages, s_ready = empty + 8 * kStages,
                   p_ready = s_ready + 8 * kSlots, o_ready = p_ready + 8 * kSlots,
                   q_ready = o_ready + 8 * kSlots, drained = q_ready + 8;

    const int per = gridDim.x / a.splits;                       // row groups * KV heads
    const int split = blockIdx.x / per, unit = blockIdx.x - split * per;
    const int h = unit / a.row_groups, group = unit - h * a.row_groups;
    const int t0 = (int)((long long)split * a.n_tiles / a.splits);
    const int t1 = (int)((long long)(split + 1) * a.n_tiles / a.splits);
    const bool shared = a.two_blocks || kSlots == 1;
    const Walk walk{t1 - t0, kSlots, shared};
    const int row0 = group * kRows * (shared ? kSlots : 1);     // of slot 0
    const int d = a.head_dim, G = a.q.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *stop = &s_stop;

    if (threadIdx.x == 0) {
        s_stop = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(s_ready + 8 * s, 1);
            mbar_init(p_ready + 8 * s, 4);
            mbar_init(o_ready + 8 * s, 1);
        }
        mbar_init(q_ready, 4 * kSlots);
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // by a warp that does nothing else: after code for one of its lanes a warp need not be together
    // again for an aligned instruction
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&s_tmem)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    const uint32_t o_col = kSlots * kTile;                      // O of slot s at o_col + s*d

    if (warp == 0) {
        // ------------------------------------------------------ copies
        const int shift = a.page_shift, box = min(1 << shift, kTile);
        const int boxes = kTile / box;                          // per 64-channel block
        int issued = 0;
        bool ok = true, bad = false;
        auto load = [&](const CUtensorMap *map, int tile) {
            const int stage = issued % kStages;
            ok = mbar_wait(empty + 8 * stage, ((issued / kStages) & 1) ^ 1, stop);
            if (!ok) return;
            // lane x: the page of box x
            const int key0 = (t0 + tile) * kTile, key = key0 + lane * box;
            int page = a.n_pages;
            if (lane < boxes && key < a.prefix_len) {
                page = a.table[key >> shift];
                if (page < 0 || page >= a.n_pages) {
                    bad = true;
                    page = a.n_pages;
                }
            }
            const uint32_t dst = ring + stage * kTileBytes, bar = full + 8 * stage;
            const int slot0 = key0 & ((1 << shift) - 1);        // not 0 where a page holds several tiles
            __syncwarp();
            if (elect_one()) mbar_expect(bar, kTileBytes);
            __syncwarp();
            for (int x = 0; x < boxes; ++x) {
                const int p = __shfl_sync(0xFFFFFFFFu, page, x);
                if (elect_one()) {
#pragma unroll
                    for (int cb = 0; cb < NB; ++cb)
                        tma_load(dst + cb * kBlockBytes + x * box * 128, map, bar, cb * 64, slot0, h, p);
                }
                __syncwarp();
            }
            ++issued;
        };
        const int n = walk.iterations();
        for (int i = 0; i <= n && ok; ++i)
            for (int s = 0; s < kSlots && ok; ++s) {
                if (shared && s > 0) continue;
                if (walk.has(i - 1, s)) load(&vmap, walk.tile(i - 1, s));
                if (i < n && walk.has(i, s)) load(&kmap, walk.tile(i, s));
            }
        if (bad) set_status(a.status, FATHOM_ERR_INVALID_ARG);
        if (!ok)                                                // let the copies land
            for (int x = max(0, issued - kStages); x < issued; ++x)
                wait_anyway(full + 8 * (x % kStages), (x / kStages) & 1);
    } else if (warp == 1) {
        // ---------------------------------------------------- products
        const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        const uint32_t common = (1u << 4) | (type << 7) | (type << 10) | ((128u >> 4) << 24);
        const uint32_t idesc_qk = common | ((uint32_t)(kTile >> 3) << 17);
        const uint32_t idesc_pv = common | (1u << 16) | ((uint32_t)(d >> 3) << 17);
        int used = 0, k_use = 0, v_use = 0;
        bool ok = mbar_wait(q_ready, 0, stop);
        const int n = walk.iterations();
        for (int i = 0; i <= n && ok; ++i)
            for (int s = 0; s < kSlots && ok; ++s) {
                const bool take = !shared || s == 0, last = !shared || s == kSlots - 1;
                if (walk.has(i - 1, s)) {
                    if (take) {
                        v_use = used++;
                        ok = mbar_wait(full + 8 * (v_use % kStages), (v_use / kStages) & 1, stop);
                    }
                    ok = ok && mbar_wait(p_ready + 8 * s, (i - 1) & 1, stop);
                    if (!ok) break;
                    tc_after();
                    const uint64_t v = umma_desc(ring + v_use % kStages * kTileBytes, kBlockBytes);
                    const bool ends = !walk.has(i, s);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)    // 16 keys: 2048 bytes of V, 8 columns of P
                            umma_ts(tmem + o_col + s * d, tmem + s * kTile + k * 8, v + k * (2048 >> 4), idesc_pv,
                                    i > 1 || k > 0);
                        if (last) umma_commit(empty + 8 * (v_use % kStages));
                        if (ends) umma_commit(o_ready + 8 * s);
                    }
                    __syncwarp();
                }
                if (i < n && walk.has(i, s)) {
                    if (take) {
                        k_use = used++;
                        ok = mbar_wait(full + 8 * (k_use % kStages), (k_use / kStages) & 1, stop);
                        if (!ok) break;
                        tc_after();
                    }
                    const uint64_t k_desc = umma_desc(ring + k_use % kStages * kTileBytes, 16);
                    const uint64_t q_desc = umma_desc(q_addr + (shared ? s * kTileBytes : 0), 16);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < NB * 4; ++k) {      // 16 channels: 32 bytes of a 64-channel block
                            const int off = ((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4;
                            if (k < d / 16) umma_ss(tmem + s * kTile, q_desc + off, k_desc + off, idesc_qk, k > 0);
                        }
                        if (last) umma_commit(empty + 8 * (k_use % kStages));
                        umma_commit(s_ready + 8 * s);
                    }
                    __syncwarp();
                }
            }
        if (!ok) {                                              // let the products end
            if (elect_one()) umma_commit(drained);
            __syncwarp();
            wait_anyway(drained, 0);
        }
    } else if (warp >= 4) {
        // ----------------------------------------------------- softmax
        const int s = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
        const int row = row0 + (shared ? s * kRows : 0) + r;
        const bool live = row - lane < a.rows;                  // of the warp: any row at all
        const int b = min(row, a.rows - 1) / G, head = h * G + min(row, a.rows - 1) - b * G;
        {
            // the warp's 32 rows of Q into their swizzled tile; slots with the same rows take turns
            const long long mine = b * a.q.q_ts + head * a.q.q_hs;
            const uint16_t *q = static_cast<const uint16_t *>(a.q.q);
            const uint32_t to = q_addr + (shared ? s * kTileBytes : 0);
            constexpr int kChunks = NB * 8, kBatch = 8;
            const int first = shared ? 0 : s, step = shared ? 1 : kSlots;
            for (int i0 = first; i0 < kChunks; i0 += kBatch * step) {
                uint4 u[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * step, x = (i * 32 + lane) / kChunks, c = (i * 32 + lane) - x * kChunks;
                    const long long off = __shfl_sync(0xFFFFFFFFu, mine, x & 31);
                    u[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (i < kChunks && c * 8 < d && live) u[k] = *reinterpret_cast<const uint4 *>(q + off + 8 * c);
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * step, x = (i * 32 + lane) / kChunks, c = (i * 32 + lane) - x * kChunks;
                    const int at = (warp & 3) * 32 + x;
                    if (i < kChunks)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         to + (c >> 3) * kBlockBytes + at * 128 + (((c & 7) ^ (at & 7)) << 4)),
                                     "r"(u[k].x), "r"(u[k].y), "r"(u[k].z), "r"(u[k].w)
                                     : "memory");
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);
        }
        const int seq_len = a.q.seq_lens[b];
        const float slope = a.q.slopes ? a.q.slopes[head] * kLog2e : 0.0f;
        const bool plain = a.score.cap == 0.0f && !a.q.slopes && a.score.scale > 0.0f;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + s * kTile, o_addr = lane_addr + o_col + s * d;
        const int count = walk.count(s);
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            ok = mbar_wait(s_ready + 8 * s, i & 1, stop);
            if (!ok) break;
            tc_after();
            if (live) {
                // Twice over the row, 32 columns at a time and the next ones on their way: the
                // maximum, then the probabilities.  (A row held in registers would be 128 of them.)
                const int key0 = (t0 + walk.tile(i, s)) * kTile;
                const int valid = a.prefix_len - key0;          // keys of this tile
                const bool as_is = plain && valid >= kTile;
                const float mult = as_is ? a.score.scale : 1.0f;
                const float dist = (float)(seq_len - 1 - key0);
                __syncwarp();
                float x[2][32];
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (as_is) {
                    tmem_ld32(s_addr, x[0]);
#pragma unroll
                    for (int c = 0; c < kTile; c += 32) {
                        const float *const y = x[(c >> 5) & 1];
                        tc_wait_ld();
                        if (c + 32 < kTile) tmem_ld32(s_addr + c + 32, x[((c >> 5) & 1) ^ 1]);
#pragma unroll
                        for (int j = 0; j < 32; ++j) tops[j & 3] = fmaxf(tops[j & 3], y[j]);
                    }
                } else {
                    // no load is under way across the branches of a score
#pragma unroll 1
                    for (int c = 0; c < kTile; c += 32) {
                        float *const y = x[0];
                        tmem_ld32(s_addr + c, y);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            y[j] = score_logit(y[j], a.score) - slope * (dist - (float)(c + j));
                            if (c + j >= valid) y[j] = -INFINITY;
                            tops[j & 3] = fmaxf(tops[j & 3], y[j]);
                        }
                        tmem_st32(s_addr + c, y);
                    }
                    tc_wait_st();
                }
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * mult;
                if (__any_sync(0xFFFFFFFFu, top > m + kRescale)) {
                    const float next = fmaxf(m, top);
                    const float w = m == next ? 1.0f : exp2_fast(m - next);
                    m = next;
                    l *= w;
                    if (i > 0) {
                        // the products over earlier tiles are done: S of this tile came after them
#pragma unroll 1
                        for (int c = 0; c < d; c += 16) {
                            float o[16];
                            tmem_ld16(o_addr + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= w;
                            tmem_st16(o_addr + c, reinterpret_cast<const uint32_t *>(o));
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                const Pair mult2(mult, mult), ref2(-ref, -ref);
                Pair sum[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] = Pair(0.0f, 0.0f);
                tmem_ld32(s_addr, x[0]);
#pragma unroll
                for (int c = 0; c < kTile; c += 32) {
                    const float *const y = x[(c >> 5) & 1];
                    tc_wait_ld();
                    if (c + 32 < kTile) tmem_ld32(s_addr + c + 32, x[((c >> 5) & 1) ^ 1]);
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float p0, p1;
                        fma2(Pair(y[j], y[j + 1]), mult2, ref2).split(p0, p1);
                        p0 = exp2_fast(p0);
                        p1 = exp2_fast(p1);
                        sum[(j >> 1) & 3] = sum[(j >> 1) & 3] + Pair(p0, p1);
                        p[j >> 1] = narrow2<T>(p0, p1);
                    }
                    tmem_st16(s_addr + c / 2, p);           // over columns that are read
                }
                {
                    float s0, s1;
                    ((sum[0] + sum[1]) + (sum[2] + sum[3])).split(s0, s1);
                    l += s0 + s1;
                }
                tc_wait_st();
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready + 8 * s);
        }
        if (ok && count > 0) ok = mbar_wait(o_ready + 8 * s, 0, stop);
        if (ok && live) {
            tc_after();
            const int part = shared ? split : split * kSlots + s;
            const size_t place = (size_t)(b * a.n_heads + head) * a.parts + part;
            if (count > 0) {
                for (int c = 0; c < d; c += 32) {
                    float o[32];
                    __syncwarp();
                    tmem_ld32(o_addr + c, o);
                    tc_wait_ld();
                    if (row < a.rows)
#pragma unroll
                        for (int j = 0; j < 32; j += 8) store8(a.pv.o + place * d + c + j, o + j);
                }
            }
            if (row < a.rows) a.pv.ml[place] = make_float2(m, l);
        }
    }
    tc_before();
    __syncthreads();
    if (threadIdx.x == 0 && s_stop) set_status(a.status, FATHOM_ERR_TIMEOUT);
    if (warp == 2) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult res{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &res) == cudaSuccess &&
            res == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// Boxes of 64 channels by the slots of a page (at most a tile), of one head and page.
bool encode(CUtensorMap *map, const void *base, const PagedView &kv)
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int page = 1 << kv.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, (cuuint64_t)page, (cuuint64_t)kv.n_kv_heads,
                                (cuuint64_t)kv.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)kv.slot_stride * 2, (cuuint64_t)kv.head_stride * 2,
                                   (cuuint64_t)kv.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(page, kTile), 1, 1}, step[4] = {1, 1, 1, 1};
    return fn(map,
              kv.dtype == FATHOM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              4, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int NB>
cudaError_t launch_shape(const CUtensorMap &kmap, const CUtensorMap &vmap, const PrefixArgs &a, int ctas,
                         cudaStream_t stream)
{
    using Shape = PrefixShape<NB>;
    const cudaError_t e = cudaFuncSetAttribute(paged_prefix_kernel<T, NB>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    paged_prefix_kernel<T, NB><<<ctas, Shape::kThreads, Shape::kSmem, stream>>>(kmap, vmap, a);
    note_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const CUtensorMap &kmap, const CUtensorMap &vmap, const PrefixArgs &a, int ctas,
                        cudaStream_t stream)
{
    switch ((a.head_dim + 63) / 64) {
    case 1: return launch_shape<T, 1>(kmap, vmap, a, ctas, stream);
    case 2: return launch_shape<T, 2>(kmap, vmap, a, ctas, stream);
    case 3: return launch_shape<T, 3>(kmap, vmap, a, ctas, stream);
    default: return launch_shape<T, 4>(kmap, vmap, a, ctas, stream);
    }
}

}  // namespace

PrefixPlan plan_prefix(int n_kv_heads, int head_dim, int n_seqs, int group, int prefix_len)
{
    PrefixPlan p{};
    if (prefix_len == 0) return p;
    const int slots = head_dim <= 128 ? 2 : 1;
    p.rows = n_seqs * group;
    p.two_blocks = slots == 2 && p.rows > kRows;
    const int cta_rows = kRows * (p.two_blocks ? 2 : 1);
    p.row_groups = (p.rows + cta_rows - 1) / cta_rows;
    p.n_tiles = (prefix_len + kTile - 1) / kTile;
    const int units = p.row_groups * n_kv_heads;
    p.splits = std::max(1, std::min(148 / units, p.n_tiles));
    p.parts = p.splits * (slots == 2 && !p.two_blocks ? 2 : 1);
    return p;
}

cudaError_t launch_paged_prefix(const PagedView &kv, const PagedQuery &q, const PrefixPlan &p,
                                const PartsView &pv, int prefix_len, cudaStream_t stream)
{
    CUtensorMap kmap, vmap;
    if (!encode(&kmap, kv.k, kv) || !encode(&vmap, kv.v, kv)) return cudaErrorInvalidValue;
    PrefixArgs a{};
    a.q = q;
    a.pv = pv;
    a.score = score_args(q.softmax_scale, q.softcap);
    a.table = kv.table;
    a.n_heads = kv.n_kv_heads * q.group;
    a.n_pages = kv.n_pages;
    a.page_shift = kv.page_shift;
    a.head_dim = kv.head_dim;
    a.prefix_len = prefix_len;
    a.rows = p.rows;
    a.n_tiles = p.n_tiles;
    a.splits = p.splits;
    a.row_groups = p.row_groups;
    a.two_blocks = p.two_blocks;
    a.parts = p.parts;
    a.status = device_status_ptr();
    const int ctas = p.row_groups * kv.n_kv_heads * p.splits;
    return kv.dtype == FATHOM_BF16 ? launch_type<__nv_bfloat16>(kmap, vmap, a, ctas, stream)
                                   : launch_type<__half>(kmap, vmap, a, ctas, stream);
}

}  // namespace fathom
