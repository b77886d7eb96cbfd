// Attention of all queries of a batch over the prefix that its sequences share.
//
// The rows of KV head h are the G query heads of every sequence: R = n_seqs*G
// rows over the same keys, 4*R*d flops for 4*d bytes.  From some 250 rows on
// the tensor cores bound it, below that memory, so the products run on the
// 5th-generation tensor cores (tcgen05, accumulators in TMEM):
//   S [128 rows x 64 keys] = Q K^T   both operands K-major in shared memory,
//   O [128 rows x d]      += P V     P from TMEM, V as it is stored (N-major).
// A CTA per SM takes one KV head, up to 256 rows and a run of tiles of 128 keys:
//   warps 0, 3  copy Q and K, and V, by TMA, one box per page, through a ring of
//               stages; a page past the prefix, or a bad one, becomes an
//               out-of-range coordinate, which TMA fills with zeros;
//   warps 1, 2  issue the products of a slot each (one warp for both spent
//               as long between the products as on them);
//   warps 4-7   softmax of slot 0, thread = row: S from TMEM, running maximum
//   warps 8-11  and sum in registers, P back to TMEM over S; slot 1 likewise.
// Two slots keep the tensor cores busy while a slot's softmax runs, and S of a
// step is made while the softmax of the step before runs: TMEM has two S of 64
// keys and the sums of 128 channels for each slot, 512 columns in all.  With
// more than 128 rows the slots are two row blocks over the same tiles; with
// fewer they are the even and the odd tiles of the same rows.  Head dims over
// 128 leave TMEM for one slot.
// O is rescaled (in TMEM, by the softmax warps) only when a row's maximum grew
// by more than 2^8.  The parts of all runs are joined with the sequences' own
// keys by merge_parts_kernel.
//
// Measured on B200: 256 rows of 8 KV heads over 32768 keys of 128 channels 45
// to 48 us alone (floor 21 us by either bound), the tensor pipe 42 to 46% busy;
// with 64 sequences' own keys behind them and the joining 133 to 138 us a call.
// A step of both slots takes 1800 cycles; its products alone would take 1280, as
// those of 64 keys read 6 KB of shared memory for 32 cycles of work.  The first
// product with V is issued after 7900 cycles: page table, copies, scores and
// softmax in turn.
//
// Every wait has a time limit.  Where one runs out all warps stop at their next
// one; when they are together again the CTA waits (with a limit) for every copy
// and product that it issued, marks its parts as holding no key, so that
// nothing that was not written is joined, and records FATHOM_ERR_TIMEOUT.  A
// barrier is waited for by the parity of its phase, so whoever waits must have
// seen the phase before: see the barriers of a step, and passing on.
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
constexpr int kStep = 64;                        // keys of a product
constexpr int kBlockBytes = kTile * 128;         // 128 rows of 64 channels (128 bytes, swizzled)
constexpr unsigned long long kSettleNs = 500000000ull;  // for what is under way after a stop
constexpr int kTmemCols = 512;
constexpr int kStageBytes = 4 * 32 * 128;        // 32 channels of a slot's rows in float32

template <int NB>
struct PrefixShape {                             // NB = 64-channel blocks of a row
    static constexpr int kSlots = NB <= 2 ? 2 : 1;
    static constexpr int kStages = NB == 1 ? 8 : NB == 2 ? 5 : NB == 3 ? 3 : 2;
    static constexpr int kTileBytes = NB * kBlockBytes;
    static constexpr int kThreads = 128 + 128 * kSlots;
    // Q of the slots; where they have the same rows, one tile and the stages of both
    static constexpr int kQueryBytes = kSlots == 2 ? (kTileBytes > 2 * kStageBytes ? kTileBytes : 2 * kStageBytes) + kTileBytes
                                                   : kTileBytes;
    static constexpr int kSmem = kQueryBytes + kStages * kTileBytes + 1024;
};

struct PrefixArgs {
    PagedQuery q;
    PartsView pv;
    ScoreArgs score;
    unsigned long long wait_ns;                  // limit of a wait
    const int32_t *table;
    int table_stride, max_len;
    int n_heads, n_pages, page_shift, head_dim;
    int prefix_len, seqs, slot_seqs, split_tiles, split_rest, two_blocks, parts;
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
// Whether the phase of the given parity is over; waits for it a while (the hardware's own limit: one
// given with the instruction cost 0.5% with 64 agents), or not at all.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity, bool linger = true)
{
    uint32_t ok;
    if (!linger)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
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
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *stop, unsigned long long limit)
{
    bool ok = mbar_try(bar, parity, limit > 0);
    if (!ok) {
        const unsigned long long start = global_ns();
        do {
            if (*stop || global_ns() - start >= limit) {
                *stop = 1;
                break;
            }
            ok = mbar_try(bar, parity);
        } while (!ok);
    }
    return __all_sync(0xFFFFFFFFu, ok);
}
// The same after a stop, for what is still under way; gives up after the limit.
__device__ __forceinline__ void wait_anyway(uint32_t bar, uint32_t parity)
{
    const unsigned long long start = global_ns();
    while (!mbar_try(bar, parity) && global_ns() - start < kSettleNs) {
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
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c, int head,
                                          int seq)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(c), "r"(head), "r"(seq), "r"(bar)
        : "memory");
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

// Which tiles the slots of a CTA take, each in two steps of kStep keys.  The
// warps that copy and the one that issues products walk the same order: K of
// every slot's first tile, then at each even step j, slot by slot, V of the
// tile of step j and K of the tile of step j + 2.
struct Walk {
    int tiles;        // of this CTA
    int slots;
    bool shared;      // the slots take the same tiles (else tile slots*i + s)
    __device__ int tile(int i, int s) const { return shared ? i : i * slots + s; }
    __device__ int steps(int s) const { return 2 * (shared ? tiles : (tiles - s + slots - 1) / slots); }
    __device__ int takers() const { return shared ? 1 : slots; }
};
// Place in the ring of stages.
template <int STAGES>
struct Place {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// grid (row groups, KV heads, runs of tiles)
template <typename T, int NB>
__global__ void __launch_bounds__(PrefixShape<NB>::kThreads, 1)
paged_prefix_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const PrefixArgs a)
{
    using Shape = PrefixShape<NB>;
    constexpr int kSlots = Shape::kSlots, kStages = Shape::kStages, kTileBytes = Shape::kTileBytes;
    constexpr int kThreads = Shape::kThreads;
    wait_for_earlier_kernels();
    let_next_kernel_start();
    extern __shared__ unsigned char s_raw[];
    // Of slot s and step j: S, P and the product with V each at 2*s + (j & 1) of their barriers,
    // phase j / 2.  With one barrier for every step a waiter could be two phases off, which a
    // phase's parity does not show.
    constexpr int kFull = 0, kEmpty = kStages, kScores = 2 * kStages, kProbs = kScores + 2 * kSlots,
                  kDone = kProbs + 2 * kSlots, kQueries = kDone + 2 * kSlots, kDrained = kQueries + 1,
                  kBarriers = kDrained + kSlots;
    __shared__ alignas(8) uint64_t s_bar[kBarriers];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    // parity of the last phase of each stage that a copy was issued for, -1 for none
    __shared__ int s_copied[kStages];
    const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
    const uint32_t q_addr = base, ring = base + Shape::kQueryBytes, bars = smem_u32(s_bar);
    const auto bar = [&](int i) { return bars + 8 * i; };

    const int group = blockIdx.x, h = blockIdx.y, split = blockIdx.z;
    const int t0 = split * a.split_tiles + min(split, a.split_rest);
    const int t1 = t0 + a.split_tiles + (split < a.split_rest ? 1 : 0);
    const bool shared = a.two_blocks || kSlots == 1;
    const Walk walk{t1 - t0, kSlots, shared};
    const int seq0 = group * a.slot_seqs * (shared ? kSlots : 1);   // of slot 0
    const int d = a.head_dim, G = a.q.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *stop = &s_stop;
    // sequence of row r of slot s, and the place of its part; -1 where there is none
    const auto sequence_of = [&](int s, int r) {
        const int seq = seq0 + (shared ? s * a.slot_seqs : 0) + r / G;
        return r < a.slot_seqs * G && seq < a.seqs ? seq : -1;
    };
    const auto place_of = [&](int s, int r) {
        const int seq = sequence_of(s, r), part = shared ? split : split * kSlots + s;
        return seq < 0 ? -1ll : ((long long)seq * a.n_heads + h * G + r % G) * a.parts + part;
    };
    const uint32_t o_col = kSlots * kTile;                      // O of slot s at o_col + s*d

    if (warp == 0) {
        // a stage is freed by both slots, whether they read it or not; P comes from four warps
        for (int i = lane; i < kBarriers; i += 32)
            mbar_init(bar(i), i >= kEmpty && i < kScores ? kSlots : i >= kProbs && i < kDone ? 4 : 1);
        if (lane == 0) s_stop = 0;
        if (lane < kStages) s_copied[lane] = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------ copies: K (and Q) or V
        const bool keys = warp == 0;
        const CUtensorMap *map = keys ? &kmap : &vmap;
        const int shift = a.page_shift, box = min(1 << shift, kTile);
        const int boxes = kTile / box;                          // per 64-channel block
        // lane x: the page of box x of a tile, looked up a tile ahead, in the row of the first
        // sequence that takes part: the row of an empty one (a padded batch row) may hold anything
        const int32_t *table = a.table;
        const auto page_of = [&](int tile) {
            const int key = (t0 + tile) * kTile + lane * box;
            return lane < boxes && key < a.prefix_len ? table[key >> shift] : a.n_pages;
        };
        const auto length_of = [&](int s) { return s < a.seqs ? a.q.seq_lens[s] : 0; };
        int page = page_of(0), len = length_of(lane);           // mostly it is the first row
        __syncwarp();
        if (elect_one()) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
            if (keys) asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
        }
        __syncwarp();
        if (keys) {
            // the others wait for this, and for TMEM; the first copies of Q and K do not
            asm volatile("barrier.cta.arrive 1, %0;" ::"n"(kThreads) : "memory");
            const int slots = shared ? kSlots : 1, box_bytes = a.slot_seqs * G * 128;
            if (elect_one()) {
                mbar_expect(bar(kQueries), slots * NB * box_bytes);
                for (int s = 0; s < slots; ++s)
#pragma unroll
                    for (int cb = 0; cb < NB; ++cb)
                        tma_load3(q_addr + s * kTileBytes + cb * kBlockBytes, &qmap, bar(kQueries), cb * 64, h * G,
                                  seq0 + s * a.slot_seqs);
            }
            __syncwarp();
        } else {
            asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory");
        }
        // which row it is, once the first copies that need none are on their way
        int from = -1;
        for (int s = 0; s < a.seqs && from < 0; s += 32) {
            if (s > 0) len = length_of(s + lane);
            const unsigned in = __ballot_sync(0xFFFFFFFFu, len > 0 && !refused_length(len, a.prefix_len, a.max_len));
            if (in) from = s + __ffs(in) - 1;
        }
        const int keys_end = from < 0 ? 0 : a.prefix_len;       // with no sequence, no page is used
        if (from > 0) {
            table += (size_t)from * a.table_stride;
            page = page_of(0);
        }
        Place<kStages> at;
        bool ok = true, bad = false;
        const auto load = [&](bool mine, int tile) {
            if (ok && mine) ok = mbar_wait(bar(kEmpty + at.stage), at.phase ^ 1, stop, a.wait_ns);
            if (ok && mine) {
                int p = page;
                if (lane >= boxes || (t0 + tile) * kTile + lane * box >= keys_end) {
                    p = a.n_pages;
                } else if (p < 0 || p >= a.n_pages) {
                    bad = true;
                    p = a.n_pages;
                }
                page = page_of(tile + 1);
                const uint32_t dst = ring + at.stage * kTileBytes, full = bar(kFull + at.stage);
                const int slot0 = ((t0 + tile) * kTile) & ((1 << shift) - 1);   // a page may hold several tiles
                if (elect_one()) {
                    s_copied[at.stage] = (int)at.phase;
                    mbar_expect(full, kTileBytes);
                }
                __syncwarp();
#pragma unroll 1
                for (int x = 0; x < boxes; ++x) {
                    const int px = __shfl_sync(0xFFFFFFFFu, p, x);
                    if (elect_one())
#pragma unroll
                        for (int cb = 0; cb < NB; ++cb)
                            tma_load(dst + cb * kBlockBytes + x * box * 128, map, full, cb * 64, slot0, h, px);
                }
                __syncwarp();
            }
            at.next();
        };
        const int takers = walk.takers(), n = walk.steps(0);
        for (int s = 0; s < takers; ++s)
            if (walk.steps(s) > 0) load(keys, walk.tile(0, s));
        for (int j = 0; j < n && ok; j += 2)
            for (int s = 0; s < takers; ++s) {
                if (j < walk.steps(s)) load(!keys, walk.tile(j >> 1, s));
                if (j + 2 < walk.steps(s)) load(keys, walk.tile((j + 2) >> 1, s));
            }
        if (bad) set_status(a.status, FATHOM_ERR_INVALID_ARG);
    } else if (warp < 4) {
        // ---------------------------------------------------- products: a warp for each slot, so
        // that one waits and prepares while the other's are in the pipe
        const int me = warp - 1;
        if (warp == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&s_tmem)),
                         "n"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
            tc_before();
        }
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory");
        if (me < kSlots) {
            tc_after();
            const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
            const uint32_t common = (1u << 4) | (type << 7) | (type << 10) | ((128u >> 4) << 24);
            const uint32_t idesc_qk = common | ((uint32_t)(kStep >> 3) << 17);
            const uint32_t idesc_pv = common | (1u << 16) | ((uint32_t)(d >> 3) << 17);
            constexpr int kStageStep = kTileBytes >> 4, kHalfStep = (kStep * 128) >> 4;
            const uint64_t k_ring = umma_desc(ring, 16), v_ring = umma_desc(ring, kBlockBytes);
            const uint64_t q_desc = umma_desc(q_addr, 16) + (shared ? me * kStageStep : 0);
            const uint32_t s_col = s_tmem + me * kTile, o_at = s_tmem + o_col + me * d;
            const int takers = walk.takers(), steps = walk.steps(me);
            Place<kStages> at;
            int k = 0, v = 0;                                   // stages of the tiles in use
            bool ok = mbar_wait(bar(kQueries), 0, stop, a.wait_ns);
            const auto take = [&](int &stage) {
                stage = at.stage;
                ok = ok && mbar_wait(bar(kFull + at.stage), at.phase, stop, a.wait_ns);
                at.next();
            };
            // The other slot's tile is passed on: seen full and freed.  A warp that left such phases
            // out could come back to a stage two of them early, which their parity does not show.
            const auto pass = [&](const Place<kStages> &of) {
                ok = ok && mbar_wait(bar(kFull + of.stage), of.phase, stop, a.wait_ns);
                if (ok && elect_one()) mbar_arrive(bar(kEmpty + of.stage));
                __syncwarp();
            };
            // S = Q K^T of step j, by one lane
            const auto scores = [&](int j) {
                const uint64_t k_desc = k_ring + k * kStageStep + (j & 1) * kHalfStep;
#pragma unroll
                for (int x = 0; x < NB * 4; ++x) {              // 16 channels: 32 bytes of a 64-channel block
                    const int off = ((x >> 2) * kBlockBytes + (x & 3) * 32) >> 4;
                    if (x < d / 16) umma_ss(s_col + (j & 1) * kStep, q_desc + off, k_desc + off, idesc_qk, x > 0);
                }
                umma_commit(bar(kScores + 2 * me + (j & 1)));
            };
            for (int s = 0; s < takers; ++s) {
                if (walk.steps(s) == 0) continue;
                if (shared || s == me) {
                    take(k);
                } else {
                    pass(at);
                    at.next();
                }
            }
            tc_after();
            if (ok && steps > 0 && elect_one()) {
                scores(0);
                scores(1);
                umma_commit(bar(kEmpty + k));
            }
            __syncwarp();
            for (int j = 0; j < walk.steps(0) && ok; ++j) {
                const bool more = j + 2 < steps;
                Place<kStages> others[2];                       // of V and K, passed on when this step is out
                int n_others = 0;
                if (!(j & 1))
                    for (int s = 0; s < takers; ++s) {
                        const bool has[2] = {j < walk.steps(s), j + 2 < walk.steps(s)};
                        if (shared || s == me) {
                            if (has[0]) take(v);
                            if (has[1]) take(k);
                        } else {
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (has[x]) {
                                    others[x] = at;
                                    n_others = x + 1;
                                    at.next();
                                }
                        }
                    }
                if (j < steps) {
                    const uint64_t v_desc = v_ring + v * kStageStep + (j & 1) * kHalfStep;
                    ok = ok && mbar_wait(bar(kProbs + 2 * me + (j & 1)), (j >> 1) & 1, stop, a.wait_ns);
                    tc_after();
                    if (ok && elect_one()) {
                        // O += P V of step j; then S of step j + 2 goes where P was
#pragma unroll
                        for (int x = 0; x < kStep / 16; ++x)    // 16 keys: 2048 bytes of V, 8 columns of P
                            umma_ts(o_at, s_col + (j & 1) * kStep + x * 8, v_desc + x * (2048 >> 4), idesc_pv,
                                    j > 0 || x > 0);
                        // the last one's sums are what the CTA ends with: nothing arrives after that
                        if (j & 1) umma_commit(bar(kEmpty + v));
                        umma_commit(bar(kDone + 2 * me + (j & 1)));
                        if (more) {
                            scores(j + 2);
                            if (j & 1) umma_commit(bar(kEmpty + k));
                        }
                    }
                    __syncwarp();
                }
                if (n_others > 0) pass(others[0]);
                if (n_others > 1) pass(others[1]);
            }
        }
    } else {
        // ----------------------------------------------------- softmax
        const int s = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
        const int seq = sequence_of(s, r);
        const bool mine = seq >= 0;
        const bool live = __any_sync(0xFFFFFFFFu, mine);
        const int b = mine ? seq : 0, head = h * G + r % G;
        const int seq_len = a.q.seq_lens[b];
        const float slope = a.q.slopes ? a.q.slopes[head] * kLog2e : 0.0f;
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory");
        tc_after();
        const bool plain = a.score.cap == 0.0f && !a.q.slopes && a.score.scale > 0.0f;
        const uint32_t lane_addr = s_tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_addr + o_col + s * d;
        const int steps = walk.steps(s);
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            const int which = 2 * s + (j & 1);
            const uint32_t s_addr = lane_addr + s * kTile + (j & 1) * kStep;
            ok = mbar_wait(bar(kScores + which), (j >> 1) & 1, stop, a.wait_ns);
            if (!ok) break;
            tc_after();
            if (live) {
                const int key0 = (t0 + walk.tile(j >> 1, s)) * kTile + (j & 1) * kStep;
                const int valid = a.prefix_len - key0;          // keys of this step
                float x[kStep];
#pragma unroll
                for (int c = 0; c < kStep; c += 32) tmem_ld32(s_addr + c, x + c);
                tc_wait_ld();
                float mult = a.score.scale;
                if (!plain || valid < kStep) {
                    const float dist = (float)(seq_len - 1 - key0);
#pragma unroll
                    for (int k = 0; k < kStep; ++k) {
                        x[k] = score_logit(x[k], a.score) - slope * (dist - (float)k);
                        if (k >= valid) x[k] = -INFINITY;
                    }
                    mult = 1.0f;
                }
                float tops[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int k = 4; k < kStep; ++k) tops[k & 3] = fmaxf(tops[k & 3], x[k]);
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * mult;
                // rows of no sequence have no vote: behind the slot's last, Q is whatever lay in shared memory
                if (__any_sync(0xFFFFFFFFu, mine && top > m + kRescale)) {
                    const float next = fmaxf(m, top);
                    const float w = m == next ? 1.0f : exp2_fast(m - next);
                    m = next;
                    l *= w;
                    if (j > 0) {
                        ok = mbar_wait(bar(kDone + 2 * s + ((j - 1) & 1)), ((j - 1) >> 1) & 1, stop,
                                       a.wait_ns);
                        if (!ok) break;
                        tc_after();
#pragma unroll 1
                        for (int c = 0; c < d; c += 16) {
                            float o[16];
                            tmem_ld16(o_addr + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= w;
                            tmem_st16(o_addr + c, reinterpret_cast<const uint32_t *>(o));
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : prob_reference<T>(m);
                const Pair mult2(mult, mult), ref2(-ref, -ref);
                Pair sum[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] = Pair(0.0f, 0.0f);
                uint32_t p[kStep / 2];
#pragma unroll
                for (int k = 0; k < kStep; k += 2) {
                    float p0, p1;
                    fma2(Pair(x[k], x[k + 1]), mult2, ref2).split(p0, p1);
                    // the sum is of the rounded probabilities, those that V is weighted with: where few
                    // keys have most of the weight, their rounding then cancels
                    p[k >> 1] = narrow2<T>(exp2_fast(p0), exp2_fast(p1));
                    const float2 w = widen2<T>(p[k >> 1]);
                    sum[(k >> 1) & 3] = sum[(k >> 1) & 3] + Pair(w.x, w.y);
                }
                tmem_st32(s_addr, reinterpret_cast<const float *>(p));
                {
                    float s0, s1;
                    ((sum[0] + sum[1]) + (sum[2] + sum[3])).split(s0, s1);
                    l += s0 + s1;
                }
                tc_wait_st();
            }
            tc_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(bar(kProbs + which));
        }
        for (int x = 0; x < 2; ++x)
            if (ok && steps > 0) ok = mbar_wait(bar(kDone + 2 * s + x), (steps / 2 - 1) & 1, stop, a.wait_ns);
        if (ok && live) {
            tc_after();
            const long long place = place_of(s, r);
            if (mine) a.pv.ml[place] = make_float2(prob_reference<T>(m), l);
            if (steps > 0) {
                // 32 channels of the warp's 32 rows at a time through shared memory, so that a store
                // is four rows of 128 bytes (a lane's own row at a time: 32 rows, 1.6 us longer)
                // the slot's own tile of Q, done with, or room behind the one that the other may read
                const uint32_t stage = q_addr + (shared ? s * kTileBytes : kTileBytes + s * kStageBytes) +
                                       (warp & 3) * (kStageBytes / 4);
                long long to[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) to[x] = __shfl_sync(0xFFFFFFFFu, place, 4 * x + (lane >> 3));
#pragma unroll 1
                for (int c = 0; c < d; c += 32) {
                    float o[32];
                    __syncwarp();
                    tmem_ld32(o_addr + c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         stage + lane * 128 + ((k ^ (lane & 7)) << 4)),
                                     "f"(o[4 * k]), "f"(o[4 * k + 1]), "f"(o[4 * k + 2]), "f"(o[4 * k + 3])
                                     : "memory");
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int row = 4 * x + (lane >> 3), k = lane & 7;
                        float4 v;
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                                     : "r"(stage + row * 128 + ((k ^ (row & 7)) << 4)));
                        if (to[x] >= 0) *reinterpret_cast<float4 *>(a.pv.o + to[x] * d + c + 4 * k) = v;
                    }
                }
            }
        }
    }
    tc_before();
    __syncthreads();
    if (*stop) {                                                // the same for all: no warp waits any more
        if (warp == 0) {
            wait_anyway(bar(kQueries), 0);
            for (int x = 0; x < kStages; ++x)
                if (s_copied[x] >= 0) wait_anyway(bar(kFull + x), s_copied[x]);
            if (lane == 0) set_status(a.status, FATHOM_ERR_TIMEOUT);
        } else if (warp <= kSlots) {
            if (elect_one()) umma_commit(bar(kDrained + warp - 1));   // by the lane that issued the products
            __syncwarp();
            wait_anyway(bar(kDrained + warp - 1), 0);
        } else if (warp >= 4) {
            const long long place = place_of((warp - 4) >> 2, (warp & 3) * 32 + lane);
            if (place >= 0) a.pv.ml[place] = make_float2(-INFINITY, 0.0f);
        }
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(kTmemCols));
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

// A tensor of 16-bit elements, innermost dimension contiguous; strides in
// elements of the others (of no account where there is one of them).
template <int RANK>
bool encode(CUtensorMap *map, const void *base, int dtype, const long long (&size)[RANK],
            const long long (&stride)[RANK - 1], const int (&box)[RANK])
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[RANK], strides[RANK - 1];
    cuuint32_t boxes[RANK], step[RANK];
    for (int i = 0; i < RANK; ++i) {
        dims[i] = (cuuint64_t)size[i];
        boxes[i] = (cuuint32_t)box[i];
        step[i] = 1;
        if (i > 0) strides[i - 1] = (cuuint64_t)(size[i] > 1 ? stride[i - 1] : size[0]) * 2;
    }
    return fn(map, dtype == FATHOM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              RANK, const_cast<void *>(base), dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Boxes of 64 channels by the slots of a page (at most a tile), of one head and page.
bool encode_pages(CUtensorMap *map, const void *base, const PagedView &kv)
{
    const int page = 1 << kv.page_shift;
    return encode<4>(map, base, kv.dtype, {kv.head_dim, page, kv.n_kv_heads, kv.n_pages},
                     {kv.slot_stride, kv.head_stride, kv.page_stride}, {64, std::min(page, kTile), 1, 1});
}

template <typename T, int NB>
cudaError_t launch_shape(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap, const PrefixArgs &a, dim3 ctas,
                         cudaStream_t stream)
{
    using Shape = PrefixShape<NB>;
    const cudaError_t e = cudaFuncSetAttribute(paged_prefix_kernel<T, NB>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    note_launch();
    return launch_overlapped(paged_prefix_kernel<T, NB>, ctas, Shape::kThreads, Shape::kSmem, stream, qmap, kmap, vmap,
                             a);
}

template <typename T>
cudaError_t launch_type(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap, const PrefixArgs &a, dim3 ctas,
                        cudaStream_t stream)
{
    switch ((a.head_dim + 63) / 64) {
    case 1: return launch_shape<T, 1>(qmap, kmap, vmap, a, ctas, stream);
    case 2: return launch_shape<T, 2>(qmap, kmap, vmap, a, ctas, stream);
    case 3: return launch_shape<T, 3>(qmap, kmap, vmap, a, ctas, stream);
    default: return launch_shape<T, 4>(qmap, kmap, vmap, a, ctas, stream);
    }
}

}  // namespace

PrefixPlan plan_prefix(int n_kv_heads, int head_dim, int n_seqs, int group, int prefix_len)
{
    PrefixPlan p{};
    // Below some 8 MB of repeated reads, which mostly hit L2, each sequence reads the prefix for
    // itself: this kernel takes 10 us for the least prefix, the sequences' own 7 us.  Measured with
    // it and without at 8 KV heads of 128: 2 sequences of 1024 keys (4 MB) 9.9 and 8.3 us, of 4096
    // (17 MB) 12.3 and 14.1; 8 of 256 (7 MB) 10.3 and 9.9, of 1024 (29 MB) 10.7 and 14.4, of 16384
    // 28 and 66; at 2 heads of 64 8 of 1024 (4 MB) 9.6 and 7.4, 2 of 16384 (8 MB) 10.7 and 11.3; at
    // 4 of 256 2 of 1024 (4 MB) 10.4 and 9.2, of 4096 (17 MB) 13.7 and 14.5.
    const long long repeated = (long long)(n_seqs - 1) * prefix_len * n_kv_heads * head_dim * 4;
    if (repeated < (8ll << 20)) return p;
    const int slots = head_dim <= 128 ? 2 : 1;
    p.slot_seqs = kRows / group;                     // whole sequences: up to 7 rows of 128 are none
    p.two_blocks = slots == 2 && n_seqs > p.slot_seqs;
    const int cta_seqs = p.slot_seqs * (p.two_blocks ? 2 : 1);
    p.row_groups = (n_seqs + cta_seqs - 1) / cta_seqs;
    p.n_tiles = (prefix_len + kTile - 1) / kTile;
    // one wave of CTAs, of a tile for every slot at least
    const int units = p.row_groups * n_kv_heads, both = slots == 2 && !p.two_blocks ? 2 : 1;
    p.splits = std::max(1, std::min(148 / units, p.n_tiles / both));
    p.parts = p.splits * both;
    return p;
}

cudaError_t launch_paged_prefix(const PagedView &kv, const PagedQuery &q, const PrefixPlan &p,
                                const PartsView &pv, int prefix_len, int max_len, cudaStream_t stream)
{
    CUtensorMap qmap, kmap, vmap;
    if (!encode_pages(&kmap, kv.k, kv) || !encode_pages(&vmap, kv.v, kv) ||
        !encode<3>(&qmap, q.q, kv.dtype, {kv.head_dim, kv.n_kv_heads * q.group, q.n_seqs}, {q.q_hs, q.q_ts},
                   {64, q.group, p.slot_seqs}))
        return cudaErrorInvalidValue;
    PrefixArgs a{};
    a.q = q;
    a.pv = pv;
    a.score = score_args(q.softmax_scale, q.softcap);
    a.table = kv.table;
    a.table_stride = kv.table_stride;
    a.max_len = max_len;
    a.n_heads = kv.n_kv_heads * q.group;
    a.n_pages = kv.n_pages;
    a.page_shift = kv.page_shift;
    a.head_dim = kv.head_dim;
    a.prefix_len = prefix_len;
    a.seqs = q.n_seqs;
    a.slot_seqs = p.slot_seqs;
    a.split_tiles = p.n_tiles / p.splits;
    a.split_rest = p.n_tiles % p.splits;
    a.two_blocks = p.two_blocks;
    a.parts = p.parts;
    a.wait_ns = wait_limit_ns();
    a.status = device_status_ptr();
    const dim3 ctas(p.row_groups, kv.n_kv_heads, p.splits);
    return kv.dtype == FATHOM_BF16 ? launch_type<__nv_bfloat16>(qmap, kmap, vmap, a, ctas, stream)
                                   : launch_type<__half>(qmap, kmap, vmap, a, ctas, stream);
}

}  // namespace fathom
