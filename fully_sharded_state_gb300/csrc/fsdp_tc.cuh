// fsdp_tc.cuh -- the matrix product of the operators, on the 5th-generation
// tensor cores of sm_103a:  D[M, N] = A[M, K] B[N, K]^T  in fp32, from two
// bf16 or two fp16 operands, with an epilogue of the operator's own.
//
// One CTA (or a pair of CTAs on two SMs, kCtas = 2) works on one output tile
// of 128 * kCtas rows and TN columns at a time:
//   warp 0    TMA: 64-wide K blocks of A and B into a ring of 128-byte
//             swizzled shared-memory stages (zeros past every edge, so any
//             M, N, K works)
//   warp 1    one thread issues tcgen05.mma; the accumulator is TN columns of
//             tensor memory, double-buffered
//   warps 4.. eight epilogue warps read the finished accumulator, 32 rows
//             and 32 columns of it at a time (a thread holds one row), while
//             the next tile is being multiplied. (Sixteen were no faster: an
//             epilogue is bound by the 128 bytes a clock of shared memory and
//             L1, which the MMAs' operands use as well.) What they read and
//             write in memory goes through 4 KB of shared memory per warp,
//             by bulk copies where rows start on 16 bytes, else so that lanes
//             touch whole lines of a row; with each lane on a row of its own,
//             a 512 x 512 update spent 17 us per tile on its accesses
// The grid is persistent. An operand may be stored with K adjacent
// (row-major [rows, K]) or with its rows adjacent ([K, rows], "MN-major"),
// which the descriptors express; nothing is transposed in memory.
//
// Measured (2048 x 4096 x 32768, bf16, each alone): 1,840 to 1,880 TFLOP/s
// with the loss's exponentials as epilogue, 1,780 to 1,810 and 1,950 to 1,970
// for its two gradients; the tensor pipe is active for 91 to 97 % of the time. Back to back for longer
// the power limit holds all three at 1,620 to 1,720 (8192 x 4096 x 65536).
//
// Every wait is bounded (kWaitNs); a role that gives up leaves its loop, and
// the block counts itself.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fsdp_ops_internal.h"
#include "fsdp_launch.cuh"
#include "fsdp_wait.cuh"

namespace fsdp {
namespace tc {
namespace {

using namespace wait;

constexpr int kBK = 64;        // K elements of a stage: 128 bytes, one swizzle row
constexpr int kTM = 128;       // rows of a CTA's tile: the lanes of tensor memory
constexpr int kEpiWarps = 8;
constexpr int kSplitSms = 152; // multiprocessors that a split sum is spread over at most
constexpr int kParts = kEpiWarps / 4;  // warps that share 32 rows of a tile
constexpr int kThreads = 128 + 32 * kEpiWarps;

// One arrival on the barrier at the same place in CTA `rank` of the cluster.
// Of CTA scope: what it orders is the reads of tensor memory before it, by the
// tcgen05 fence. A release at cluster scope would also wait until the
// epilogue's stores to memory are done, some microseconds for every tile.
__device__ __forceinline__ void bar_arrive_at(uint64_t *bar, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr(bar)), "r"(rank));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// One lane of a converged warp. The warps that issue copies and MMAs run their
// loops whole and elect a lane for the instruction alone: addresses and
// descriptors stay in uniform registers, which these instructions take. With
// the loop inside `if (lane == 0)`, four MMAs and their commit took 220 ns.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// ------------------------------------------------------------ copies, MMA ----

// A box of a 3-D tensor map (x innermost) into shared memory, completing on
// `bar` (of the pair's even CTA when the CTA is one of two).
template <int kCtas>
__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y, int z,
                                         uint64_t *bar)
{
    if (kCtas == 2) {
        // the same offset in the even CTA: its address has the rank bit clear
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(saddr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar) & 0xFEFFFFFFu)
            : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(saddr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar))
            : "memory");
    }
}

// A box of 64 x 32 16-bit elements from shared memory to a tensor map, as one
// of this thread's bulk stores; and waits until those have read their source,
// or are done.
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(saddr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int kCtas>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    if (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}

// One arrival on `bar` (in both CTAs of a pair) when all MMAs issued so far
// are done.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    if (kCtas == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
            " [%0], %1;" ::"r"(saddr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         saddr(bar))
                     : "memory");
}

template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t cols)
{
    if (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(where)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(where)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols)
{
    if (kCtas == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: thread t gets row t's.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i++)
        v[i] = __uint_as_float(r[i]);
}

// The reverse: thread t's values become row t's.
__device__ __forceinline__ void tmem_store32(uint32_t addr, const float (&v)[32])
{
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; i++)
        r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor of a 128-byte swizzled operand tile.
//   K adjacent: rows of 128 bytes (64 of K); 8-row groups 1024 bytes apart.
//     The next 16 of K start 32 bytes on.
//   rows adjacent: blocks of [64 of K][64 rows] (8192 bytes, one after the
//     other along the rows); 8-K groups 1024 bytes apart. The next 16 of K
//     start 2048 bytes on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn)
{
    const uint64_t lead = mn ? (kBK * 128) >> 4 : 1;
    return (uint64_t)((addr >> 4) & 0x3FFF) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__host__ __device__ constexpr uint32_t k_step(bool mn) { return (mn ? 2048 : 32) >> 4; }

// Instruction descriptor: D fp32; A, B bf16 (1) or fp16 (0); majors; N / 8; M / 16.
__host__ __device__ constexpr uint32_t instruction(int rows, int cols, bool bf16, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(cols / 8) << 17) | ((uint32_t)(rows / 16) << 24);
}

// ---------------------------------------------------------------- shapes ----

struct Shape {
    int M, N, K;      // K: the whole contraction
    int batch;        // matrices, on the maps' third axis
    int splits;       // parts of K, each its own tile (its results are partial
                      // sums): at most so many, chosen by Tiles on the device
    int *splits_out;  // where the number is left, or NULL
    int tn;           // columns of a tile, at most TN; a multiple of 16, of 32 for a pair of CTAs
    int whole_units;  // tiles' columns are multiples of 64
    int epi_bytes;    // what the epilogue moves per element, for the choice of the tile
    int sym;          // only the squares on and above the diagonal (M = N)
    int square;       // tiles' columns start on multiples of 32, as their rows do
    int group;        // row tiles that are walked together, for reuse in L2
    uint32_t idesc;
    const int *dyn;   // NULL, or a device count that limits M or K:
    int dyn_base;     //   rows = clamp(*dyn - dyn_base, 0, M or K)
    int dyn_is_k;
};

// Tensor maps of an epilogue's own inputs and outputs, boxes of 64 x 32.
constexpr int kEpiMaps = 3;
struct EpiMaps {
    CUtensorMap m[kEpiMaps];
};

struct Work {
    int z, split;
    int row, col;     // first row and column of the (pair's) tile
    int kb, nkb;      // first K block and their number
};

template <int kCtas, int TN>
struct Tiles {
    static constexpr int kRows = kTM * kCtas;
    static constexpr int kSquare = kRows > TN ? kRows : TN;  // of sym
    int m_tiles, n_tiles, M, K;
    int splits, split_blocks;  // parts of K and the K blocks of one
    uint32_t per_z, total;     // below 2^31

    __device__ __forceinline__ Tiles(const Shape &s)
    {
        M = s.M;
        K = s.K;
        if (s.dyn) {
            int n = *s.dyn - s.dyn_base;
            int &lim = s.dyn_is_k ? K : M;
            lim = n < 0 ? 0 : n < lim ? n : lim;
        }
        m_tiles = (M + kRows - 1) / kRows;
        n_tiles = (s.N + s.tn - 1) / s.tn;
        if (s.sym) {
            const uint32_t q = (M + kSquare - 1) / kSquare;
            per_z = q * (q + 1) / 2 * (kSquare / kRows) * (kSquare / TN);
        } else {
            per_z = (uint32_t)m_tiles * n_tiles;
        }
        splits = 1;
        split_blocks = (K + kBK - 1) / kBK;
        if (s.splits > 1 && per_z > 0)
            choose_splits(s);
        total = per_z * s.batch * splits;
    }

    // K in parts where the tiles, as many as the device's counts leave, do not
    // fill the grid: one to four waves, whichever is estimated shortest, a
    // part's clocks being its blocks' and those of its own start and end, and
    // of the joining (8 bytes per element and part, at 3,000 a clock).
    __device__ void choose_splits(const Shape &s)
    {
        const int blocks = split_blocks, slots = gridDim.x / kCtas, base = (int)per_z * s.batch;
        const int per_block = kCtas == 2 || s.tn > 128 ? 512 : 364;
        const float join = (float)M * (float)s.N * (8.0f / 3000.0f);
        float best = 0.0f;
        int chosen = 1;
        for (int w = 1; w <= 4; w++) {
            int n = slots * w / base;
            n = n < 1 ? 1 : n < s.splits ? n : s.splits;
            const int per = (blocks + n - 1) / n;
            n = (blocks + per - 1) / per;
            const int waves = (base * n + slots - 1) / slots;
            const float t = (float)waves * (float)((int64_t)per * per_block + 4000) + (float)n * join;
            if (w == 1 || t < best) {
                best = t;
                chosen = n;
            }
        }
        split_blocks = (blocks + chosen - 1) / chosen;
        splits = chosen;
        if (s.splits_out && blockIdx.x == 0 && threadIdx.x == 0)
            *s.splits_out = splits;
    }

    __device__ __forceinline__ Work at(const Shape &s, uint32_t t) const
    {
        Work w;
        const uint32_t zs = t / per_z;
        int i = (int)(t - zs * per_z);
        w.split = (int)(zs % (uint32_t)splits);
        w.z = (int)(zs / (uint32_t)splits);
        if (s.sym) {
            constexpr int kSubM = kSquare / kRows, kSubN = kSquare / TN;
            const int sub = i % (kSubM * kSubN);
            const int sq = i / (kSubM * kSubN);
            int c = (int)((sqrtf(8.0f * (float)sq + 1.0f) - 1.0f) * 0.5f);
            while ((c + 1) * (c + 2) / 2 <= sq)
                c++;
            while (c * (c + 1) / 2 > sq)
                c--;
            const int r = sq - c * (c + 1) / 2;
            w.row = r * kSquare + (sub % kSubM) * kRows;
            w.col = c * kSquare + (sub / kSubM) * TN;
        } else {
            const int in_group = s.group * n_tiles;
            const int g = i / in_group;
            i -= g * in_group;
            const int left = m_tiles - g * s.group;
            const int rows = left < s.group ? left : s.group;
            w.row = (g * s.group + i % rows) * kRows;
            w.col = i / rows * s.tn;
        }
        const int nk = (K + kBK - 1) / kBK;
        w.kb = w.split * split_blocks;
        int n = nk - w.kb;
        w.nkb = n < 0 ? 0 : n < split_blocks ? n : split_blocks;
        return w;
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t two(float lo, float hi)
{
    return kBf16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

// 8 of the 16-bit elements of a and b, from number `from` (0 to 7) on.
__device__ __forceinline__ uint4 eight_from(const uint4 &a, const uint4 &b, int from)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; i++)
        w[i] = from & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; i++)
        w[i] = from & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; i++)
        w[i] = from & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What an epilogue thread is given: its row, the tile's first column, and
// where they are in tensor memory. The tile's columns are taken in chunks of
// 32, or units of two chunks: warp `part` of the kParts that share a row takes
// chunks (or units) part, part + kParts, ... below `chunks` (`units`).
struct Slot {
    int z, split, splits, row, col, M, N;
    int part, chunks;
    __device__ __forceinline__ int units() const { return (chunks + 1) / 2; }
    uint32_t tmem;
    unsigned char *stage;  // the warp's stages of 4 KB: 32 rows of 128 bytes
    int lane;
    uint64_t *bar;              // two, of the warp's own loads
    mutable uint32_t bar_phase; // a bit of each
    mutable bool failed;        // a wait on one was given up
    bool mirror;  // sym: also store the transposed element
    bool empty;   // K was empty (only a dynamic one can be): the accumulator
                  // holds nothing, the sum is 0

    __device__ __forceinline__ void load(int chunk, float (&v)[32]) const
    {
        __syncwarp();  // the load is the whole warp's
        tmem_load32(tmem + chunk * 32, v);
    }

    // 16-byte piece c (0..7) of line r (0..31) of the stage. Pieces of a line
    // are permuted by its number: eight lanes on one piece of eight lines, and
    // eight lanes on the pieces of one line, both touch every bank once.
    __device__ __forceinline__ uint4 *piece(int r, int c, int which = 0) const
    {
        return reinterpret_cast<uint4 *>(stage + which * 4096 + r * 128 + ((c ^ (r & 7)) << 4));
    }

    // Group i (0..7) of this lane in a chunk: 4 adjacent columns of a row, the
    // 8 groups of a row on 8 adjacent lanes.
    __device__ __forceinline__ int group_row(int i) const { return row - lane + i * 4 + lane / 8; }
    __device__ __forceinline__ int group_col(int chunk) const { return col + chunk * 32 + lane % 8 * 4; }

    // The threads' own rows of 32 values into the warp's stage.
    __device__ __forceinline__ void put_stage(const float (&mine)[32]) const
    {
#pragma unroll
        for (int c = 0; c < 8; c++)
            *piece(lane, c) = make_uint4(__float_as_uint(mine[4 * c]), __float_as_uint(mine[4 * c + 1]),
                                         __float_as_uint(mine[4 * c + 2]), __float_as_uint(mine[4 * c + 3]));
        __syncwarp();
    }
    __device__ __forceinline__ void get_stage(float (&mine)[32]) const
    {
#pragma unroll
        for (int c = 0; c < 8; c++) {
            const uint4 u = *piece(lane, c);
            mine[4 * c] = __uint_as_float(u.x);
            mine[4 * c + 1] = __uint_as_float(u.y);
            mine[4 * c + 2] = __uint_as_float(u.z);
            mine[4 * c + 3] = __uint_as_float(u.w);
        }
        __syncwarp();
    }
    __device__ __forceinline__ uint4 *group(int i) const { return piece(i * 4 + lane / 8, lane % 8); }

    __device__ __forceinline__ void load_sum(int chunk, float (&mine)[32]) const
    {
        load(chunk, mine);
        if (empty) {
#pragma unroll
            for (int i = 0; i < 32; i++)
                mine[i] = 0.0f;
        }
    }

    // Takes the threads' own rows of a chunk to the lanes by groups and calls
    // f(i, v) for each of this lane's 8. `staged` is called when `mine` is in
    // the stage and its registers are free.
    template <class F, class G>
    __device__ __forceinline__ void spread(float (&mine)[32], F f, G staged) const
    {
        put_stage(mine);
        staged();
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint4 u = *group(i);
            float v[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
            f(i, v);
        }
        __syncwarp();
    }
    template <class F>
    __device__ __forceinline__ void spread(float (&mine)[32], F f) const
    {
        spread(mine, f, [] {});
    }
    template <class F>
    __device__ __forceinline__ void across(int chunk, F f) const
    {
        float mine[32];
        load_sum(chunk, mine);
        spread(mine, f);
    }
    // A unit as 16-bit numbers, for results that need nothing from memory by
    // groups: op(h, v) works on the thread's own row of chunk h (0, 1) of the
    // unit, f(i, u) gets 8 adjacent results for row group_row(i), from column
    // unit_col(unit) on. Half the traffic of taking fp32 across.
    __device__ __forceinline__ int unit_col(int unit) const { return col + unit * 64 + lane % 8 * 8; }
    template <bool kBf16, class Op, class F>
    __device__ __forceinline__ void emit16(int unit, Op op, F f) const
    {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float v[32];
            load_sum(unit * 2 + h, v);
            op(h, v);
#pragma unroll
            for (int g = 0; g < 4; g++)
                *piece(lane, h * 4 + g) = make_uint4(
                    two<kBf16>(v[8 * g], v[8 * g + 1]), two<kBf16>(v[8 * g + 2], v[8 * g + 3]),
                    two<kBf16>(v[8 * g + 4], v[8 * g + 5]), two<kBf16>(v[8 * g + 6], v[8 * g + 7]));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; i++)
            f(i, *group(i));
        __syncwarp();
    }

    // A unit as 16-bit numbers to rows that may start anywhere: to(r) is where
    // the unit's first column of row r (0..31) goes, or NULL. Eight lanes have
    // a row: its whole 16-byte pieces, each cut out of two of the stage's, and
    // the 8 elements before and after them one each.
    template <bool kBf16, class Get, class To>
    __device__ __forceinline__ void emit_rows(int unit, Get get, To to) const
    {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float v[32];
            get(h, v);
#pragma unroll
            for (int g = 0; g < 4; g++)
                *piece(lane, h * 4 + g) = make_uint4(
                    two<kBf16>(v[8 * g], v[8 * g + 1]), two<kBf16>(v[8 * g + 2], v[8 * g + 3]),
                    two<kBf16>(v[8 * g + 4], v[8 * g + 5]), two<kBf16>(v[8 * g + 6], v[8 * g + 7]));
        }
        __syncwarp();
        const int left = N - (col + unit * 64), k = lane % 8;
#pragma unroll 2
        for (int i = 0; i < 8; i++) {
            const int r = i * 4 + lane / 8;
            uint16_t *p = to(r);
            auto element = [&](int e) { return reinterpret_cast<const uint16_t *>(piece(r, e / 8))[e % 8]; };
            if (p == nullptr)
                continue;
            const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15) / 2;  // elements past a 16-byte boundary
            if (left >= 64) {
                if (off == 0) {
                    *reinterpret_cast<uint4 *>(p + k * 8) = *piece(r, k);
                } else {
                    if (k > 0)
                        *reinterpret_cast<uint4 *>(p + k * 8 - off) = eight_from(*piece(r, k - 1), *piece(r, k), 8 - off);
                    const int e = k < 8 - off ? k : 56 + k;
                    p[e] = element(e);
                }
            } else {
                for (int e = k; e < left; e += 8)
                    p[e] = element(e);
            }
        }
        __syncwarp();
    }

    // The stage is free of the bulk store before.
    __device__ __forceinline__ void stage_free() const
    {
        if (lane == 0)
            store_read_wait();
        __syncwarp();
    }
    // A unit of each of n tensor maps into the warp's stages from `at` on (rows
    // and columns past a map are zeros), and the wait for them; bar i. The
    // stages are free before (stage_free, where stores leave from them).
    __device__ __forceinline__ void load_units(const CUtensorMap *maps, int n, int at, int i, int unit) const
    {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            bar_expect(bar + i, n * 4096);
            for (int k = 0; k < n; k++)
                tma_load<1>(stage + (at + k) * 4096, maps + k, col + unit * 64, row, z, bar + i);
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool units_loaded(int i) const
    {
        if (!warp_wait(bar + i, bar_phase >> i & 1))
            failed = true;
        bar_phase ^= 1u << i;
        return !failed;
    }
    // And back out of two of them.
    __device__ __forceinline__ void store_units(const CUtensorMap *a, const CUtensorMap *b, int at, int unit) const
    {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && row < M) {
            tma_store(a, stage + at * 4096, col + unit * 64, row, z);
            tma_store(b, stage + (at + 1) * 4096, col + unit * 64, row, z);
        }
        __syncwarp();
    }

    // A unit as 16-bit numbers to its place in the output's tensor map, whose
    // swizzle is the stage's: no thread reads it back or stores it. get(h, v)
    // makes the thread's own row of chunk h (0, 1) of the unit. Rows and
    // columns past the map are dropped; a tile's columns are whole units.
    template <bool kBf16, class Get>
    __device__ __forceinline__ void emit_map(const CUtensorMap *map, int unit, Get get) const
    {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float v[32];
            get(h, v);
            if (h == 0)
                stage_free();
#pragma unroll
            for (int g = 0; g < 4; g++)
                *piece(lane, h * 4 + g) = make_uint4(
                    two<kBf16>(v[8 * g], v[8 * g + 1]), two<kBf16>(v[8 * g + 2], v[8 * g + 3]),
                    two<kBf16>(v[8 * g + 4], v[8 * g + 5]), two<kBf16>(v[8 * g + 6], v[8 * g + 7]));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && row < M)
            tma_store(map, stage, col + unit * 64, row, z);
        __syncwarp();
    }

    // The reverse: f(i, v) makes this lane's 8 groups, `mine` becomes the
    // thread's own row of them.
    template <class F>
    __device__ __forceinline__ void collect(float (&mine)[32], F f) const
    {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float v[4];
            f(i, v);
            *group(i) = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                   __float_as_uint(v[3]));
        }
        __syncwarp();
        get_stage(mine);
    }
};

// An epilogue E has
//   Params, kLeastTN   its arguments; the narrowest tile it takes
//   kStages            4 KB stages of a warp
//   Pre                what it reads from memory for a chunk or unit, in registers
//   fetch(p, x, part, pre, maps)   starts the first such reads, before the
//                      accumulator is waited for
//   run(p, x, pre, maps)   finishes the tile
//   kPromote           0, or: the sums over K are taken in parts of so many
//                      blocks, each part by add(x, pre) to registers; run
//                      finds them there
// The tensor cores cut their sums off where fp32 would round them, always
// toward zero, so that the error of a long sum grows with its length and does
// not average out; a sum of parts in registers is as exact as a part's.
struct EpiDefaults {
    static constexpr int kLeastTN = 64, kStages = 1, kPromote = 0;
};
// Registers of a thread of warps 0 to 3 and of the epilogue, where the latter
// holds sums: as many together as the launch has (kLaunchRegs of 65,536 / 384).
constexpr int kLaunchRegs = 168, kFewRegs = 72, kManyRegs = 216;
static_assert(kFewRegs * 4 + kManyRegs * kEpiWarps <= kLaunchRegs * (4 + kEpiWarps), "registers of a block");
struct NoPre {
};

template <int kCtas, int TN, int kEpiStages = 1>
struct Ring {
    static constexpr int kRowsB = TN / kCtas;
    static constexpr int kBytesA = kTM * kBK * 2;
    static constexpr int kBytesB = kRowsB * kBK * 2;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kEpiBytes = kEpiWarps * kEpiStages * 4096;
    static constexpr int kFit = (225 * 1024 + 512 - kEpiBytes) / kStageBytes;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kBarriers = 2 * kStages + 4 + 2 * kEpiWarps;
    // 1024 bytes for the swizzle's alignment, the epilogue's stages, the
    // barriers and the TMEM address
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiBytes + kBarriers * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

template <int kCtas, int TN, bool kAMN, bool kBMN, class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ EpiMaps maps, const __grid_constant__ Shape s,
                   const __grid_constant__ typename Epi::Params ep)
{
    using R = Ring<kCtas, TN, Epi::kStages>;
    extern __shared__ unsigned char raw[];
    // the same offset in both CTAs of a pair: dynamic shared memory starts at
    // one address in every CTA
    unsigned char *ring = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
    unsigned char *epi = ring + R::kStages * R::kStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(epi + R::kEpiBytes);
    uint64_t *empty = full + R::kStages;
    uint64_t *acc_full = empty + R::kStages;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *epi_bar = acc_empty + 2;
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(epi_bar + 2 * kEpiWarps);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = kCtas == 2 ? cluster_rank() : 0;
    using T = Tiles<kCtas, TN>;
    const uint32_t first = blockIdx.x / kCtas, step = gridDim.x / kCtas;

    if (warp == 2)
        tmem_alloc<kCtas>(tmem_at, 2 * TN);
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_b) : "memory");
        for (int i = 0; i < R::kStages; i++) {
            bar_init(full + i, 1);
            bar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(acc_full + i, 1);
            bar_init(acc_empty + i, kEpiWarps * kCtas);
        }
        for (int i = 0; i < 2 * kEpiWarps; i++)
            bar_init(epi_bar + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    if (kCtas == 2)
        cluster_sync();
    else
        __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_at;
    bool ok = true;
    // what follows reads the launches before this one's results
    launch_wait();
    launch_next();
    const T tiles(s);
    const int rows_b = s.tn / kCtas;  // of B in this CTA
    const uint32_t stage_bytes = R::kBytesA + (kBMN ? (rows_b + 63) / 64 * 8192 : rows_b * 128);

    if (warp < 4) {
        if (Epi::kPromote > 0)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (uint32_t t = first; ok && t < tiles.total; t += step) {
                const Work w = tiles.at(s, t);
                const int row = w.row + (int)rank * kTM, col = w.col + (int)rank * rows_b;
                for (int kb = 0; kb < w.nkb; kb++) {
                    if (!(ok = warp_wait(empty + stage, phase ^ 1)))
                        break;
                    if (elect_one()) {
                        if (rank == 0)
                            bar_expect(full + stage, stage_bytes * kCtas);
                        unsigned char *a = ring + stage * R::kStageBytes, *b = a + R::kBytesA;
                        const int k = (w.kb + kb) * kBK;
                        if (kAMN) {
    #pragma unroll
                            for (int i = 0; i < kTM / 64; i++)
                                tma_load<kCtas>(a + i * 8192, &map_a, row + i * 64, k, w.z, full + stage);
                        } else {
                            tma_load<kCtas>(a, &map_a, k, row, w.z, full + stage);
                        }
                        if (kBMN) {
    #pragma unroll
                            for (int i = 0; i < R::kRowsB / 64; i++)
                                if (i * 64 < rows_b)
                                    tma_load<kCtas>(b + i * 8192, &map_b, col + i * 64, k, w.z, full + stage);
                        } else {
                            tma_load<kCtas>(b, &map_b, k, col, w.z, full + stage);
                        }
                    }
                    __syncwarp();
                    if (++stage == R::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)
                let_copies_land();
        } else if (warp == 1) {
            if (rank == 0) {
                int stage = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 0;
                for (uint32_t t = first; ok && t < tiles.total; t += step) {
                    const Work w = tiles.at(s, t);
                    if (!(ok = warp_wait(acc_empty + acc, acc_phase ^ 1)))
                        break;
                    fence_after();
                    int part = 0;  // K blocks of the sum so far
                    for (int kb = 0; kb < w.nkb; kb++, part++) {
                        if (Epi::kPromote > 0 && part == Epi::kPromote) {
                            if (elect_one())
                                mma_commit<kCtas>(acc_full + acc);
                            __syncwarp();
                            part = 0;
                            if (++acc == 2) {
                                acc = 0;
                                acc_phase ^= 1;
                            }
                            if (!(ok = warp_wait(acc_empty + acc, acc_phase ^ 1)))
                                break;
                            fence_after();
                        }
                        const uint32_t d = tmem + acc * TN;
                        if (!(ok = warp_wait(full + stage, phase)))
                            break;
                        fence_after();
                        const uint32_t a = saddr(ring + stage * R::kStageBytes);
                        const uint64_t da = operand_desc(a, kAMN), db = operand_desc(a + R::kBytesA, kBMN);
                        if (elect_one()) {
    #pragma unroll
                            for (int k = 0; k < kBK / 16; k++)
                                mma_f16<kCtas>(d, da + k * k_step(kAMN), db + k * k_step(kBMN), s.idesc,
                                               part > 0 || k > 0);
                            mma_commit<kCtas>(empty + stage);
                        }
                        __syncwarp();
                        if (++stage == R::kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (elect_one())
                        mma_commit<kCtas>(acc_full + acc);
                    __syncwarp();
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1;
                    }
                }
            }
        }
    } else {
        if (Epi::kPromote > 0)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        int acc = 0;
        uint32_t acc_phase = 0, bar_phase = 0;
        const int quarter = warp % 4, part = (warp - 4) / 4;
        for (uint32_t t = first; t < tiles.total; t += step) {
            const Work w = tiles.at(s, t);
            Slot x;
            x.z = w.z;
            x.split = w.split;
            x.splits = tiles.splits;
            x.row = w.row + (int)rank * kTM + quarter * 32 + lane;
            x.col = w.col;
            x.M = tiles.M;
            x.N = s.N - w.col < s.tn ? s.N : w.col + s.tn;
            x.part = part;
            x.chunks = (x.N - w.col + 31) / 32;
            x.lane = lane;
            x.stage = epi + (warp - 4) * Epi::kStages * 4096;
            x.bar = epi_bar + 2 * (warp - 4);
            x.bar_phase = bar_phase;
            x.failed = false;
            x.mirror = s.sym && w.row / T::kSquare != w.col / T::kSquare;
            x.empty = w.nkb == 0;
            typename Epi::Pre pre;
            Epi::fetch(ep, x, part, pre, maps);
            int left = w.nkb;
            do {
                ok = bar_wait(acc_full + acc, acc_phase);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                fence_after();
                x.tmem = tmem + acc * TN + ((uint32_t)(quarter * 32) << 16);
                if constexpr (Epi::kPromote > 0)
                    Epi::add(x, pre);
                else
                    Epi::run(ep, x, pre, maps);
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive_at(acc_empty + acc, 0);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
                left -= Epi::kPromote;
            } while (Epi::kPromote > 0 && left > 0);
            if constexpr (Epi::kPromote > 0)
                if (ok)
                    Epi::run(ep, x, pre, maps);
            bar_phase = x.bar_phase;
            ok = ok && !x.failed;
            if (!ok)
                break;
        }
        if (lane == 0)
            store_wait();
        if (!ok)
            let_copies_land();
    }
    if (!ok && lane == 0)
        atomicAdd(&g_wait_timeouts, 1ull);
    __syncwarp();
    fence_before();
    if (kCtas == 2)
        cluster_sync();
    else
        __syncthreads();
    fence_after();
    if (warp == 2)
        tmem_free<kCtas>(tmem, 2 * TN);
}

// ------------------------------------------------------------- launching ----

// An operand: [outer, inner] with row stride ld, `batch` of them. K adjacent
// means inner = K, outer = rows; otherwise inner = rows, outer = K.
struct Operand {
    const void *p;
    int64_t inner, outer, ld, batch_stride;
};

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn()
{
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

inline fsdp_status make_map(CUtensorMap *map, const Operand &o, int batch, int box_outer, bool bf16)
{
    EncodeFn fn = encode_fn();
    if (!fn)
        return set_error(FSDP_ECUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2,
                                   (cuuint64_t)(batch > 1 ? o.batch_stride : o.ld * o.outer) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kBK, (cuuint32_t)box_outer, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    const CUresult r =
        fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
           const_cast<void *>(o.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(FSDP_ECUDA, "cuTensorMapEncodeTiled: error %d (%lld x %lld, ld %lld)", (int)r,
                         (long long)o.inner, (long long)o.outer, (long long)o.ld);
    return FSDP_OK;
}

template <int kCtas, int TN, bool kAMN, bool kBMN, class Epi>
fsdp_status product_as(Shape s, const Operand &a, const Operand &b, bool bf16, const typename Epi::Params &ep,
                       const Operand *const *own, int64_t tiles, int dev, cudaStream_t stream, const char *what)
{
    using R = Ring<kCtas, TN, Epi::kStages>;
    if (s.tn < 1 || s.tn > TN || s.tn % (16 * kCtas) != 0)
        return set_error(FSDP_EUNSUPPORTED, "%s: tiles of %d columns", what, s.tn);
    if (Record *r = current_record())
        return r->add("%s: product ctas %d tile %d columns %d tiles %lld sym %d splits %d stages %d parts %d", what, kCtas, TN,
                      s.tn, (long long)tiles, s.sym, s.splits, Epi::kStages, Epi::kPromote);
    auto kernel = product_kernel<kCtas, TN, kAMN, kBMN, Epi>;
    static std::atomic<uint64_t> ready{0};  // devices (of the first 64) whose attribute is set
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
        if (e != cudaSuccess)
            return set_error(FSDP_ECUDA, "%s: cudaFuncSetAttribute: %s", what, cudaGetErrorString(e));
        cudaFuncAttributes attr;
        if (Epi::kPromote > 0 && (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess || attr.numRegs < kLaunchRegs))
            return set_error(FSDP_ECUDA, "%s: built with too few registers", what);
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    CUtensorMap ma, mb;
    EpiMaps mo{};
    fsdp_status st = make_map(&ma, a, s.batch, kAMN ? kBK : kTM, bf16);
    if (st == FSDP_OK)
        st = make_map(&mb, b, s.batch, kBMN ? kBK : s.tn / kCtas, bf16);
    for (int i = 0; own && i < kEpiMaps && own[i]; i++)
        if (st == FSDP_OK)
            st = make_map(&mo.m[i], *own[i], s.batch, 32, bf16);
    if (st != FSDP_OK)
        return st;
    s.idesc = instruction(kTM * kCtas, s.tn, bf16, kAMN, kBMN);
    const int sms = device_sms(dev);
    const int64_t most = (s.splits > 1 && sms > kSplitSms ? kSplitSms : sms) / kCtas;
    const int64_t grid = s.splits > 1 || tiles > most ? most : tiles;
    return launch(what, kernel, dim3((unsigned)(grid * kCtas)), kThreads, R::kSmem, stream,
                  kCtas, ma, mb, mo, s, ep);
}

// Output tiles of rows x cols, over the batch and the parts of K.
inline int64_t count_tiles(const Shape &s, int64_t rows, int64_t cols)
{
    int64_t n = ((s.M + rows - 1) / rows) * ((s.N + cols - 1) / cols);
    if (s.sym) {
        const int64_t square = rows > cols ? rows : cols, q = (s.M + square - 1) / square;
        n = q * (q + 1) / 2 * (square / rows) * (square / cols);
    }
    return n * s.batch;
}

// The tile of a product. The largest output tile makes the fewest trips to L2,
// a smaller one spreads a small product over more multiprocessors. Taken is
// the one with the least estimate: per wave of tiles the longer of the K
// blocks' clocks and the epilogue's, the shorter once, and a start. A block's
// clocks are those of its MMAs (2 per column of the tile) or of its loads at
// 90 bytes per clock; the epilogue moves its bytes at 35 per clock (measured
// with all multiprocessors at it, 48 x 512 x 512).
struct Form {
    int ctas, tn;
    int columns;          // of a tile: tn, or less where that leaves less of the last tile empty
    int64_t tiles, cost;  // clocks
};
inline int64_t block_clocks(int ctas, int tn)
{
    const int64_t loads = (kTM + tn / ctas) * 128 / 90, mmas = 2 * tn;
    return loads > mmas ? loads : mmas;
}
inline Form best_form(const Shape &s, int64_t sms, int least_tn)
{
    const int64_t nk = (s.K + kBK - 1) / kBK;
    Form best{};
    static const int kForms[4][2] = {{2, 256}, {1, 256}, {1, 128}, {1, 64}};
    for (const int *f : kForms) {
        if (f[1] < least_tn)
            continue;
        const int64_t across = (s.N + f[1] - 1) / f[1];
        // N of an MMA goes in steps of 16 with the 128 rows of one CTA, of 32 with the 256 of a pair
        const int step = s.whole_units ? 64 : 16 * f[0];
        const int columns = s.square || least_tn == 256 ? f[1] : (int)ceil_to((s.N + across - 1) / across, step);
        Form g{f[0], f[1], columns, count_tiles(s, kTM * f[0], f[1]), 0};
        const int64_t slots = sms / g.ctas < 1 ? 1 : sms / g.ctas, waves = (g.tiles + slots - 1) / slots;
        const int64_t mma = nk * block_clocks(g.ctas, columns), epi = 1000 + kTM * columns * s.epi_bytes / 35;
        g.cost = (mma > epi ? waves * mma + epi : waves * epi + mma) + 2500;
        if (s.splits > 1)  // spread over the grid whatever the tiles: what one costs, times their number
            g.cost = g.tiles * g.ctas * mma;
        if (best.tn == 0 || g.cost < best.cost)
            best = g;
    }
    return best;
}

// Launches D = A B^T. `s` needs M, N, K, batch, epi_bytes, sym, dyn* and, for
// split sums, splits; the rest is filled in here. own0..2: what the epilogue
// reads and stores through tensor maps (16-bit, of the operands' type).
template <bool kAMN, bool kBMN, class Epi>
fsdp_status product(Shape s, const Operand &a, const Operand &b, bool bf16, const typename Epi::Params &ep,
                    int dev, cudaStream_t stream, const char *what, const Operand *own0 = nullptr,
                    const Operand *own1 = nullptr, const Operand *own2 = nullptr)
{
    const Operand *const own[kEpiMaps] = {own0, own1, own2};
    s.group = s.group > 0 ? s.group : 8;
    s.whole_units = own0 != nullptr;
    const Form best = best_form(s, device_sms(dev), Epi::kLeastTN);
    s.tn = best.columns;
    if (best.tiles < 1)
        return FSDP_OK;
    if (best.tiles >= (int64_t)1 << 31)
        return set_error(FSDP_ERANGE, "%s: %lld tiles", what, (long long)best.tiles);
    if (best.ctas == 2)
        return product_as<2, 256, kAMN, kBMN, Epi>(s, a, b, bf16, ep, own, best.tiles, dev, stream, what);
    if (best.tn == 256)
        return product_as<1, 256, kAMN, kBMN, Epi>(s, a, b, bf16, ep, own, best.tiles, dev, stream, what);
    if constexpr (Epi::kLeastTN <= 64) {
        if (best.tn == 128)
            return product_as<1, 128, kAMN, kBMN, Epi>(s, a, b, bf16, ep, own, best.tiles, dev, stream, what);
        return product_as<1, 64, kAMN, kBMN, Epi>(s, a, b, bf16, ep, own, best.tiles, dev, stream, what);
    }
    return FSDP_OK;
}

// ------------------------------------------------- rows of an epilogue ----

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ uint16_t to_bf16(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

__device__ __forceinline__ bool aligned(const void *p, unsigned bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Whether all rows from p on, ld 16-bit elements apart, start on 16 bytes.
__device__ __forceinline__ bool rows_of_16(const uint16_t *p, int64_t ld)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 2)) & 15) == 0;
}
template <bool kBf16>
__device__ __forceinline__ uint2 four_16(const float (&v)[4])
{
    return make_uint2(two<kBf16>(v[0], v[1]), two<kBf16>(v[2], v[3]));
}
// 8 adjacent 16-bit elements, of which the first n exist; p is aligned where
// all do.
__device__ __forceinline__ void put8_16(uint16_t *p, const uint4 &u, int n)
{
    if (n >= 8) {
        *reinterpret_cast<uint4 *>(p) = u;
    } else {
        const uint16_t *e = reinterpret_cast<const uint16_t *>(&u);
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n)
                p[i] = e[i];
    }
}
// 4 adjacent elements of a row, of which the first n exist; one access where
// all do and p is aligned.
template <bool kBf16>
__device__ __forceinline__ void put4_16(uint16_t *p, const float (&v)[4], int n)
{
    if (n >= 4 && aligned(p, 8)) {
        *reinterpret_cast<uint2 *>(p) = four_16<kBf16>(v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < n)
                p[i] = kBf16 ? to_bf16(v[i]) : __half_as_ushort(__float2half_rn(v[i]));
    }
}
__device__ __forceinline__ void get4_f32(const float *p, float (&v)[4], int n)
{
    if (n >= 4 && aligned(p, 16)) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = i < n ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void put4_f32(float *p, const float (&v)[4], int n)
{
    if (n >= 4 && aligned(p, 16)) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < n)
                p[i] = v[i];
    }
}

// Partial sums of split products, fp32.
struct PartEpi : EpiDefaults {
    struct Params {
        float *out;  // [batch][splits][M][ld], M as the device's counts leave it, ld a multiple of 8
        int64_t ld;
    };
    using Pre = NoPre;
    static __device__ __forceinline__ void fetch(const Params &, const Slot &, int, Pre &, const EpiMaps &) {}
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &, const EpiMaps &)
    {
        const int rows = x.M - x.group_row(0);
        float *row = p.out + (((int64_t)x.z * x.splits + x.split) * x.M + x.group_row(0)) * p.ld;
#pragma unroll 1
        for (int c = x.part; c < x.chunks; c += kParts) {
            const int col = x.group_col(c);
            x.across(c, [&](int i, float(&v)[4]) {
                if (i * 4 < rows && col < x.N)
                    *reinterpret_cast<float4 *>(row + i * 4 * p.ld + col) = make_float4(v[0], v[1], v[2], v[3]);
            });
        }
    }
};

// fp32 numbers that the parts of split sums take: choose_splits makes four
// waves of tiles at most, each of 128 x 256 per multiprocessor and a row's
// padding, and never more than all parts whole.
inline int64_t parts_floats(int64_t ld, int64_t splits, int64_t rows)
{
    const int64_t waves = 4 * kSplitSms * int64_t(kTM) * (256 + 8), whole = splits * rows * ld;
    return waves < whole ? waves : whole;
}

}  // namespace
}  // namespace tc
}  // namespace fsdp
