// fsdp_group.cu -- matrix products grouped by expert, with ragged numbers of
// rows, for sm_103a:
//
//   forward   y_r = W_e x_r          for the rows r of expert e
//   backward  dx_r = W_e^T dy_r,     dW_e = sum over the rows of e of dy_r x_r^T
//
// The rows lie expert by expert; where each one's begin is known on the device
// alone, so the tiles are found there: a warp scans the offsets, 32 experts at
// a time, as its tiles lead it on (Walk). Rows of no expert get zeros from
// tiles without products.
//
// The products are fsdp_tc.cuh's (TMA into a ring, tcgen05.mma, accumulators in
// tensor memory, an epilogue per warp); a tile's rows are of one expert. An
// operand's tile may run into the next expert's rows: those make rows of the
// result that are not stored. That does not hold for dW, where they would be
// summed. What follows an expert's last rows, up to the end of their K block, is
// therefore zeros: an idle warp puts them into the tiles (Product::mend), or,
// where two CTAs share one barrier for their copies, the block comes from a
// copy that dx's idle warps make (copy_tails).
//
// Many rows an expert are bound by the tensor cores, at the clock that the power
// limit leaves: 16384 rows at 8 experts of 14336 x 4096 forward in 1,180 to 1,240
// us, 1,550 to 1,630 TFLOP/s (alone and cool 1,815, the tensor pipe active for 92
// % of the time), backward of 4096 x 14336 in 2,340 to 2,430. Few rows are bound
// by the weights' way from memory: a row at each of two experts of 14336 x 4096 in
// 42 us, 5.6 TB/s; 1024 rows at 64 of 1024 x 512 forward in 15 us, backward in 33,
// where a block's start, its first loads and its last epilogue show.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "fsdp_copy.cuh"
#include "fsdp_divide.cuh"

namespace fsdp {
namespace {

using namespace tc;

// What a kernel multiplies. The *T forms have the experts' features on the
// tile's 128 rows and their few rows of x (or dy) as its columns.
enum Mode { kForward, kInput, kWeight, kForwardT, kInputT };
constexpr bool a_mn(int m) { return m == kWeight || m == kInputT; }
constexpr bool b_mn(int m) { return m == kWeight || m == kInput; }
constexpr bool turned(int m) { return m == kForwardT || m == kInputT; }

struct GroupShape {
    const int64_t *offsets;  // [experts + 1], as the caller gave them
    int experts, rows;
    int features;            // columns of the result; kWeight: its rows too, `outer`
    int outer;
    int K;                   // of the contraction; kWeight: the expert's rows
    int tn;                  // columns of a tile
    int n_tiles;             // tiles of the features' columns (not turned)
    int bytes_a;             // of A in a stage
    int group;               // row tiles that are walked together, for reuse in L2
    int cut;                 // whether the last round of tiles may be cut
    uint32_t idesc;          // of the MMAs but for their columns
    uint16_t *out;
    int64_t ld, stride;      // of the result; stride: from expert to expert (kWeight)
    int mapped;              // the result has its tensor map
    int split;               // whether sums may be taken over parts of K
    float *parts;            // where they go then: [part][columns][128 rows]
    int *splits;             // into how many parts: left here
};

// Where dW is multiplied by pairs of CTAs: the rows of each expert's last K
// block, to be followed by zeros up to the next 16 (which is what that block's
// MMAs read), of dy and of x. All rows start on 16 bytes.
struct TailJob {
    const uint16_t *from;
    uint16_t *to;  // [experts][64][ld_to]
    int64_t ld, ld_to;
    int cols;
};
struct Tails {
    TailJob job[2];
    bool wanted;
};

struct GroupTile {
    int z;                   // expert, or -1: rows of none
    int a, b;                // first row of A's and B's tile (of the pair's)
    int width;               // its columns
    int lo, hi;              // the expert's rows
    int part;                // where its sums go; -1: it is whole
    int k0, nkb, tail;       // first element of K, K blocks, kWeight: rows of the last one, 0 where it is whole
};

// The tiles of the rows' segments, in order: segment 0 lies before the first
// expert's rows, segment e + 1 is expert e's, the last lies behind them all.
// Offsets are clamped to [0, rows] and to their running maximum, so that no
// value of theirs leads out of the buffers.
//
// Up to kTable segments their ends are put into shared memory first, and the
// tiles counted. The last round of tiles, which would leave multiprocessors
// idle, is then cut into slices of their columns (Cut): with 1024 rows at 8
// experts of 4096 x 4096, 192 tiles on 152 multiprocessors kept them busy for
// 70 % of the time.
constexpr int kTable = 128;

struct Cut {
    uint32_t from;  // tiles from here on are cut
    int slices;     // into so many
    int splits;     // parts of K, of every tile
};

// The segments by windows of 32, a lane each, and pieces of them (tiles, rows
// to copy), numbered through: count(rows) says how many a segment has.
struct Window {
    const int *table;        // the segments' ends, or NULL
    int base, lo, hi;        // the first segment; this lane's rows
    uint32_t first, count;   // its pieces

    template <class Count>
    __device__ __forceinline__ void load(const GroupShape &s, int lane, int at, int carry, uint32_t done, Count pieces)
    {
        base = at;
        if (table) {
            hi = at + lane < s.experts + 2 ? table[at + lane] : s.rows;
        } else {
            int64_t v = at + lane <= s.experts ? s.offsets[at + lane] : s.rows;
            v = v < 0 ? 0 : v > s.rows ? s.rows : v;
            hi = max((int)v, carry);
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int w = __shfl_up_sync(0xffffffffu, hi, o);
                hi = lane >= o ? max(hi, w) : hi;
            }
        }
        lo = __shfl_up_sync(0xffffffffu, hi, 1);
        lo = lane == 0 ? carry : lo;
        count = (uint32_t)pieces(at + lane, hi - lo);
        uint32_t sum = count;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t w = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane >= o ? w : 0;
        }
        first = done + sum - count;
    }
    // All pieces there are; the window goes to the last one's.
    template <class Count>
    __device__ __forceinline__ uint32_t total(const GroupShape &s, int lane, Count pieces)
    {
        while (next(s, lane, pieces)) {
        }
        return __shfl_sync(0xffffffffu, first + count, 31);
    }
    template <class Count>
    __device__ __forceinline__ bool next(const GroupShape &s, int lane, Count pieces)
    {
        if (base + 32 > s.experts + 1)
            return false;
        load(s, lane, base + 32, __shfl_sync(0xffffffffu, hi, 31), __shfl_sync(0xffffffffu, first + count, 31), pieces);
        return true;
    }
    // The lane whose segment has piece t, t rising from call to call; -1 past
    // the last. A converged warp's.
    template <class Count>
    __device__ __forceinline__ int find(const GroupShape &s, int lane, uint32_t t, Count pieces)
    {
        unsigned mine;
        while ((mine = __ballot_sync(0xffffffffu, t >= first && t < first + count)) == 0)
            if (!next(s, lane, pieces))
                return -1;
        return __ffs(mine) - 1;
    }
};

// Tile i of mt x nt: row i, column 0 on entry. `group` rows are walked together.
// (With four divisions a tile, 1024 rows at 64 experts of 1024 x 512 took 15.4 us
// forward, not 14.6.)
__device__ __forceinline__ void raster(int group, int mt, int nt, int &i, int &c)
{
    if (nt == 1)
        return;
    int row0 = 0;
    if (mt > group) {
        const int g = i / (group * nt);
        i -= g * group * nt;
        row0 = g * group;
    }
    const int rows = min(mt - row0, group);
    c = rows == 1 ? i : i / rows;
    i = row0 + i - c * rows;
}

// Part v % splits of a tile's K blocks.
__device__ __forceinline__ void part_of(const Cut &cut, uint32_t v, GroupTile &w)
{
    if (cut.splits == 1)
        return;
    const int i = (int)(v % (uint32_t)cut.splits), from = w.nkb * i / cut.splits, to = w.nkb * (i + 1) / cut.splits;
    w.part = (int)v;
    w.k0 += from * kBK;
    w.tail = to == w.nkb && to > from ? w.tail : 0;
    w.nkb = to - from;
}

template <int kRows, int TN, bool kTurned, bool kSplit>
struct Walk {
    Window win;
    Cut cut;

    static __device__ __forceinline__ int m_tiles(const GroupShape &s, int n)
    {
        return ((kTurned ? s.features : n) + kRows - 1) / kRows;
    }
    static __device__ __forceinline__ int n_tiles(const GroupShape &s, int n)
    {
        return kTurned ? (n + TN - 1) / TN : s.n_tiles;
    }
    __device__ __forceinline__ Walk(const GroupShape &s, int lane, const int *ends, const Cut &c) : cut(c)
    {
        win.table = ends;
        win.load(s, lane, 0, 0, 0, [&](int, int n) { return m_tiles(s, n) * n_tiles(s, n); });
    }
    __device__ __forceinline__ uint32_t total(const GroupShape &s, int lane)
    {
        return win.total(s, lane, [&](int, int n) { return m_tiles(s, n) * n_tiles(s, n); });
    }

    // Tile t of all, t rising from call to call; false past the last. A
    // converged warp's.
    __device__ __forceinline__ bool at(const GroupShape &s, int lane, uint32_t t, GroupTile &w)
    {
        int slice = 0;
        w.width = kTurned ? TN : s.tn;
        const uint32_t v = t;
        if (kSplit)
            t = v / (uint32_t)cut.splits;
        if (!kTurned && t >= cut.from) {
            const uint32_t u = t - cut.from;
            w.width = s.tn / cut.slices;
            slice = (int)(u % cut.slices);
            t = cut.from + u / cut.slices;
        }
        const int l = win.find(s, lane, t, [&](int, int n) { return m_tiles(s, n) * n_tiles(s, n); });
        if (l < 0)
            return false;
        const int seg = win.base + l;
        w.z = seg == s.experts + 1 ? -1 : seg - 1;
        w.lo = __shfl_sync(0xffffffffu, win.lo, l);
        w.hi = __shfl_sync(0xffffffffu, win.hi, l);
        int i = (int)(t - __shfl_sync(0xffffffffu, win.first, l));
        const int n = w.hi - w.lo, mt = m_tiles(s, n), nt = n_tiles(s, n);
        int mi = i, ci = 0;
        raster(s.group, mt, nt, mi, ci);
        const int m = mi * kRows, c = ci * (kTurned ? TN : s.tn) + slice * w.width;
        w.a = kTurned ? m : w.lo + m;
        w.b = kTurned ? w.lo + c : c;
        w.k0 = 0;
        w.nkb = w.z < 0 ? 0 : (s.K + kBK - 1) / kBK;
        w.tail = 0;
        w.part = -1;
        if (kSplit)
            part_of(cut, v, w);
        return true;
    }
};

// The segments' ends into `table` and how their tiles are cut, by the whole
// block; `shared`: two ints per warp of the table.
template <int kCtas>
__device__ __forceinline__ Cut cut_of(const GroupShape &s, int *table, int *shared)
{
    constexpr int kRows = kTM * kCtas, kWarps = kTable / 32;
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    int hi = 0;
    if (t < kTable) {
        const int64_t v = t <= s.experts ? s.offsets[t] : s.rows;
        hi = (int)(v < 0 ? 0 : v > s.rows ? s.rows : v);
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int w = __shfl_up_sync(0xffffffffu, hi, o);
            hi = lane >= o ? max(hi, w) : hi;
        }
        if (lane == 31)
            shared[warp] = hi;
    }
    __syncthreads();
    if (t < kTable) {
        for (int i = 0; i < warp; i++)
            hi = max(hi, shared[i]);
        table[t] = hi;
    }
    __syncthreads();
    Cut c{0xffffffffu, 1, 1};
    if (t < kTable) {
        const int n = hi - (t ? table[t - 1] : 0);
        const uint32_t mine = t < s.experts + 2 ? (uint32_t)((n + kRows - 1) / kRows) * s.n_tiles : 0;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0)
            shared[kWarps + warp] = (int)sum;
    }
    __syncthreads();
    uint32_t total = 0;
    for (int i = 0; i < kWarps; i++)
        total += (uint32_t)shared[kWarps + i];
    const uint32_t slots = gridDim.x / kCtas, left = total % slots;
    if (left == 0)
        return c;
    // rounds of the slices times their clocks: the longer of loads and MMAs, and the epilogue's
    const float blocks = (float)((s.K + kBK - 1) / kBK);
    float best = 0.0f;
    for (int k = 1; k <= 4; k++) {
        if (s.tn % (64 * k) != 0)
            continue;
        const int width = s.tn / k;
        const float loads = (float)(kTM + width / kCtas) * (128.0f / 90.0f), mmas = 2.0f * (float)width;
        const float time = (float)((left * k + slots - 1) / slots) *
                           (blocks * fmaxf(loads, mmas) + 1000.0f + (float)(kTM * 3 / 35) * (float)width);
        if (k == 1 || time < best) {
            best = time;
            c.slices = k;
        }
    }
    if (c.slices > 1)
        c.from = total - left;
    return c;
}

// dW: the same tiles for every expert with rows.
template <int kRows, bool kSplit>
struct WalkWeight {
    Window win;
    Cut cut;
    int m_tiles, n_tiles;
    __device__ __forceinline__ int pieces(const GroupShape &s, int seg, int n) const
    {
        return n > 0 && seg >= 1 && seg <= s.experts ? m_tiles * n_tiles : 0;
    }
    __device__ __forceinline__ WalkWeight(const GroupShape &s, int lane, const int *ends, const Cut &c) : cut(c)
    {
        m_tiles = (s.outer + kRows - 1) / kRows;
        n_tiles = s.n_tiles;
        win.table = ends;
        win.load(s, lane, 0, 0, 0, [&](int seg, int n) { return pieces(s, seg, n); });
    }
    __device__ __forceinline__ uint32_t total(const GroupShape &s, int lane)
    {
        return win.total(s, lane, [&](int seg, int n) { return pieces(s, seg, n); });
    }
    __device__ __forceinline__ bool at(const GroupShape &s, int lane, uint32_t t, GroupTile &w)
    {
        const uint32_t v = t;
        if (kSplit)
            t = v / (uint32_t)cut.splits;
        const int l = win.find(s, lane, t, [&](int seg, int n) { return pieces(s, seg, n); });
        if (l < 0)
            return false;
        w.z = win.base + l - 1;
        w.lo = __shfl_sync(0xffffffffu, win.lo, l);
        w.hi = __shfl_sync(0xffffffffu, win.hi, l);
        int i = (int)(t - __shfl_sync(0xffffffffu, win.first, l));
        int c = 0;
        raster(s.group, m_tiles, n_tiles, i, c);
        w.a = i * kRows;
        w.b = c * s.tn;
        w.width = s.tn;
        w.k0 = w.lo;
        w.nkb = (w.hi - w.lo + kBK - 1) / kBK;
        w.tail = (w.hi - w.lo) % kBK;
        w.part = -1;
        if (kSplit)
            part_of(cut, v, w);
        return true;
    }
};

// A box of rows of x (or dy) that L2 keeps for longer than the weights that
// pass through it: they are read again for every other tile of the columns
// (1024 rows at 8 experts of 4096 x 4096: dx and forward 2 % faster).
template <int kCtas>
__device__ __forceinline__ void tma_load_kept(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar,
                                              uint64_t policy)
{
    if (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(saddr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar) & 0xFEFFFFFFu), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(saddr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar)), "l"(policy)
            : "memory");
}

// The ring of a block. Turned results leave without an epilogue's stages, so
// there is room for more of the narrow ones.
template <int kCtas, int TN, bool kTurned>
struct GroupRing {
    static constexpr int kBytesA = kTM * kBK * 2, kStageBytes = kBytesA + TN / kCtas * kBK * 2;
    static constexpr int kEpiBytes = kTurned ? 0 : kEpiWarps * 4096;
    static constexpr int kFit = (225 * 1024 + 512 - kEpiBytes) / kStageBytes, kMost = 8;
    static constexpr int kStages = kFit < kMost ? kFit : kMost;
    // 1024 bytes for the swizzle's alignment; barriers, the TMEM address, the table
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiBytes + (3 * kStages + 4) * 8 + 8 + (kTable + 16) * 4;
    static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};
constexpr int kBothTN = 256;  // dW's tiles where one kernel has both products (128: 1024 rows at 64 experts 35.8 us, not 33.1)
// Rows of a box of A where its K is adjacent; turned, no more than there are features.
inline int box_a(int mode, int features)
{
    return a_mn(mode) ? kBK : turned(mode) && features < kTM ? (int)ceil_to(features, 8) : kTM;
}
// Rows of a box of B where its K is adjacent: the narrowest slice's, or the
// whole tile's.
constexpr int box_b(int mode, int ctas, int tn) { return b_mn(mode) ? kBK : turned(mode) ? tn : 64 / ctas; }

struct GroupMaps {
    CUtensorMap a, b, a_tail, b_tail, out;
};

// A unit (32 rows of 64 columns) to rows that start anywhere: a row's elements
// side by side on the lanes, two to a lane where rows start on 4 bytes (kTwo).
// (Cut into the 16-byte pieces that a row has, with its ends one by one, dW of
// 113 experts of 1854 x 390 took 108 us, not 90. Words from an odd row's second
// element on, by a shuffle, 326 us for 34 experts of 5662 x 869, not 140.)
template <bool kTwo>
__device__ __forceinline__ void emit_words(const GroupShape &s, const Slot &x, int u, uint16_t *out)
{
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float v[32];
        x.load_sum(u * 2 + h, v);
#pragma unroll
        for (int g = 0; g < 4; g++)
            *x.piece(x.lane, h * 4 + g) =
                make_uint4(two<true>(v[8 * g], v[8 * g + 1]), two<true>(v[8 * g + 2], v[8 * g + 3]),
                           two<true>(v[8 * g + 4], v[8 * g + 5]), two<true>(v[8 * g + 6], v[8 * g + 7]));
    }
    __syncwarp();
    const int row0 = x.row - x.lane, rows = min(32, x.M - row0), left = x.N - (x.col + u * 64);
    uint16_t *to = out + (int64_t)row0 * s.ld + x.col + u * 64 + (kTwo ? 2 * x.lane : x.lane);
#pragma unroll 4
    for (int r = 0; r < rows; r++, to += s.ld) {
        const unsigned char *line = x.stage + r * 128;
        if (kTwo) {
            const uint32_t e = *reinterpret_cast<const uint32_t *>(line + ((x.lane / 4 ^ (r & 7)) << 4) + x.lane % 4 * 4);
            if (2 * x.lane + 1 < left)
                *reinterpret_cast<uint32_t *>(to) = e;
            else if (2 * x.lane < left)
                *to = (uint16_t)e;
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int c = x.lane / 8 + 4 * h;
                const uint16_t e = *reinterpret_cast<const uint16_t *>(line + ((c ^ (r & 7)) << 4) + x.lane % 8 * 2);
                if (x.lane + 32 * h < left)
                    to[32 * h] = e;
            }
        }
    }
    __syncwarp();
}

// The finished accumulator of a tile whose rows are rows of the result. kEnds:
// the result's tensor map ends where its rows do.
template <bool kEnds>
__device__ __forceinline__ void store_rows(const GroupShape &s, const Slot &x, const CUtensorMap *map, uint16_t *out)
{
    const int row0 = x.row - x.lane;
    if (row0 >= x.M)
        return;
    // else a box of 32 rows must not reach into the next expert's
    if (s.mapped && (kEnds || row0 + 32 <= x.M)) {
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts)
            x.emit_map<true>(map, u, [&](int h, float(&v)[32]) { x.load_sum(u * 2 + h, v); });
        return;
    }
    x.stage_free();
    if (rows_of_16(out, s.ld)) {
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts) {
            const int col = x.unit_col(u);
            x.emit16<true>(
                u, [](int, float(&)[32]) {},
                [&](int i, const uint4 &e) {
                    if (x.group_row(i) < x.M)
                        put8_16(out + (int64_t)x.group_row(i) * s.ld + col, e, x.N - col);
                });
        }
    } else if (((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(s.ld * 2)) & 3) == 0) {
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts)
            emit_words<true>(s, x, u, out);
    } else {
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts)
            emit_words<false>(s, x, u, out);
    }
}

// The sums of a part of K as they are, for join_kernel.
__device__ __forceinline__ void store_part(float *part, const Slot &x)
{
    const int row = x.lane + (int)threadIdx.x / 32 % 4 * 32;
#pragma unroll 1
    for (int c = x.part; c < x.chunks; c += kParts) {
        float v[32];
        x.load_sum(c, v);
#pragma unroll
        for (int i = 0; i < 32; i++)
            part[(c * 32 + i) * kTM + row] = v[i];
    }
}

// The same where its columns are: lanes have adjacent columns of the result.
__device__ __forceinline__ void store_turned(const GroupShape &s, const Slot &x)
{
#pragma unroll 1
    for (int c = x.part; c < x.chunks; c += kParts) {
        float v[32];
        x.load_sum(c, v);
        const int r0 = x.col + c * 32;
        uint16_t *to = s.out + (int64_t)r0 * s.ld + x.row;
        if (x.row < x.M) {
#pragma unroll
            for (int i = 0; i < 32; i++)
                if (r0 + i < x.N)
                    to[i * s.ld] = to_bf16(v[i]);
        }
    }
}

// dx's idle warps make what dW needs (a kernel of their own took 27 us of a
// call over 64 experts, and a launch).
__device__ __forceinline__ void copy_tails(const GroupShape &s, const Tails &p, const int *table, int lane, uint32_t warp,
                                           uint32_t warps)
{
    Window win;
    win.table = table;
    auto rows = [&](int seg, int n) { return seg >= 1 && seg <= s.experts ? (n % kBK + 15) / 16 * 16 : 0; };
    win.load(s, lane, 0, 0, 0, rows);
    for (uint32_t u = warp;; u += warps) {
        const int l = win.find(s, lane, u, rows);
        if (l < 0)
            return;
        const int lo = __shfl_sync(0xffffffffu, win.lo, l), hi = __shfl_sync(0xffffffffu, win.hi, l);
        const int r = (int)(u - __shfl_sync(0xffffffffu, win.first, l)), e = win.base + l - 1, rem = (hi - lo) % kBK;
        // the row of both operands at once, 2 x 4 pieces of 16 bytes a lane in flight
        constexpr int kFlight = 4;
        const int64_t from = hi - rem + r, to = (int64_t)e * kBK + r;
        const int most = max(p.job[0].cols, p.job[1].cols);
        for (int c0 = lane * 8; c0 < most; c0 += 256 * kFlight) {
            uint4 v[2][kFlight];
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < kFlight; i++) {
                    const int c = c0 + i * 256, n = p.job[j].cols - c;
                    const uint16_t *q = p.job[j].from + from * p.job[j].ld + c;
                    v[j][i] = make_uint4(0, 0, 0, 0);
                    if (r < rem && n >= 8) {
                        v[j][i] = *reinterpret_cast<const uint4 *>(q);
                    } else if (r < rem && n > 0) {
                        uint16_t *d = reinterpret_cast<uint16_t *>(&v[j][i]);
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            if (k < n)
                                d[k] = q[k];
                    }
                }
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < kFlight; i++)
                    if (c0 + i * 256 < p.job[j].cols)
                        *reinterpret_cast<uint4 *>(p.job[j].to + to * p.job[j].ld_to + c0 + i * 256) = v[j][i];
        }
    }
}

// dW of the experts without rows: zeros, by warps that have nothing else to do
// (as tiles, in rows that do not start on 16 bytes, 16 rows at 46 experts of
// 3619 x 539 took 168 us, not 111).
__device__ __forceinline__ void zero_experts(const GroupShape &s, int lane, uint32_t warp, uint32_t warps)
{
    Window win;
    win.table = nullptr;
    const int some = max(1, 32768 / s.features);  // rows of a piece: 64 KB
    auto pieces = [&](int seg, int n) { return n == 0 && seg >= 1 && seg <= s.experts ? (s.outer + some - 1) / some : 0; };
    win.load(s, lane, 0, 0, 0, pieces);
    for (uint32_t u = warp;; u += warps) {
        const int l = win.find(s, lane, u, pieces);
        if (l < 0)
            return;
        const int r0 = (int)(u - __shfl_sync(0xffffffffu, win.first, l)) * some, rows = min(some, s.outer - r0);
        uint16_t *to = s.out + (int64_t)(win.base + l - 1) * s.stride + (int64_t)r0 * s.ld;
        // one range where the rows are adjacent
        const bool whole = s.ld == s.features;
        const int64_t n = whole ? (int64_t)rows * s.features : s.features;
        for (int r = 0; r < (whole ? 1 : rows); r++, to += s.ld) {
            const int head = (int)min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(to) & 15)) & 15) / 2);
            const int64_t body = (n - head) / 8;
            if (lane < head)
                to[lane] = 0;
            for (int64_t i = lane; i < body; i += 32)
                *reinterpret_cast<uint4 *>(to + head + i * 8) = make_uint4(0, 0, 0, 0);
            const int64_t rest = head + body * 8 + lane;
            if (rest < n)
                to[rest] = 0;
        }
    }
}

// -- the warps' roles -----------------------------------------------------------------

// What a block's warps share.
struct Block {
    unsigned char *ring, *epi;
    uint64_t *full, *empty, *acc_full, *acc_empty, *mended;
    uint32_t *tmem_at;
    int *table, *per_warp;
    uint32_t rank, first, step;
    int warp, lane;
};
template <class R>
__device__ __forceinline__ Block block_of(unsigned char *raw, int ctas)
{
    Block b;
    b.ring = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
    b.epi = b.ring + R::kStages * R::kStageBytes;
    b.full = reinterpret_cast<uint64_t *>(b.epi + R::kEpiBytes);
    b.empty = b.full + R::kStages;
    b.acc_full = b.empty + R::kStages;
    b.acc_empty = b.acc_full + 2;
    b.mended = b.acc_empty + 2;
    b.tmem_at = reinterpret_cast<uint32_t *>(b.mended + R::kStages);
    b.table = reinterpret_cast<int *>(b.tmem_at + 2);
    b.per_warp = b.table + kTable;
    b.rank = ctas == 2 ? cluster_rank() : 0;
    b.first = blockIdx.x / ctas;
    b.step = gridDim.x / ctas;
    b.warp = threadIdx.x / 32;
    b.lane = threadIdx.x % 32;
    return b;
}
// Where a role is in the ring and in the accumulators; a kernel that takes two
// products carries it from one to the next.
struct Place {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    uint32_t mended = 0;  // the phases of those barriers, a bit each
    bool ok = true;
    template <class R>
    __device__ __forceinline__ void next_stage()
    {
        if (++stage == R::kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void next_acc()
    {
        if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1;
        }
    }
};

// kMends: a warp that mends blocks has its part in giving stages back.
template <class R, int kCtas, bool kMends>
__device__ __forceinline__ uint32_t begin_block(const Block &b, int tmem_cols)
{
    if (b.warp == 2)
        tmem_alloc<kCtas>(b.tmem_at, tmem_cols);
    if (threadIdx.x == 0) {
        for (int i = 0; i < R::kStages; i++) {
            bar_init(b.full + i, 1);
            bar_init(b.empty + i, kMends ? 2 : 1);
            bar_init(b.mended + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(b.acc_full + i, 1);
            bar_init(b.acc_empty + i, kEpiWarps * kCtas);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    if (kCtas == 2)
        cluster_sync();
    else
        __syncthreads();
    fence_after();
    return *b.tmem_at;
}
template <int kCtas>
__device__ __forceinline__ void end_block(const Block &b, uint32_t tmem, int tmem_cols, bool ok)
{
    if (b.warp >= 4 && b.lane == 0)
        store_wait();
    if (!ok) {
        if (b.warp != 1)
            let_copies_land();
        if (b.lane == 0)
            atomicAdd(&g_wait_timeouts, 1ull);
    }
    __syncwarp();
    fence_before();
    if (kCtas == 2)
        cluster_sync();
    else
        __syncthreads();
    fence_after();
    if (b.warp == 2)
        tmem_free<kCtas>(tmem, tmem_cols);
}

// One product's tiles. R: the ring; kAcc: columns from one accumulator to the
// other.
template <class R, int kCtas, int TN, int kAcc, int kMode, bool kSplit>
struct Product {
    static constexpr bool kAMN = a_mn(kMode), kBMN = b_mn(kMode), kTurned = turned(kMode);
    static constexpr int kRows = kTM * kCtas, kRowsB = TN / kCtas;
    // dW: where a last K block of few rows gets its zeros from
    static constexpr bool kPadded = kMode == kWeight && kCtas == 2, kMended = kMode == kWeight && kCtas == 1;
    using W = std::conditional_t<kMode == kWeight, WalkWeight<kRows, kSplit>, Walk<kRows, TN, kTurned, kSplit>>;

    static __device__ __forceinline__ void load(const Block &b, const GroupMaps &maps, const GroupShape &s, const int *table,
                                                const Cut &cut, Place &at)
    {
        W walk(s, b.lane, table, cut);
        GroupTile w;
        uint64_t keep;
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        for (uint32_t t = b.first; at.ok && walk.at(s, b.lane, t, w); t += b.step) {
            const int za = kTurned ? w.z : 0, zb = kTurned || kMode == kWeight ? 0 : w.z;
            const int rows_b = w.width / kCtas;
            const uint32_t stage_bytes = (kTurned ? (uint32_t)s.bytes_a : R::kBytesA) + (kBMN ? (rows_b + 63) / 64 * 8192 : rows_b * 128);
            const int row = w.a + (int)b.rank * kTM, col = w.b + (int)b.rank * rows_b;
            for (int kb = 0; kb < w.nkb; kb++) {
                if (!(at.ok = warp_wait(b.empty + at.stage, at.phase ^ 1)))
                    break;
                if (elect_one()) {
                    uint64_t *full = b.full + at.stage;
                    if (b.rank == 0)
                        bar_expect(full, stage_bytes * kCtas);
                    unsigned char *to_a = b.ring + at.stage * R::kStageBytes, *to_b = to_a + R::kBytesA;
                    const bool padded = kPadded && w.tail && kb + 1 == w.nkb;
                    const CUtensorMap *ma = padded ? &maps.a_tail : &maps.a, *mb = padded ? &maps.b_tail : &maps.b;
                    const int k = padded ? w.z * kBK : w.k0 + kb * kBK;
                    if (kAMN) {
#pragma unroll
                        for (int i = 0; i < kTM / 64; i++)
                            tma_load<kCtas>(to_a + i * 8192, ma, row + i * 64, k, za, full);
                    } else if (kTurned) {
                        tma_load<kCtas>(to_a, ma, k, row, za, full);
                    } else {
                        tma_load_kept<kCtas>(to_a, ma, k, row, za, full, keep);
                    }
                    if (kBMN) {
#pragma unroll
                        for (int i = 0; i < kRowsB / 64; i++)
                            if (i * 64 < rows_b)
                                tma_load<kCtas>(to_b + i * 8192, mb, col + i * 64, k, zb, full);
                    } else if (kTurned) {
                        tma_load<kCtas>(to_b, mb, k, col, zb, full);
                    } else {
                        constexpr int kBox = box_b(kMode, kCtas, TN);
#pragma unroll
                        for (int i = 0; i < kRowsB / kBox; i++)
                            if (i * kBox < rows_b)
                                tma_load<kCtas>(to_b + i * kBox * 128, mb, k, col + i * kBox, zb, full);
                    }
                }
                __syncwarp();
                at.template next_stage<R>();
            }
        }
    }

    static __device__ __forceinline__ void multiply(const Block &b, const GroupShape &s, const int *table, const Cut &cut,
                                                    uint32_t tmem, Place &at)
    {
        W walk(s, b.lane, table, cut);
        GroupTile w;
        for (uint32_t t = b.first; at.ok && walk.at(s, b.lane, t, w); t += b.step) {
            if (!(at.ok = warp_wait(b.acc_empty + at.acc, at.acc_phase ^ 1)))
                break;
            fence_after();
            const uint32_t d = tmem + at.acc * kAcc, idesc = s.idesc | (uint32_t)(w.width / 8) << 17;
            for (int kb = 0; kb < w.nkb; kb++) {
                // of a last block of few rows, the steps that have some
                const bool last = kMode == kWeight && w.tail && kb + 1 == w.nkb;
                const int steps = last ? (w.tail + 15) / 16 : kBK / 16;
                if (!(at.ok = warp_wait(b.full + at.stage, at.phase)))
                    break;
                if (kMended && last) {
                    if (!(at.ok = warp_wait(b.mended + at.stage, at.mended >> at.stage & 1)))
                        break;
                    at.mended ^= 1u << at.stage;
                }
                fence_after();
                const uint32_t a = saddr(b.ring + at.stage * R::kStageBytes);
                const uint64_t da = operand_desc(a, kAMN), db = operand_desc(a + R::kBytesA, kBMN);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBK / 16; k++)
                        if (kMode != kWeight || k < steps)
                            mma_f16<kCtas>(d, da + k * k_step(kAMN), db + k * k_step(kBMN), idesc, kb > 0 || k > 0);
                    mma_commit<kCtas>(b.empty + at.stage);
                }
                __syncwarp();
                at.template next_stage<R>();
            }
            if (!at.ok)
                break;
            if (elect_one())
                mma_commit<kCtas>(b.acc_full + at.acc);
            __syncwarp();
            at.next_acc();
        }
    }

    // kMended: a last K block of w.tail rows came with the next expert's behind
    // them. This puts zeros there, up to the next 16, in both operands' tiles: a
    // row of K is a line of 128 bytes in each block of 64 columns, however its
    // 16-byte pieces are permuted. It goes along with every stage, of the other
    // product too, and has a part in giving it back: ahead of the copies it would
    // take a barrier's last but one phase for the one that it waits for, and
    // behind them the next.
    static __device__ __forceinline__ void mend(const Block &b, const GroupShape &s, const int *table, const Cut &cut, Place &at)
    {
        W walk(s, b.lane, table, cut);
        GroupTile w;
        for (uint32_t t = b.first; at.ok && walk.at(s, b.lane, t, w); t += b.step) {
            for (int kb = 0; kb < w.nkb; kb++) {
                if (!(at.ok = warp_wait(b.full + at.stage, at.phase)))
                    break;
                if (kMended && w.tail && kb + 1 == w.nkb) {
                    const int lines = (w.tail + 15) / 16 * 16 - w.tail, blocks = kTM / 64 + w.width / 64;
                    unsigned char *to = b.ring + at.stage * R::kStageBytes + w.tail * 128 + b.lane % 8 * 16;
                    for (int i = b.lane / 8; i < lines * blocks; i += 4) {
                        const int block = i / lines, line = i - block * lines;
                        *reinterpret_cast<uint4 *>(to + block * 8192 + line * 128) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (b.lane == 0)
                        bar_arrive_at(b.mended + at.stage, 0);
                }
                if (b.lane == 0)
                    bar_arrive_at(b.empty + at.stage, 0);
                __syncwarp();
                at.template next_stage<R>();
            }
        }
    }

    static __device__ __forceinline__ void store(const Block &b, const GroupMaps &maps, const GroupShape &s, const int *table,
                                                 const Cut &cut, uint32_t tmem, Place &at)
    {
        W walk(s, b.lane, table, cut);
        GroupTile w;
        const int quarter = b.warp % 4;
        Slot x;
        x.split = 0;
        x.splits = 1;
        x.part = (b.warp - 4) / 4;
        x.lane = b.lane;
        x.stage = b.epi + (b.warp - 4) * 4096;
        x.bar = nullptr;
        x.bar_phase = 0;
        x.failed = x.mirror = false;
        for (uint32_t t = b.first; at.ok && walk.at(s, b.lane, t, w); t += b.step) {
            x.z = kMode == kWeight ? w.z : 0;
            x.row = w.a + (int)b.rank * kTM + quarter * 32 + b.lane;
            x.col = w.b;
            x.M = kTurned ? s.features : kMode == kWeight ? s.outer : w.hi;
            const int end = kTurned ? w.hi : s.features;
            x.N = end - w.b < w.width ? end : w.b + w.width;
            x.chunks = (x.N - w.b + 31) / 32;
            x.empty = w.nkb == 0;
            if (!(at.ok = __all_sync(0xffffffffu, bar_wait(b.acc_full + at.acc, at.acc_phase))))
                break;
            fence_after();
            x.tmem = tmem + at.acc * kAcc + ((uint32_t)(quarter * 32) << 16);
            if (kSplit && w.part >= 0)
                store_part(s.parts + (int64_t)w.part * (kTM * TN), x);
            else if constexpr (kTurned)
                store_turned(s, x);
            else
                store_rows<kMode == kWeight>(s, x, &maps.out, s.out + (kMode == kWeight ? w.z * s.stride : 0));
            fence_before();
            __syncwarp();
            if (b.lane == 0)
                bar_arrive_at(b.acc_empty + at.acc, 0);
            at.next_acc();
        }
    }
};

// Few tiles: the parts of K that fill the multiprocessors, each a tile of its
// own. (One alone takes in 80 GB/s, whatever is on its way to it.)
constexpr int kMostSplits = 32;
__device__ __forceinline__ int splits_for(uint32_t tiles)
{
    const uint32_t n = gridDim.x / max(tiles, 1u);
    return (int)min(max(n, 1u), (uint32_t)kMostSplits);
}

// Adds the parts up, in their order: a warp has 32 rows and 8 columns of a tile.
template <int TN, int kMode>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ GroupShape s)
{
    constexpr bool kTurned = turned(kMode);
    using W = std::conditional_t<kMode == kWeight, WalkWeight<kTM, false>, Walk<kTM, TN, kTurned, false>>;
    launch_wait();
    launch_next();
    const int lane = threadIdx.x % 32, splits = *s.splits;
    if (splits == 1)
        return;
    const Cut cut{0xffffffffu, 1, 1};
    W walk(s, lane, nullptr, cut);
    GroupTile w;
    constexpr int kUnits = kTM / 32 * (TN / 8);
    for (uint32_t u = blockIdx.x * 8 + threadIdx.x / 32; walk.at(s, lane, u / kUnits, w); u += gridDim.x * 8) {
        const int i = (int)(u % kUnits), row = i % 4 * 32 + lane, col = i / 4 * 8;
        const int m = kTurned ? s.features : kMode == kWeight ? s.outer : w.hi;
        const int end = kTurned ? w.hi : s.features, n = end - w.b < w.width ? end - w.b : w.width;
        if (w.a + i % 4 * 32 >= m || col >= n)
            continue;
        const float *part = s.parts + (int64_t)(u / kUnits) * splits * (kTM * TN) + col * kTM + row;
        float v[8] = {};
#pragma unroll 4
        for (int q = 0; q < splits; q++)
#pragma unroll
            for (int c = 0; c < 8; c++)
                v[c] += __ldcg(part + (int64_t)q * (kTM * TN) + c * kTM);
        if (w.a + row >= m)
            continue;
        // a column's 32 rows are adjacent in a turned result, a row's 8 columns in others
        uint16_t *out = s.out + (kMode == kWeight ? w.z * s.stride : 0);
        if (!kTurned && col + 8 <= n && rows_of_16(out, s.ld)) {
            *reinterpret_cast<uint4 *>(out + (int64_t)(w.a + row) * s.ld + w.b + col) =
                make_uint4(two<true>(v[0], v[1]), two<true>(v[2], v[3]), two<true>(v[4], v[5]), two<true>(v[6], v[7]));
            continue;
        }
#pragma unroll
        for (int c = 0; c < 8; c++)
            if (col + c < n)
                out[kTurned ? (int64_t)(w.b + col + c) * s.ld + w.a + row : (int64_t)(w.a + row) * s.ld + w.b + col + c] =
                    to_bf16(v[c]);
    }
}

template <int kCtas, int TN, int kMode, bool kSplit>
__global__ void __launch_bounds__(tc::kThreads, 1)
    group_kernel(const __grid_constant__ GroupMaps maps, const __grid_constant__ GroupShape s,
                 const __grid_constant__ Tails tails)
{
    using R = GroupRing<kCtas, TN, turned(kMode)>;
    using P = Product<R, kCtas, TN, TN, kMode, kSplit>;
    extern __shared__ unsigned char raw[];
    const Block b = block_of<R>(raw, kCtas);
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.b) : "memory");
    }
    const uint32_t tmem = begin_block<R, kCtas, P::kMended>(b, 2 * TN);
    launch_wait();
    launch_next();
    Cut cut{0xffffffffu, 1, 1};
    const int *table = nullptr;
    if (!kSplit && kMode != kWeight && !turned(kMode) && s.cut && s.experts + 2 <= kTable) {
        cut = cut_of<kCtas>(s, b.table, b.per_warp);
        table = b.table;
    }
    if constexpr (kSplit) {
        typename P::W walk(s, b.lane, table, cut);
        cut.splits = splits_for(walk.total(s, b.lane));
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *s.splits = cut.splits;
    }
    Place at;
    if (b.warp == 0)
        P::load(b, maps, s, table, cut, at);
    else if (b.warp == 1 && b.rank == 0)
        P::multiply(b, s, table, cut, tmem, at);
    else if (b.warp >= 4)
        P::store(b, maps, s, table, cut, tmem, at);
    else if ((kMode == kInput || kMode == kInputT) && b.warp > 1 && tails.wanted)
        copy_tails(s, tails, table, b.lane, blockIdx.x * 2 + b.warp - 2, gridDim.x * 2);
    else if (P::kMended && b.warp == 2)
        P::mend(b, s, table, cut, at);
    else if (P::kMended)
        zero_experts(s, b.lane, blockIdx.x, gridDim.x);
    else if (kMode == kWeight && b.warp > 1)
        zero_experts(s, b.lane, blockIdx.x * 2 + b.warp - 2, gridDim.x * 2);
    end_block<kCtas>(b, tmem, 2 * TN, at.ok);
}

// Both products of a backward pass over few rows, one after the other, in
// every other block dW first: dx reads the weights, dW writes as much, and
// neither waits for the other's last tiles.
template <int TN>
__global__ void __launch_bounds__(tc::kThreads, 1)
    group_both_kernel(const __grid_constant__ GroupMaps maps_x, const __grid_constant__ GroupShape sx,
                      const __grid_constant__ GroupMaps maps_w, const __grid_constant__ GroupShape sw)
{
    using R = GroupRing<1, kBothTN, false>;
    using X = Product<R, 1, TN, kBothTN, kInputT, false>;
    using W = Product<R, 1, kBothTN, kBothTN, kWeight, false>;
    extern __shared__ unsigned char raw[];
    const Block b = block_of<R>(raw, 1);
    const uint32_t tmem = begin_block<R, 1, true>(b, 2 * kBothTN);
    launch_wait();
    launch_next();
    const Cut cut{0xffffffffu, 1, 1};
    Place at;
    for (int i = 0; i < 2; i++) {
        const bool first = (i ^ blockIdx.x) & 1;
        if (b.warp == 0)
            first ? W::load(b, maps_w, sw, nullptr, cut, at) : X::load(b, maps_x, sx, nullptr, cut, at);
        else if (b.warp == 1)
            first ? W::multiply(b, sw, nullptr, cut, tmem, at) : X::multiply(b, sx, nullptr, cut, tmem, at);
        else if (b.warp == 2)
            first ? W::mend(b, sw, nullptr, cut, at) : X::mend(b, sx, nullptr, cut, at);
        else if (b.warp == 3 && first)
            zero_experts(sw, b.lane, blockIdx.x, gridDim.x);
        else if (b.warp >= 4)
            first ? W::store(b, maps_w, sw, nullptr, cut, tmem, at) : X::store(b, maps_x, sx, nullptr, cut, tmem, at);
    }
    end_block<1>(b, tmem, 2 * kBothTN, at.ok);
}

// ------------------------------------------------------------------ prep ----

// Matrices to copy so that their rows start on 16 bytes, piece by piece of 8
// elements, one of a thread at a time, whatever the rows' length (a warp per row
// took 94 us for 113 matrices of 1854 x 390, and 37 for one of 84 x 15805; with two
// pieces of a thread on their way, forward over the 113 takes 130 us, not 109, with four 243).
struct PackJob {
    const uint16_t *from;
    uint16_t *to;
    int64_t ld, stride, ld_to;  // stride: from matrix to matrix
    int64_t rows, pieces;       // rows of one matrix; pieces of all of them
    int cols;
    Divide per_row, per_matrix; // pieces of a row; rows of a matrix
    int weights;                // the matrices are the experts', some of which may have no rows
};
struct PackParams {
    PackJob job[3];
    int jobs;
    const int64_t *offsets;
};
// Whether expert e can have rows: it has none for sure where its offsets do not
// rise. Their weights need no copy (16 rows at one of 46 experts of 3619 x 539:
// backward 206 us with all of them copied, 145 without).
__device__ __forceinline__ bool may_have_rows(const int64_t *offsets, int64_t e) { return offsets[e + 1] > offsets[e]; }

// n / d for any n.
__device__ __forceinline__ int64_t over(int64_t n, const Divide &d)
{
    return n < (int64_t)1 << 31 ? (int64_t)d((uint32_t)n) : n / d.d;
}
__global__ void __launch_bounds__(256, 8) group_pack_kernel(const __grid_constant__ PackParams p)
{
    launch_wait();
    launch_next();
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int j = 0; j < p.jobs; j++) {
        const PackJob &q = p.job[j];
        const uint16_t *end = q.from + (over(over(q.pieces - 1, q.per_row), q.per_matrix)) * q.stride + (q.rows - 1) * q.ld + q.cols;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < q.pieces; i += step) {
            const int64_t row = over(i, q.per_row), z = over(row, q.per_matrix);
            const int col = (int)(i - row * q.per_row.d) * 8;
            if (q.weights && !may_have_rows(p.offsets, z))
                continue;
            Piece v;
            v.load(q.from + z * q.stride + (row - z * q.rows) * q.ld + col, q.cols - col, q.from, end);
            *reinterpret_cast<uint4 *>(q.to + row * q.ld_to + col) = v.get();
        }
    }
}

// ------------------------------------------------------------- launching ----

// The tile of a product of about `average` rows for each of `experts`: the
// one with the least estimate, as best_form's. How ragged the rows are only the
// device knows; for numbers that fall off exponentially, ceil(rows / size) is
// 1 / (1 - exp(-size / average)) on average, between 1 and half a tile more than
// the rows fill. So 16 rows each ask for tiles of 32, not 16 (64 experts of
// 1024 x 512: forward 15.3 us, of 16 17.1).
//
// A block takes in 70 bytes a clock where many do (with 90, as for best_form's
// dense products, tiles of 128 x 256 seemed as good as those of pairs: 100 to 600
// rows each at 8 experts of 4096 x 4096 forward were 10 to 17 % slower), and from
// memory, alone or nearly so, 45: few tiles with a long K are split along it (16384 rows at 2
// experts of 128 x 1024: backward 66 us, 35 with both products split). The sizes are taken as for
// kSplitSms multiprocessors, because the workspace is asked for without a device.
struct GroupForm {
    int ctas, tn, columns;
    bool turned, split;
    double rounds, cost;
};
GroupForm group_form(int mode, int64_t experts, double average, int64_t outer, int64_t features, int64_t K)
{
    GroupForm best{};
    auto parts = [&](int64_t size) { return 1.0 / (1.0 - std::exp(-(double)size / average)); };
    auto over = [](int64_t n, int64_t size) { return (double)((n + size - 1) / size); };
    auto consider = [&](int ctas, int tn, bool turn) {
        const int64_t across = (features + tn - 1) / tn;
        const int64_t columns = turn ? tn : ceil_to((features + across - 1) / across, 64);
        const int rows = kTM * ctas;
        double tiles, nk;
        if (mode == kWeight) {
            tiles = (double)experts * over(outer, rows) * over(features, columns);
            nk = average / kBK + 0.5;
        } else {
            nk = over(K, kBK);
            tiles = (double)experts * (turn ? parts(columns) * over(features, rows) : parts(rows) * over(features, columns));
        }
        const double slots = kSplitSms / ctas, waves = tiles < slots ? 1.0 : tiles / slots + 0.5;
        // turned results leave two bytes at a time
        const double epi = 1000 + kTM * (double)columns * (turn ? 6 : 3) / 35;
        const bool few = 2 * tiles <= slots;
        const double mma = nk * std::fmax((double)(kTM + columns / ctas) * 128 / (few ? 45 : 70), 2.0 * (double)columns);
        double cost = (mma > epi ? waves * mma + epi : waves * epi + mma) + 2500;
        bool split = false;
        if (few && ctas == 1 && tn <= 128 && mma > (mode == kForward ? 30000 : 40000)) {
            // the parts' stores, and the launch that adds them up, which the caller's
            // thread takes 3 us for. With and without parts, by the clocks of a tile's
            // loads and multiplications (810 sizes of 1 to 4 experts, inputs from memory or
            // from L2 alike; time over time, geometric means): forward 16,000 1.7, 23,000 1.3, 32,000
            // 1.1, 45,000 0.9, 64,000 0.74; dx 1.5, 1.3, 1.2, 1.06, 0.83; dW 1.6, 1.5, 1.3, 1.1, 0.86
            const double splits = std::fmin((double)kMostSplits, std::floor(slots / tiles)), c = mma / splits + 2 * epi + 2500 + 9000;
            split = c < cost;
            cost = split ? c : cost;
        }
        if (best.tn == 0 || cost < best.cost)
            best = GroupForm{ctas, tn, (int)columns, turn, split, tiles / slots, cost};
    };
    consider(2, 256, false);
    if (mode != kWeight)
        consider(1, 256, false);
    consider(1, 128, false);
    if (mode != kWeight) {
        consider(1, 32, true);
        consider(1, 64, true);
    }
    return best;
}
GroupForm form_of(int mode, int64_t experts, int64_t rows, int64_t outer, int64_t features, int64_t K)
{
    const int64_t used = experts < rows ? experts : rows < 1 ? 1 : rows;
    return group_form(mode, mode == kWeight ? experts : used, (double)rows / (double)used, outer, features, K);
}
int64_t parts_floats_of(const GroupForm &f) { return f.split ? (int64_t)kSplitSms * kTM * f.tn : 0; }

struct GroupOperand {
    Operand o;
    int batch;
};

// A kernel's shared memory, set once for each device (of the first 64).
template <class K>
fsdp_status allow_smem(K kernel, int bytes, int dev, std::atomic<uint64_t> &ready, const char *what)
{
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (ready.load(std::memory_order_relaxed) & bit)
        return FSDP_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess)
        return set_error(FSDP_ECUDA, "%s: cudaFuncSetAttribute: %s", what, cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_relaxed);
    return FSDP_OK;
}

// What a product reads and writes; a and b as the plain form has them (the
// turned one takes them the other way about). a_tail, b_tail, out: or NULL.
struct GroupOperands {
    GroupOperand a, b;
    const GroupOperand *a_tail, *b_tail, *out;
};

template <int kCtas, int kMode>
fsdp_status group_maps(GroupMaps &m, GroupShape &s, const GroupOperands &o)
{
    const GroupOperand &a = turned(kMode) ? o.b : o.a, &b = turned(kMode) ? o.a : o.b;
    const int rows_a = box_a(kMode, s.features), box = box_b(kMode, kCtas, s.tn);
    const GroupOperand *out = turned(kMode) ? nullptr : o.out;
    fsdp_status st = make_map(&m.a, a.o, a.batch, rows_a, true);
    if (st == FSDP_OK)
        st = make_map(&m.b, b.o, b.batch, box, true);
    if (st == FSDP_OK && kMode == kWeight && kCtas == 2)
        st = make_map(&m.a_tail, o.a_tail->o, 1, rows_a, true);
    if (st == FSDP_OK && kMode == kWeight && kCtas == 2)
        st = make_map(&m.b_tail, o.b_tail->o, 1, box, true);
    if (st == FSDP_OK && out)
        st = make_map(&m.out, out->o, out->batch, 32, true);
    s.mapped = out != nullptr;
    s.bytes_a = a_mn(kMode) ? kTM * kBK * 2 : rows_a * kBK * 2;
    s.group = 8;
    s.n_tiles = (s.features + s.tn - 1) / s.tn;
    s.idesc = instruction(kTM * kCtas, 0, true, a_mn(kMode), b_mn(kMode));
    return st;
}

template <int kCtas, int TN, int kMode, bool kSplit = false>
fsdp_status group_as(GroupShape s, const Tails &tails, const GroupOperands &o, int64_t tiles, int dev, cudaStream_t stream,
                     const char *what)
{
    if constexpr (kCtas == 1 && TN <= 128 && !kSplit)
        if (s.split)
            return group_as<kCtas, TN, kMode, true>(s, tails, o, tiles, dev, stream, what);
    using R = GroupRing<kCtas, TN, turned(kMode)>;
    if (s.tn < 1 || s.tn > TN || s.tn % (16 * kCtas) != 0)
        return set_error(FSDP_EUNSUPPORTED, "%s: tiles of %d columns", what, s.tn);
    if (Record *r = current_record())
        return r->add("%s: mode %d ctas %d tile %d columns %d stages %d split %d", what, kMode, kCtas, TN, s.tn, R::kStages,
                      kSplit);
    auto kernel = group_kernel<kCtas, TN, kMode, kSplit>;
    static std::atomic<uint64_t> ready{0};
    GroupMaps m{};
    fsdp_status st = allow_smem(kernel, R::kSmem, dev, ready, what);
    if (st == FSDP_OK)
        st = group_maps<kCtas, kMode>(m, s, o);
    if (st != FSDP_OK)
        return st;
    const int64_t slots = device_sms(dev) / kCtas < 1 ? 1 : device_sms(dev) / kCtas;
    tiles *= kMode == kWeight || turned(kMode) ? 1 : s.tn / 64;  // slices
    // dx may have the last rows to copy too
    int64_t grid = tiles < slots && !tails.wanted ? tiles : slots;
    if (kSplit)
        grid = slots < kSplitSms ? slots : kSplitSms;
    if ((st = launch(what, kernel, dim3((unsigned)(grid * kCtas)), tc::kThreads, R::kSmem, stream, kCtas, m, s, tails)) != FSDP_OK)
        return st;
    if constexpr (kSplit)
        return launch(what, join_kernel<TN, kMode>, dim3((unsigned)(2 * slots)), 256, 0, stream, 1, s);
    return FSDP_OK;
}

// Most tiles that there can be: every segment's last one may be all but empty.
fsdp_status most_tiles(int mode, const GroupShape &s, const GroupForm &f, const char *what, int64_t &tiles)
{
    const int64_t height = kTM * f.ctas, segments = (int64_t)s.experts + 2;
    if (mode == kWeight) {
        tiles = s.experts * ((s.outer + height - 1) / height) * ((s.features + s.tn - 1) / s.tn);
    } else {
        const int64_t size = f.turned ? s.tn : height, other = f.turned ? height : s.tn;
        const int64_t most = s.rows / size + (segments < s.rows ? segments : s.rows);
        tiles = most * ((s.features + other - 1) / other);
    }
    return tiles >= (int64_t)1 << 31 ? set_error(FSDP_ERANGE, "%s: %lld tiles", what, (long long)tiles) : FSDP_OK;
}

// One product in the form that its sizes ask for. s needs offsets, experts,
// rows, features, outer, K and the result.
template <int kMode>
fsdp_status group_product(GroupShape s, const GroupForm &f, const Tails &tails, const GroupOperands &o, int dev,
                          cudaStream_t stream, const char *what)
{
    s.tn = f.columns;
    s.cut = f.rounds < 6 && !f.split;
    s.split = f.split;
    int64_t tiles;
    const fsdp_status st = most_tiles(kMode, s, f, what, tiles);
    if (st != FSDP_OK)
        return st;
    if constexpr (kMode != kWeight) {
        constexpr int kT = kMode == kForward ? kForwardT : kInputT;
        if (f.turned && f.tn == 64)
            return group_as<1, 64, kT>(s, tails, o, tiles, dev, stream, what);
        if (f.turned)
            return group_as<1, 32, kT>(s, tails, o, tiles, dev, stream, what);
    }
    if (f.ctas == 2)
        return group_as<2, 256, kMode>(s, tails, o, tiles, dev, stream, what);
    if constexpr (kMode != kWeight)
        if (f.tn == 256)
            return group_as<1, 256, kMode>(s, tails, o, tiles, dev, stream, what);
    return group_as<1, 128, kMode>(s, tails, o, tiles, dev, stream, what);
}

// Both products of a backward pass in one kernel.
template <int TN>
fsdp_status group_both(GroupShape sx, const GroupOperands &ox, GroupShape sw, const GroupOperands &ow, int dev,
                       cudaStream_t stream, const char *what)
{
    using R = GroupRing<1, kBothTN, false>;
    sx.tn = TN;
    const int64_t across = (sw.features + kBothTN - 1) / kBothTN;
    sw.tn = (int)ceil_to((sw.features + across - 1) / across, 64);
    int64_t tiles_x, tiles_w;
    fsdp_status st = most_tiles(kInput, sx, GroupForm{1, TN, TN, true, false, 0, 0}, what, tiles_x);
    if (st == FSDP_OK)
        st = most_tiles(kWeight, sw, GroupForm{1, kBothTN, sw.tn, false, false, 0, 0}, what, tiles_w);
    if (st != FSDP_OK)
        return st;
    if (Record *r = current_record())
        return r->add("%s: both %d columns %d stages %d", what, TN, sw.tn, R::kStages);
    auto kernel = group_both_kernel<TN>;
    static std::atomic<uint64_t> ready{0};
    GroupMaps mx{}, mw{};
    st = allow_smem(kernel, R::kSmem, dev, ready, what);
    if (st == FSDP_OK)
        st = group_maps<1, kInputT>(mx, sx, ox);
    if (st == FSDP_OK)
        st = group_maps<1, kWeight>(mw, sw, ow);
    if (st != FSDP_OK)
        return st;
    const int64_t most = tiles_x > tiles_w ? tiles_x : tiles_w, sms = device_sms(dev);
    return launch(what, kernel, dim3((unsigned)(most < sms ? most : sms)), tc::kThreads, R::kSmem, stream, 1, mx, sx, mw, sw);
}

bool starts_on_16(const void *p, int64_t ld, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 && stride % 8 == 0;
}

// Whether a backward pass takes both products in one kernel: that saves a launch
// and fills one product's last tiles with the other's, but its tiles are narrow
// (dx 32 or 64 rows, dW one CTA) and its sums whole. Each bound lies where the two
// cross: the one kernel's time over the two kernels', geometric means over 2,800 sizes
// of 1 to 512 experts, those inside the other bounds.
//   rows of an expert   512 0.92, 1024 1.00, 1536 1.07, 4096 1.30: dW in parts is shorter;
//                       of little work later (2^24 products: 1536 0.91, 2048 0.95, 3000 1.04)
//   rows n k            2^30 0.90, 2^31 0.97, 2^31.5 1.00, 2^32 1.11: wider tiles are
//   weights             2^25 0.93, 2^25.5 0.97, 2^26.25 1.01
//   n, dx's K           1024 0.91, 2048 0.97, 4096 1.05: dx's few tiles are long
//   rows k              2^22 0.95, 2^22.5 0.88, 2^23 1.07, 2^24 1.39: its dx leaves two bytes at a time
bool takes_both(const GroupArgs &a)
{
    const int64_t used = a.experts < a.rows ? a.experts : a.rows;
    const double products = (double)a.rows * (double)a.n * (double)a.k;
    return a.rows <= (products <= (double)(1 << 24) ? 2048 : 1024) * used && a.n <= 40 * kBK &&
           a.rows * a.k <= int64_t(7) << 20 && products <= 3e9 && a.experts * a.n * a.k <= int64_t(50) << 20;
}

// The workspace of one call, and its forms.
struct GroupPlan {
    int64_t ldk, ldn;  // row strides of copies with k and n columns
    GroupForm y, dx, dw;
    bool both;
    uint16_t *x, *dy, *w, *x_tail, *dy_tail;
    float *parts;
    int *splits;
    int64_t bytes;
};
GroupPlan group_plan(const GroupArgs &a, bool backward, bool x_on_16, bool dy_on_16, bool w_on_16, void *base)
{
    GroupPlan q{};
    q.ldk = ceil_to(a.k, 8);
    q.ldn = ceil_to(a.n, 8);
    if (backward) {
        q.dx = form_of(kInput, a.experts, a.rows, 0, a.k, a.n);
        q.dw = form_of(kWeight, a.experts, a.rows, a.n, a.k, 0);
        q.both = a.rows > 0 && takes_both(a);
    } else {
        q.y = form_of(kForward, a.experts, a.rows, 0, a.n, a.k);
    }
    Carver c(base);
    q.x = c.take<uint16_t>(x_on_16 ? 0 : a.rows * q.ldk);
    q.w = c.take<uint16_t>(w_on_16 || a.rows == 0 ? 0 : a.experts * a.n * q.ldk);
    if (backward) {
        // without rows, dW's operands are the last rows' copies, of which it reads none
        const bool tails = !q.both && (q.dw.ctas == 2 || a.rows == 0);
        q.dy = c.take<uint16_t>(dy_on_16 ? 0 : a.rows * q.ldn);
        q.x_tail = c.take<uint16_t>(tails ? a.experts * kBK * q.ldk : 0);
        q.dy_tail = c.take<uint16_t>(tails ? a.experts * kBK * q.ldn : 0);
    }
    const int64_t x = q.both ? 0 : parts_floats_of(q.dx), w = q.both ? 0 : parts_floats_of(q.dw), y = parts_floats_of(q.y);
    const int64_t floats = x > w ? x : w > y ? w : y;
    if (floats) {
        q.parts = c.take<float>(floats);
        q.splits = c.take<int>(1);
    }
    q.bytes = c.used();
    return q;
}

// The copies that a call needs, and what the products then read in place of
// the caller's operands.
struct Packer {
    PackParams p{};
    int64_t pieces = 0;
    Operand operand(const void *from, int64_t r, int64_t cols, int64_t ld, int64_t batch, int64_t stride, uint16_t *to,
                    int64_t ld_to, bool direct, bool some = false)
    {
        if (direct)
            return Operand{from, cols, r, ld, stride};
        const int64_t n = (cols + 7) / 8;
        p.job[p.jobs++] = PackJob{static_cast<const uint16_t *>(from), to, ld, stride, ld_to, r, r * batch * n, (int)cols,
                                  Divide((int)n), Divide((int)r), some};
        pieces += r * batch * n;
        return Operand{to, cols, r, ld_to, r * ld_to};
    }
    fsdp_status run(const char *what, const GroupArgs &a, int dev, cudaStream_t s)
    {
        p.offsets = a.offsets;
        const int64_t most = 8 * (int64_t)device_sms(dev), blocks = (pieces + 255) / 256;
        return p.jobs ? launch(what, group_pack_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, 0, s, 1, p)
                      : FSDP_OK;
    }
};

}  // namespace

int64_t group_workspace(const GroupArgs &a, bool backward, bool x_on_16, bool dy_on_16, bool w_on_16)
{
    return group_plan(a, backward, x_on_16, dy_on_16, w_on_16, nullptr).bytes;
}
bool group_x_on_16(const GroupArgs &a) { return starts_on_16(a.x, a.ldx, 0); }
bool group_dy_on_16(const GroupArgs &a) { return starts_on_16(a.dy, a.lddy, 0); }
bool group_w_on_16(const GroupArgs &a) { return starts_on_16(a.weight, a.ldw, a.w_stride); }

fsdp_status launch_grouped_linear(const GroupArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool xd = group_x_on_16(a), wd = group_w_on_16(a);
    const GroupPlan q = group_plan(a, false, xd, true, wd, workspace);
    Packer pk;
    const GroupOperand x{pk.operand(a.x, a.rows, a.k, a.ldx, 1, 0, q.x, q.ldk, xd), 1};
    const GroupOperand w{pk.operand(a.weight, a.n, a.k, a.ldw, a.experts, a.w_stride, q.w, q.ldk, wd, a.rows < 8 * a.experts), (int)a.experts};
    fsdp_status st = pk.run("grouped_linear (copies)", a, dev, s);
    if (st != FSDP_OK)
        return st;
    GroupShape sh{};
    sh.offsets = a.offsets;
    sh.experts = (int)a.experts;
    sh.rows = (int)a.rows;
    sh.features = (int)a.n;
    sh.K = (int)a.k;
    sh.out = static_cast<uint16_t *>(a.y);
    sh.ld = a.ldy;
    const GroupOperand out{Operand{a.y, a.n, a.rows, a.ldy, 0}, 1};
    const GroupOperands o{x, w, nullptr, nullptr, starts_on_16(a.y, a.ldy, 0) ? &out : nullptr};
    sh.parts = q.parts;
    sh.splits = q.splits;
    return group_product<kForward>(sh, q.y, Tails{}, o, dev, s, "grouped_linear");
}

fsdp_status launch_grouped_linear_backward(const GroupArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool xd = group_x_on_16(a), dyd = group_dy_on_16(a), wd = group_w_on_16(a);
    const GroupPlan q = group_plan(a, true, xd, dyd, wd, workspace);
    Packer pk;
    const GroupOperand dyt{Operand{q.dy_tail, a.n, a.experts * kBK, q.ldn, 0}, 1};
    const GroupOperand xt{Operand{q.x_tail, a.k, a.experts * kBK, q.ldk, 0}, 1};
    // without rows dW's maps are of memory that is there; nothing reads through them
    GroupOperand x = xt, dy = dyt, w{};
    if (a.rows > 0) {
        x.o = pk.operand(a.x, a.rows, a.k, a.ldx, 1, 0, q.x, q.ldk, xd);
        dy.o = pk.operand(a.dy, a.rows, a.n, a.lddy, 1, 0, q.dy, q.ldn, dyd);
        w = GroupOperand{pk.operand(a.weight, a.n, a.k, a.ldw, a.experts, a.w_stride, q.w, q.ldk, wd, a.rows < 8 * a.experts), (int)a.experts};
    }
    fsdp_status st = pk.run("grouped_linear_backward (copies)", a, dev, s);
    if (st != FSDP_OK)
        return st;

    // dx = dy W: the weight's rows are the contraction, its columns adjacent
    GroupShape sx{};
    sx.offsets = a.offsets;
    sx.experts = (int)a.experts;
    sx.rows = (int)a.rows;
    sx.features = (int)a.k;
    sx.parts = q.parts;
    sx.splits = q.splits;
    GroupShape sw = sx;
    sx.K = (int)a.n;
    sx.out = static_cast<uint16_t *>(a.dx);
    sx.ld = a.lddx;
    const GroupOperand out_x{Operand{a.dx, a.k, a.rows, a.lddx, 0}, 1};
    const GroupOperands ox{dy, w, nullptr, nullptr, starts_on_16(a.dx, a.lddx, 0) ? &out_x : nullptr};
    // dW = dy^T x: the rows are the contraction, adjacent in neither
    sw.outer = (int)a.n;
    sw.out = static_cast<uint16_t *>(a.dweight);
    sw.ld = a.lddw;
    sw.stride = a.dw_stride;
    const GroupOperand out_w{Operand{a.dweight, a.k, a.n, a.lddw, a.dw_stride}, (int)a.experts};
    const GroupOperands ow{dy, x, &dyt, &xt, starts_on_16(a.dweight, a.lddw, a.dw_stride) ? &out_w : nullptr};

    if (q.both) {
        const char *what = "grouped_linear_backward";
        // few rows each, or little in all: 32 rows a tile, or 64
        const int64_t used = a.experts < a.rows ? a.experts : a.rows;
        return a.rows <= 24 * used ? group_both<32>(sx, ox, sw, ow, dev, s, what) : group_both<64>(sx, ox, sw, ow, dev, s, what);
    }
    if (a.rows > 0) {
        Tails tails{};
        tails.job[0] = TailJob{static_cast<const uint16_t *>(dy.o.p), q.dy_tail, dy.o.ld, q.ldn, (int)a.n};
        tails.job[1] = TailJob{static_cast<const uint16_t *>(x.o.p), q.x_tail, x.o.ld, q.ldk, (int)a.k};
        tails.wanted = q.dw.ctas == 2;
        if ((st = group_product<kInput>(sx, q.dx, tails, ox, dev, s, "grouped_linear_backward (dx)")) !=
            FSDP_OK)
            return st;
    }
    return group_product<kWeight>(sw, q.dw, Tails{}, ow, dev, s, "grouped_linear_backward (dweight)");
}

cudaError_t group_wait_timeouts(unsigned long long *n) { return wait::wait_timeouts(n); }

}  // namespace fsdp
