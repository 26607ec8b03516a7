// fsdp_loss.cu -- softmax cross entropy of a linear head, with its gradients,
// for sm_103a, without the rows x vocab logits.
//
//   prep      keeps the rows that count, one after the other (zeros past
//             them), so ignored rows cost no products and what they hold
//             reaches nothing; their own outputs are written here. A weight
//             whose rows do not start on 16 bytes is copied to rows that do
//   logits    z = hidden weight^T on the tensor cores; the epilogue turns each
//             128-column piece of a row into its maximum, its sum of
//             exp(z - maximum) and, for the gradients, those exponentials in
//             fp16 (2^-11 of a number in (0, 1]; the logits themselves are
//             never stored)
//   rows      joins a row's pieces: log-sum-exp and loss; for the gradients it
//             turns the exponentials into G = softmax - onehot, in place, as
//             bf16: the one rounding of G. Unscaled, because 1 - p of a
//             target is near 1, which is exact, and 1/3 of it is not
//   dhidden   G weight, and dweight = G^T hidden, on the tensor cores, reading
//             weight, G and hidden as they lie (no transposes), scaled in fp32
//
// 6 * rows * cols * vocab flops for a step: nothing is computed twice. Many
// rows are bound by the tensor cores, at the clock that the power limit
// leaves: 8192 x 4096 x 65536 in 7.8 to 8.3 ms (from one board to another),
// 1,590 to 1,690 TFLOP/s. Few rows are bound by reading the weight and by six
// kernels' starts and ends: 256 x 512 x 32000 in 59 us, of which the products'
// flops are 13; the loss alone of one row in 25 us of the caller's time.
// Weights and gradients whose rows do not start on 16 bytes cost a copy each
// way: 1001 x 513 x 50021 with a third of the rows ignored 200 us, about 25 of
// them the weight's copy and 10 the gradient's cut pieces.
#include <math_constants.h>

#include "fsdp_tc.cuh"

namespace fsdp {
namespace {

using namespace tc;

constexpr int kTileN = 256;
constexpr int kPieceCols = kTileN / kParts;  // columns of one (maximum, sum): a warp's
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------ prep ----

struct PrepParams {
    int64_t rows, ldh, lddh, ldx;
    int cols, vocab, chunk;
    const uint16_t *hidden;
    const int64_t *targets;
    int64_t ignore;
    uint16_t *x;      // kept rows, at most ceil64(rows) of them
    int *source, *target;
    int *meta;        // [0] rows kept, [1] rows that count, [2] a counter, zeroed, [3] parts of dhidden's sum
    float *row_loss;
    uint16_t *dhidden;
    // the weight's copy with aligned rows, by the blocks from `packers` on
    int packers;
    const uint16_t *weight;
    uint16_t *w;
    int64_t ldw;
};

__device__ __forceinline__ bool kept(int64_t t, const PrepParams &p)
{
    return t != p.ignore && t >= 0 && t < p.vocab;
}

// A warp copies one row (or zeros it, src NULL), 8 elements a lane. A source
// that does not start on 16 bytes is read in aligned pieces all the same, two
// for a lane's 8, as far as they lie in [lo, hi), the matrix that the row is of
// (50021 x 513: L1 is busy for 32 % of the time, with 8 loads a lane 60 %; the
// time is 32 us either way, and with pieces in place of rows dealt to threads).
__device__ __forceinline__ void copy_row(uint16_t *dst, const uint16_t *src, int n, int lane, const uint16_t *lo,
                                         const uint16_t *hi)
{
    const bool wide = aligned(dst, 16);
    const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15) / 2;
#pragma unroll 2
    for (int c = lane * 8; c < n; c += 256) {
        uint4 u = make_uint4(0, 0, 0, 0);
        const uint16_t *from = src + c - off;  // on 16 bytes
        if (src && c + 8 <= n && (off == 0 || (from >= lo && from + 16 <= hi))) {
            u = *reinterpret_cast<const uint4 *>(from);
            if (off)
                u = eight_from(u, *reinterpret_cast<const uint4 *>(from + 8), off);
        } else if (src) {
            uint16_t *e = reinterpret_cast<uint16_t *>(&u);
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < n)
                    e[i] = src[c + i];
        }
        if (wide && c + 8 <= n) {
            *reinterpret_cast<uint4 *>(dst + c) = u;
        } else {
            const uint16_t *e = reinterpret_cast<const uint16_t *>(&u);
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < n)
                    dst[c + i] = e[i];
        }
    }
}

// Block b packs rows [b * chunk, (b + 1) * chunk). It counts the rows before
// them itself, so one launch does.
__global__ void __launch_bounds__(256) prep_kernel(const PrepParams p)
{
    __shared__ int sums[2];
    __shared__ int place[256];
    __shared__ int warps[8];
    launch_wait();
    launch_next();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if ((int)blockIdx.x >= p.packers) {
        const int64_t step = (int64_t)(gridDim.x - p.packers) * 8;
        const uint16_t *weight_end = p.weight + (p.vocab - 1) * p.ldw + p.cols;
        for (int64_t r = (int64_t)(blockIdx.x - p.packers) * 8 + warp; r < p.vocab; r += step)
            copy_row(p.w + r * p.ldx, p.weight + r * p.ldw, p.cols, lane, p.weight, weight_end);
        return;
    }
    const uint16_t *hidden_end = p.hidden + (p.rows - 1) * p.ldh + p.cols;
    const int64_t lo = (int64_t)blockIdx.x * p.chunk;
    const int64_t hi = lo + p.chunk < p.rows ? lo + p.chunk : p.rows;
    if (threadIdx.x < 2)
        sums[threadIdx.x] = 0;
    __syncthreads();
    int nk = 0, nc = 0;
    for (int64_t r = threadIdx.x; r < lo; r += 256) {
        const int64_t t = p.targets[r];
        nk += kept(t, p);
        nc += t != p.ignore;
    }
    nk = __reduce_add_sync(0xffffffffu, nk);
    nc = __reduce_add_sync(0xffffffffu, nc);
    if (lane == 0) {
        atomicAdd(&sums[0], nk);  // whole numbers: the order is of no matter
        atomicAdd(&sums[1], nc);
    }
    __syncthreads();
    int at = sums[0], count = sums[1];
    for (int64_t r0 = lo; r0 < hi; r0 += 256) {
        const int64_t r = r0 + threadIdx.x;
        const int64_t t = r < hi ? p.targets[r] : p.ignore;
        const bool k = r < hi && kept(t, p), c = r < hi && t != p.ignore;
        const unsigned mask = __ballot_sync(0xffffffffu, k);
        if (lane == 0)
            warps[warp] = __popc(mask);
        const int counted = __syncthreads_count(c);
        int mine = at, all = 0;
        for (int w = 0; w < 8; w++) {
            mine += w < warp ? warps[w] : 0;
            all += warps[w];
        }
        mine += __popc(mask & ((1u << lane) - 1));
        place[threadIdx.x] = k ? mine : -1;
        if (k) {
            p.source[mine] = (int)r;
            p.target[mine] = (int)t;
        } else if (r < hi) {
            p.row_loss[r] = c ? CUDART_NAN_F : 0.0f;
        }
        __syncthreads();
        const int n = (int)(hi - r0 < 256 ? hi - r0 : 256);
        for (int i = warp; i < n; i += 8) {
            if (place[i] >= 0)
                copy_row(p.x + (int64_t)place[i] * p.ldx, p.hidden + (r0 + i) * p.ldh, p.cols, lane, p.hidden, hidden_end);
            else if (p.dhidden)
                copy_row(p.dhidden + (r0 + i) * p.lddh, nullptr, p.cols, lane, nullptr, nullptr);
        }
        __syncthreads();
        at += all;
        count += counted;
    }
    if (hi == p.rows && lo < p.rows) {
        // the last block knows the totals; the rows up to the next whole K
        // block are zero, for the products over the rows
        if (threadIdx.x == 0) {
            p.meta[0] = at;
            p.meta[1] = count;
            p.meta[2] = 0;
        }
        const int end = (at + 63) / 64 * 64;
        for (int i = at + warp; i < end; i += 8)
            copy_row(p.x + (int64_t)i * p.ldx, nullptr, p.cols, lane, nullptr, nullptr);
    }
}

// ---------------------------------------------------------------- logits ----

// Each thread has a row of the tile and 128 adjacent columns, for the maximum
// and then the exponentials. Those leave by the warp's stage, 64 columns of 32
// rows at a time.
//
// kLong: the sums over K are joined in registers from parts of 512, which
// keeps the row losses 7e-8 off (relative) however wide the rows are; one sum
// in tensor memory, read twice, leaves them 7e-8 off at 512 columns, 6e-7 at
// 4096 and 2e-6 at 12288. It costs 1001 x 513 x 50021 8 us of 209, where an
// epilogue's time shows, and nothing at 8192 x 4096 x 65536: taken above 1024
// columns.
constexpr int kLongCols = 1024;
struct LogitsParams {
    bool e;           // whether the exponentials are kept, in the output's map
    float2 *stats;    // [rows][pieces]
    int pieces;
    const int *target;
    float *tlogit;
};
template <bool kLong>
struct LogitsEpi : EpiDefaults {
    static constexpr int kLeastTN = kTileN, kPromote = kLong ? 8 : 0;
    static constexpr int kChunks = kPieceCols / 32;
    using Params = LogitsParams;
    struct Pre {
        int target;
        float sum[kLong ? kChunks : 1][32];
    };
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int, Pre &pre, const EpiMaps &)
    {
        pre.target = x.row < x.M ? p.target[x.row] : -1;
        if constexpr (kLong) {
#pragma unroll
            for (int c = 0; c < kChunks; c++)
#pragma unroll
                for (int i = 0; i < 32; i++)
                    pre.sum[c][i] = 0.0f;
        }
    }
    static __device__ __forceinline__ void get(const Slot &x, const Pre &pre, int c, float (&v)[32])
    {
        if constexpr (kLong) {
#pragma unroll
            for (int i = 0; i < 32; i++)
                v[i] = pre.sum[c][i];
        } else {
            x.load(x.part * kChunks + c, v);
        }
    }
    static __device__ __forceinline__ void add(const Slot &x, Pre &pre)
    {
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
            float v[32];
            x.load(x.part * kChunks + c, v);
#pragma unroll
            for (int i = 0; i < 32; i++)
                pre.sum[c][i] += v[i];
        }
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const EpiMaps &maps)
    {
        // the columns past the vocabulary are compared only where there are some
        const int col = x.col + x.part * kPieceCols;
        if (x.N - col >= kPieceCols)
            piece<true>(p, x, col, pre, maps.m);
        else if (col < x.N)
            piece<false>(p, x, col, pre, maps.m);
    }
    template <bool kWhole>
    static __device__ __forceinline__ void piece(const Params &p, const Slot &x, int col, const Pre &pre,
                                                 const CUtensorMap *map)
    {
        const bool live = x.row < x.M;
        const int n = x.N - col, chunk0 = x.part * kChunks, t = pre.target - col;
        float top = -CUDART_INF_F, at = 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
            float v[32];
            get(x, pre, c, v);
            if (live && t >= c * 32 && t < c * 32 + 32) {
#pragma unroll
                for (int i = 0; i < 32; i++)
                    at = t == c * 32 + i ? v[i] : at;
            }
#pragma unroll
            for (int i = 0; i < 32; i++)
                if (kWhole || c * 32 + i < n)
                    top = fmaxf(top, v[i]);
        }
        // a piece of -inf alone: exp(-inf - 0) = 0, not exp(-inf + inf)
        const float ref = top == -CUDART_INF_F ? 0.0f : top;
        const float shift = ref * kLog2e;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        auto exponentials = [&](int c, float(&v)[32]) {
            get(x, pre, c, v);
#pragma unroll
            for (int i = 0; i < 32; i++) {
                v[i] = kWhole || c * 32 + i < n ? exp2_fast(fmaf(v[i], kLog2e, -shift)) : 0.0f;
                sum[i % 4] += v[i];
            }
        };
        if (p.e) {
#pragma unroll
            for (int u = 0; u < kChunks / 2; u++)
                if (x.col + (chunk0 / 2 + u) * 64 < x.N)
                    x.emit_map<false>(map, chunk0 / 2 + u,
                                      [&](int h, float(&v)[32]) { exponentials(u * 2 + h, v); });
        } else {
#pragma unroll
            for (int c = 0; c < kChunks; c++) {
                float v[32];
                exponentials(c, v);
            }
        }
        if (live) {
            p.stats[(int64_t)x.row * p.pieces + col / kPieceCols] =
                make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
            if (t >= 0 && t < kPieceCols)
                p.tlogit[x.row] = at;
        }
    }
};

// ------------------------------------------------------------------ rows ----

struct RowsParams {
    const int *meta;
    int base, piece_rows;  // this piece's first kept row; its buffer's rows
    int vocab, pieces;
    int segment;           // columns of a block, a multiple of 8
    int64_t lde, rows;
    uint16_t *e;           // exponentials in, G out; NULL: loss alone
    const float2 *stats;
    const int *source, *target;
    const float *tlogit;
    float *row_loss;
    float *loss;           // the last piece: where the loss goes
    int *done;             // blocks that are through (zero before)
    int mean;
};

__device__ __forceinline__ float reduce_max(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < 8; i++)
        v = fmaxf(v, sh[i]);
    __syncthreads();
    return v;
}
__device__ __forceinline__ float reduce_sum(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < 8; i++)
        v += sh[i];
    __syncthreads();
    return v;
}

// What a piece's exponentials count for in a row with the reference `ref`. A
// piece of -inf alone counts for nothing: its exponentials, about 0, are 0, and
// exp(0 - ref) times 0 would be NaN where ref is below -88.
__device__ __forceinline__ float piece_factor(float top, float ref)
{
    return top == -CUDART_INF_F ? 0.0f : expf(top - ref);
}

// Two exponentials as fp16 -> two elements of G as bf16; t: which of them is
// the target's, if any.
__device__ __forceinline__ uint32_t two_of_g(uint32_t e, float f, int t)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&e));
    return pack_bf16(v.x * f - (t == 0 ? 1.0f : 0.0f), v.y * f - (t == 1 ? 1.0f : 0.0f));
}

// What the gradients are multiplied by.
struct Scale {
    const int *meta;
    float grad_scale;
    int mean;
    __device__ __forceinline__ float get() const
    {
        return mean ? grad_scale / (float)max(meta[1], 1) : grad_scale;
    }
};

// Grid (rows, segments of the columns): with few rows several blocks share
// one, each joining its pieces for itself (256 x 32000: 16 us with one block
// per row).
__global__ void __launch_bounds__(256) rows_kernel(const RowsParams p)
{
    __shared__ float sh[8];
    __shared__ bool last;
    launch_wait();
    launch_next();
    const int n = min(max(p.meta[0] - p.base, 0), p.piece_rows);
    const int end = p.e ? (n + 63) / 64 * 64 : n;  // up to the next whole K block: zeros of G
    const int cols = min((p.vocab + 7) / 8 * 8, (int)(blockIdx.y + 1) * p.segment), col0 = blockIdx.y * p.segment;
    constexpr int kStep = 256 * 8, kFlight = 4;
    for (int r = blockIdx.x; r < end; r += gridDim.x) {
        uint16_t *e = p.e + (int64_t)r * p.lde;
        if (r >= n) {
            for (int c = col0 + threadIdx.x * 8; c < cols; c += kStep)
                *reinterpret_cast<uint4 *>(e + c) = make_uint4(0, 0, 0, 0);
            continue;
        }
        const float2 *st = p.stats + (int64_t)r * p.pieces;
        float top = -CUDART_INF_F;
        for (int i = threadIdx.x; i < p.pieces; i += 256)
            top = fmaxf(top, st[i].x);
        top = reduce_max(top, sh);
        const float ref = top == -CUDART_INF_F ? 0.0f : top;
        float sum = 0.0f;
        for (int i = threadIdx.x; i < p.pieces; i += 256) {
            const float2 q = st[i];
            sum += q.y * piece_factor(q.x, ref);  // a NaN in q.y stays one
        }
        sum = reduce_sum(sum, sh);
        if (threadIdx.x == 0 && blockIdx.y == 0)
            p.row_loss[p.source[r]] = ref + logf(sum) - p.tlogit[r];
        if (!p.e)
            continue;
        const int t = p.target[r];
        const float inv = 1.0f / sum;
        auto turn = [&](uint4 u, int c) {
            const float f = piece_factor(st[c / kPieceCols].x, ref) * inv;
            u.x = two_of_g(u.x, f, t - c);
            u.y = two_of_g(u.y, f, t - c - 2);
            u.z = two_of_g(u.z, f, t - c - 4);
            u.w = two_of_g(u.w, f, t - c - 6);
            *reinterpret_cast<uint4 *>(e + c) = u;
        };
        int c = col0 + threadIdx.x * 8;
        for (; c + (kFlight - 1) * kStep < cols; c += kFlight * kStep) {
            uint4 u[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; k++)
                u[k] = *reinterpret_cast<const uint4 *>(e + c + k * kStep);
#pragma unroll
            for (int k = 0; k < kFlight; k++)
                turn(u[k], c + k * kStep);
        }
        for (; c < cols; c += kStep)
            turn(*reinterpret_cast<const uint4 *>(e + c), c);
    }
    if (!p.loss)
        return;
    // The last block of the last piece's launch adds the rows' losses up, in
    // their own order.
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(p.done, 1) == (int)(gridDim.x * gridDim.y) - 1;
    }
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    float s = 0.0f;
    for (int64_t r = threadIdx.x; r < p.rows; r += 256)
        s += __ldcg(p.row_loss + r);
    s = reduce_sum(s, sh);
    if (threadIdx.x == 0)
        *p.loss = p.mean ? s / (float)max(p.meta[1], 1) : s;
}

// ------------------------------------------------------------- gradients ----

// dhidden rows back at their own places, bf16.
struct HiddenEpi : EpiDefaults {
    struct Params {
        uint16_t *out;
        int64_t ld;
        const int *source;
        Scale scale;
    };
    struct Pre {
        int row[8];
        float scale;
    };
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int, Pre &pre, const EpiMaps &)
    {
#pragma unroll
        for (int i = 0; i < 8; i++)
            pre.row[i] = x.group_row(i) < x.M ? p.source[x.group_row(i)] : -1;
        pre.scale = p.scale.get();
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const EpiMaps &)
    {
        if (rows_of_16(p.out, p.ld)) {
#pragma unroll 1
            for (int u = x.part; u < x.units(); u += kParts) {
                const int col = x.unit_col(u);
                auto scaled = [&](int, float(&v)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        v[i] *= pre.scale;
                };
                x.emit16<true>(u, scaled, [&](int i, const uint4 &e) {
                    if (pre.row[i] >= 0)
                        put8_16(p.out + (int64_t)pre.row[i] * p.ld + col, e, x.N - col);
                });
            }
        } else {
            const int row0 = x.row - x.lane;
#pragma unroll 1
            for (int u = x.part; u < x.units(); u += kParts)
                x.emit_rows<true>(
                    u,
                    [&](int h, float(&v)[32]) {
                        x.load_sum(u * 2 + h, v);
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            v[i] *= pre.scale;
                    },
                    [&](int r) {
                        return row0 + r < x.M ? p.out + (int64_t)p.source[row0 + r] * p.ld + x.col + u * 64 : nullptr;
                    });
        }
    }
};

// Adds the parts up: 64 groups of 4 columns, 4 slices of the parts (meta[3] of
// them) per block.
__global__ void __launch_bounds__(256) join_hidden_kernel(const float *parts, int64_t ldp, const int *meta, int base,
                                                          int piece_rows, int cols, const int *source, uint16_t *out,
                                                          int64_t ld, Scale scale)
{
    __shared__ float4 sh[4][64];
    launch_wait();
    launch_next();
    const int n = min(max(meta[0] - base, 0), piece_rows), splits = meta[3];
    const int group = threadIdx.x % 64, slice = threadIdx.x / 64;
    const int c = (blockIdx.y * 64 + group) * 4;
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < cols) {
            const float *src = parts + (int64_t)r * ldp + c;
#pragma unroll 8
            for (int q = slice; q < splits; q += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(src + (int64_t)q * n * ldp);
                s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
            }
        }
        sh[slice][group] = s;
        __syncthreads();
        if (slice == 0 && c < cols) {
#pragma unroll
            for (int q = 1; q < 4; q++) {
                const float4 f = sh[q][group];
                s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
            }
            const float k = scale.get(), v[4] = {s.x * k, s.y * k, s.z * k, s.w * k};
            put4_16<true>(out + (int64_t)source[r] * ld + c, v, cols - c);
        }
        __syncthreads();
    }
}

// dweight, over the pieces of the rows in fp32 where there are several.
struct WeightEpi : EpiDefaults {
    struct Params {
        uint16_t *out;
        int64_t ld;
        float *sum;  // NULL: one piece
        int64_t lds; // a multiple of 8
        int first, last;
        bool mapped;  // out has its tensor map
        Scale scale;
    };
    struct Pre {
        float4 o[8];
        float scale;
    };
    static __device__ __forceinline__ void read_sum(const Params &p, const Slot &x, int chunk, Pre &pre)
    {
        if (!p.sum || p.first || chunk >= x.chunks)
            return;
        const int rows = x.M - x.group_row(0);
        const float *from = p.sum + x.group_row(0) * p.lds + x.group_col(chunk);
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i * 4 < rows && x.group_col(chunk) < x.N)
                pre.o[i] = *reinterpret_cast<const float4 *>(from + i * 4 * p.lds);
    }
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int chunk, Pre &pre, const EpiMaps &)
    {
        pre.scale = p.scale.get();
        read_sum(p, x, chunk, pre);
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const EpiMaps &maps)
    {
        if (p.sum) {
#pragma unroll 1
            for (int c = x.part; c < x.chunks; c += kParts) {
                const int col = x.group_col(c), left = x.N - col, rows = x.M - x.group_row(0);
                uint16_t *to = p.out + x.group_row(0) * p.ld + col;
                float *sum = p.sum + x.group_row(0) * p.lds + col;
                x.across(c, [&](int i, float(&v)[4]) {
                    if (i * 4 >= rows || left <= 0)
                        return;
                    if (!p.first) {
                        v[0] += pre.o[i].x;
                        v[1] += pre.o[i].y;
                        v[2] += pre.o[i].z;
                        v[3] += pre.o[i].w;
                    }
                    if (p.last) {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            v[k] *= pre.scale;
                        put4_16<true>(to + i * 4 * p.ld, v, left);
                    } else
                        *reinterpret_cast<float4 *>(sum + i * 4 * p.lds) = make_float4(v[0], v[1], v[2], v[3]);
                });
                read_sum(p, x, c + kParts, pre);
            }
        } else if (p.mapped) {
#pragma unroll 1
            for (int u = x.part; u < x.units(); u += kParts)
                x.emit_map<true>(maps.m, u, [&](int h, float(&v)[32]) {
                    x.load_sum(u * 2 + h, v);
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        v[i] *= pre.scale;
                });
        } else {
            const int row0 = x.row - x.lane;
#pragma unroll 1
            for (int u = x.part; u < x.units(); u += kParts)
                x.emit_rows<true>(
                    u,
                    [&](int h, float(&v)[32]) {
                        x.load_sum(u * 2 + h, v);
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            v[i] *= pre.scale;
                    },
                    [&](int r) {
                        return row0 + r < x.M ? p.out + (row0 + r) * p.ld + x.col + u * 64 : nullptr;
                    });
        }
    }
};

// The workspace of one call, and how the call is cut.
struct Plan {
    int64_t piece, pieces, lde, ldx, ldw, ldp;
    int stat_pieces, splits;
    int *meta, *source, *target;
    float *tlogit;
    float2 *stats;
    uint16_t *x, *w, *e;
    float *parts, *dw;
    int64_t bytes;
};


Plan plan_of(const LossArgs &a, bool grad, void *base, bool with_weight)
{
    Plan q{};
    q.lde = ceil_to(a.vocab, 64);  // whole lines
    q.stat_pieces = (int)((a.vocab + kPieceCols - 1) / kPieceCols);
    int64_t piece = a.piece_rows;
    if (piece <= 0) {
        // 2 GiB of what is kept of a piece's rows: the exponentials, or without gradients the statistics
        piece = (int64_t(1) << 31) / (grad ? 2 * q.lde : (int64_t)sizeof(float2) * q.stat_pieces);
        piece = piece / 256 * 256;
    }
    piece = ceil_to(piece < 1 ? 1 : piece, 64);
    q.piece = piece < a.rows ? piece : a.rows;
    q.pieces = a.rows ? (a.rows + q.piece - 1) / q.piece : 0;
    q.ldx = ceil_to(a.cols, 16);
    // dhidden sums over the vocabulary. Where its 256-row tiles are few, the
    // sum may be cut in parts (Tiles::choose_splits), which are then joined.
    const int64_t tiles = (q.piece + 255) / 256 * ((a.cols + 255) / 256);
    q.splits = tiles <= kSplitSms / 2 ? (int)((a.vocab + kBK - 1) / kBK / 4) : 1;
    if (q.splits < 1)
        q.splits = 1;
    q.ldp = ceil_to(a.cols, 8);

    Carver c(base);
    q.meta = c.take<int>(4);
    q.source = c.take<int>(a.rows);
    q.target = c.take<int>(a.rows);
    q.tlogit = c.take<float>(a.rows);
    q.x = c.take<uint16_t>(ceil_to(a.rows, 64) * q.ldx);
    q.stats = c.take<float2>(q.piece * q.stat_pieces);
    q.w = c.take<uint16_t>(with_weight ? a.vocab * q.ldx : 0);
    if (grad) {
        q.e = c.take<uint16_t>(ceil_to(q.piece, 64) * q.lde);
        if (q.splits > 1)
            q.parts = c.take<float>(parts_floats(q.ldp, q.splits, q.piece));
        if (q.pieces > 1)
            q.dw = c.take<float>(a.vocab * q.ldp);
    }
    q.bytes = c.used();
    return q;
}

}  // namespace

int64_t loss_workspace(const LossArgs &a, bool grad, bool aligned_weight)
{
    return plan_of(a, grad, nullptr, !aligned_weight).bytes;
}

fsdp_status launch_linear_cross_entropy(const LossArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool grad = a.dweight != nullptr;
    const int sms = device_sms(dev);
    const bool direct = loss_weight_aligned(a.weight, a.ldw);
    const Plan q = plan_of(a, grad, workspace, !direct);
    fsdp_status st;
    if (a.rows == 0) {
        cudaError_t err = cudaMemsetAsync(a.loss, 0, sizeof(float), s);
        if (err == cudaSuccess && grad)
            err = cudaMemset2DAsync(a.dweight, (size_t)a.lddw * 2, 0, (size_t)a.cols * 2, (size_t)a.vocab, s);
        return err == cudaSuccess ? FSDP_OK
                                  : set_error(FSDP_ECUDA, "linear_cross_entropy: %s", cudaGetErrorString(err));
    }

    PrepParams pp{};
    pp.rows = a.rows;
    pp.ldh = a.ldh;
    pp.lddh = a.lddh;
    pp.ldx = q.ldx;
    pp.cols = (int)a.cols;
    pp.vocab = (int)a.vocab;
    pp.hidden = static_cast<const uint16_t *>(a.hidden);
    pp.targets = a.targets;
    pp.ignore = a.ignore_index;
    pp.x = q.x;
    pp.source = q.source;
    pp.target = q.target;
    pp.meta = q.meta;
    pp.row_loss = a.row_loss;
    pp.dhidden = static_cast<uint16_t *>(a.dhidden);
    int64_t chunk = (a.rows + 4 * sms - 1) / (4 * sms);
    pp.chunk = (int)(chunk < 8 ? 8 : chunk);
    unsigned prep_grid = (unsigned)((a.rows + pp.chunk - 1) / pp.chunk);
    pp.packers = (int)prep_grid;
    const uint16_t *w = static_cast<const uint16_t *>(a.weight);
    int64_t ldw = a.ldw;
    if (!direct) {
        const int64_t blocks = (a.vocab + 7) / 8;
        prep_grid += (unsigned)(blocks < 8 * sms ? blocks : 8 * sms);
        pp.weight = w;
        pp.w = q.w;
        pp.ldw = ldw;
        w = q.w;
        ldw = q.ldx;
    }
    if ((st = launch("linear_cross_entropy (rows kept)", prep_kernel, prep_grid, 256, 0, s, 1, pp)) != FSDP_OK)
        return st;

    for (int64_t piece = 0; piece < q.pieces; piece++) {
        const int64_t row0 = piece * q.piece;
        const int rows = (int)(a.rows - row0 < q.piece ? a.rows - row0 : q.piece);
        const uint16_t *x = q.x + row0 * q.ldx;
        Shape sh{};
        sh.M = rows;
        sh.N = (int)a.vocab;
        sh.K = (int)a.cols;
        sh.batch = 1;
        sh.epi_bytes = 5;  // 2 of each element, and the time of its exponential
        sh.dyn = q.meta;
        sh.dyn_base = (int)row0;
        const Operand ox{x, a.cols, ceil_to(rows, 64), q.ldx, 0};
        const Operand ow{w, a.cols, a.vocab, ldw, 0};
        const Operand oe{q.e, q.lde, ceil_to(rows, 64), q.lde, 0};
        const LogitsParams le{grad, q.stats, q.stat_pieces, q.target + row0, q.tlogit + row0};
        const char *what = "linear_cross_entropy (logits)";
        const Operand *out = grad ? &oe : nullptr;
        st = a.cols > kLongCols ? product<false, false, LogitsEpi<true>>(sh, ox, ow, true, le, dev, s, what, out)
                                : product<false, false, LogitsEpi<false>>(sh, ox, ow, true, le, dev, s, what, out);
        if (st != FSDP_OK)
            return st;

        RowsParams rp{};
        rp.meta = q.meta;
        rp.base = (int)row0;
        rp.piece_rows = rows;
        rp.vocab = (int)a.vocab;
        rp.pieces = q.stat_pieces;
        rp.lde = q.lde;
        rp.e = q.e;
        rp.stats = q.stats;
        rp.source = q.source + row0;
        rp.target = q.target + row0;
        rp.rows = a.rows;
        rp.loss = piece + 1 == q.pieces ? a.loss : nullptr;
        rp.done = q.meta + 2;
        rp.tlogit = q.tlogit + row0;
        rp.row_loss = a.row_loss;
        rp.mean = a.mean;
        const int64_t rows_grid = ceil_to(rows, 64) < 8 * sms ? ceil_to(rows, 64) : 8 * sms;
        int64_t segments = grad ? 8 * sms / rows_grid : 1;
        if (segments > (a.vocab + 4095) / 4096)
            segments = (a.vocab + 4095) / 4096;
        if (segments < 1)
            segments = 1;
        rp.segment = (int)ceil_to((a.vocab + segments - 1) / segments, 8);
        if ((st = launch("linear_cross_entropy (rows)", rows_kernel, dim3((unsigned)rows_grid, (unsigned)segments), 256,
                         0, s, 1, rp)) != FSDP_OK)
            return st;
        if (!grad)
            continue;

        // dhidden = G weight: K = vocab, adjacent in G; weight has its columns adjacent
        const Operand og{q.e, a.vocab, ceil_to(rows, 64), q.lde, 0};
        const Operand owt{w, a.cols, a.vocab, ldw, 0};
        Shape sd{};
        sd.M = rows;
        sd.N = (int)a.cols;
        sd.K = (int)a.vocab;
        sd.batch = 1;
        sd.epi_bytes = 3;
        sd.dyn = q.meta;
        sd.dyn_base = (int)row0;
        sd.splits = q.splits;
        sd.splits_out = q.meta + 3;
        uint16_t *dh = static_cast<uint16_t *>(a.dhidden);
        const Scale scale{q.meta, a.grad_scale, a.mean};
        if (q.splits > 1) {
            st = product<false, true, PartEpi>(sd, og, owt, true, {q.parts, q.ldp}, dev, s,
                                                          "linear_cross_entropy (dhidden)");
            if (st != FSDP_OK)
                return st;
            st = launch("linear_cross_entropy (dhidden, sum)", join_hidden_kernel,
                        dim3((unsigned)(rows < 16 * sms ? rows : 16 * sms), (unsigned)((a.cols + 255) / 256)), 256, 0,
                        s, 1, q.parts, q.ldp, q.meta, row0, rows, a.cols, q.source + row0, dh, a.lddh, scale);
        } else {
            st = product<false, true, HiddenEpi>(sd, og, owt, true, {dh, a.lddh, q.source + row0, scale}, dev, s,
                                                            "linear_cross_entropy (dhidden)");
        }
        if (st != FSDP_OK)
            return st;

        // dweight = G^T hidden: K = rows, adjacent in neither
        const Operand ogt{q.e, a.vocab, ceil_to(rows, 64), q.lde, 0};
        const Operand oxt{x, a.cols, ceil_to(rows, 64), q.ldx, 0};
        Shape sw{};
        sw.M = (int)a.vocab;
        sw.N = (int)a.cols;
        sw.K = rows;
        sw.batch = 1;
        sw.epi_bytes = 3;
        sw.dyn = q.meta;
        sw.dyn_base = (int)row0;
        sw.dyn_is_k = 1;
        const bool mapped = !q.dw && (reinterpret_cast<uintptr_t>(a.dweight) & 15u) == 0 && a.lddw % 8 == 0;
        const Operand odw{a.dweight, a.cols, a.vocab, a.lddw, 0};
        const WeightEpi::Params we{static_cast<uint16_t *>(a.dweight), a.lddw, q.dw, q.ldp, piece == 0,
                                   piece + 1 == q.pieces, mapped, scale};
        if ((st = product<true, true, WeightEpi>(sw, ogt, oxt, true, we, dev, s, "linear_cross_entropy (dweight)",
                                                 mapped ? &odw : nullptr)) != FSDP_OK)
            return st;
    }
    return FSDP_OK;
}

cudaError_t loss_wait_timeouts(unsigned long long *n) { return wait::wait_timeouts(n); }

}  // namespace fsdp
