// fsdp_norm.cu -- layer norm, forward and backward, for sm_103a.
//
// Both passes are bound by HBM: 8 (forward) or 14 (backward) flops per
// element that is read or written once. TPR threads hold one row in
// registers, as the 16-byte chunks it was loaded in, so x (and dy) is read
// once whatever the statistics need; rows past the widest such shape are
// walked again instead, from L2. A row's mean and its sum of squares about
// the mean are formed per warp, in two steps over the registers, and the
// warps' joined by their counts: fp32 precision under a large mean, where
// sum(x^2) - mean^2 would lose it.
//
// 16384 x 4096 bf16: forward 50.4 us, 5.3 TB/s (0.79 of a plain copy's rate);
// backward 77.3 us, 5.2 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fsdp_launch.cuh"
#include "fsdp_wait.cuh"

namespace fsdp {
namespace {

using namespace wait;

constexpr int kWide = 1024;      // threads of the kernels for the widest rows
constexpr int kMinThreads = 128;  // forward: narrow rows share a block of this size
constexpr int kBackThreads = 256; // backward: likewise

__device__ __forceinline__ float to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(uint16_t &d, float f) { d = __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ void from_f32(float &d, float f) { d = f; }
__device__ __forceinline__ uint32_t bits_of(uint16_t h) { return h; }
__device__ __forceinline__ uint32_t bits_of(float f) { return __float_as_uint(f); }

// Two fp32 numbers that one instruction works on (add, mul, fma .f32x2), in
// the backward pass (16384 x 4096 bf16: 91.7 -> 88.7 us; the forward pass got
// slower with them, 48.7 -> 53.4 us).
struct Pair {
    uint64_t bits;
    Pair() = default;
    __device__ __forceinline__ Pair(float lo, float hi)
    {
        asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(lo), "f"(hi));
    }
    __device__ __forceinline__ explicit Pair(float both) : Pair(both, both) {}
    __device__ __forceinline__ void get(float &lo, float &hi) const
    {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(bits));
    }
    __device__ __forceinline__ float sum() const
    {
        float lo, hi;
        get(lo, hi);
        return lo + hi;
    }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits));
    return d;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b)
{
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
    return d;
}

// A chunk: V elements of a row, as 16 bytes of registers.
template <typename T>
struct Chunk {
    static constexpr int V = 16 / (int)sizeof(T);
    uint4 raw;
    __device__ __forceinline__ void values(float (&v)[V]) const
    {
        const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int i = 0; i < V; i++)
            v[i] = to_f32(e[i]);
    }
    __device__ __forceinline__ void pairs(Pair (&v)[V / 2]) const
    {
        float f[V];
        values(f);
#pragma unroll
        for (int i = 0; i < V / 2; i++)
            v[i] = Pair(f[2 * i], f[2 * i + 1]);
    }
    // Between two uses: keeps the compiler from holding the widened values,
    // twice the registers, from one to the other.
    __device__ __forceinline__ void keep_packed()
    {
        asm volatile("" : "+r"(raw.x), "+r"(raw.y), "+r"(raw.z), "+r"(raw.w));
    }
};

// Streamed rows stay out of L1, where gamma and beta are kept.
__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}

// kFull: rows are whole chunks, and every row, gamma and beta start on 16
// bytes; nothing but vector accesses is compiled then (with the others beside
// them, unrolled, the kernels outgrow the instruction cache).
//
// The column of element i of chunk q of thread t of a row's TPR. Where the
// elements go one by one, a warp's lie side by side (16384 x 4095 bf16: 76 us
// forward and 105 backward; with a thread's side by side 167 and 236).
template <bool kFull, int TPR, int V>
__device__ __forceinline__ int column(int q, int t, int i)
{
    return kFull ? (q * TPR + t) * V + i : (q * V + i) * TPR + t;
}

template <typename T, bool kFull, int TPR>
__device__ __forceinline__ void load_chunk(Chunk<T> &c, const T *row, int q, int t, int cols)
{
    constexpr int V = Chunk<T>::V;
    if (kFull) {
        const int col = column<kFull, TPR, V>(q, t, 0);
        c.raw = col < cols ? load_stream(row + col) : make_uint4(0, 0, 0, 0);
    } else {
        T e[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int col = column<kFull, TPR, V>(q, t, i);
            e[i] = col < cols ? row[col] : T(0);
        }
        uint32_t *w = reinterpret_cast<uint32_t *>(&c.raw);
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = sizeof(T) == 4 ? bits_of(e[i]) : bits_of(e[2 * i % V]) | bits_of(e[(2 * i + 1) % V]) << 16;
    }
}

template <typename T, bool kFull, int TPR>
__device__ __forceinline__ void store_chunk(T *row, int q, int t, int cols, const float (&v)[Chunk<T>::V])
{
    constexpr int V = Chunk<T>::V;
    if (kFull) {
        const int col = column<kFull, TPR, V>(q, t, 0);
        uint4 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int i = 0; i < V; i++)
            from_f32(e[i], v[i]);
        __stcs(reinterpret_cast<uint4 *>(row + col), u);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int col = column<kFull, TPR, V>(q, t, i);
            if (col < cols)
                from_f32(row[col], v[i]);
        }
    }
}

// gamma or beta of a chunk's columns, of either type; zeros past the row.
template <int V, bool kFull, int TPR>
__device__ __forceinline__ void load_param(const void *p, bool bf16, int q, int t, int cols, float (&v)[V])
{
    if (kFull) {
        const int col = column<kFull, TPR, V>(q, t, 0);
        // volatile, "memory": neither hoisted out of the rows' loop into
        // registers nor gathered ahead of the stores before it
        if (bf16) {
            const uint16_t *from = static_cast<const uint16_t *>(p) + col;
            uint32_t u[V / 2];
            if (V == 8)
                asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(u[0]), "=r"(u[1]), "=r"(u[V / 2 - 2]), "=r"(u[V / 2 - 1])
                             : "l"(from)
                             : "memory");
            else
                asm volatile("ld.global.nc.v2.b32 {%0,%1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "l"(from) : "memory");
#pragma unroll
            for (int i = 0; i < V / 2; i++) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        } else {
            const float *from = static_cast<const float *>(p) + col;
#pragma unroll
            for (int i = 0; i < V; i += 4)
                asm volatile("ld.global.nc.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
                             : "l"(from + i)
                             : "memory");
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int col = column<kFull, TPR, V>(q, t, i);
            v[i] = col >= cols ? 0.0f
                   : bf16      ? to_f32(static_cast<const uint16_t *>(p)[col])
                               : static_cast<const float *>(p)[col];
        }
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct ForwardParams {
    int64_t rows, ldx, ldy;
    int cols;
    const void *x, *gamma, *beta;
    void *y;
    float *mean, *rstd;
    float eps;
    int param_bf16;
};

template <int TPR>
constexpr int forward_block()
{
    return TPR < kMinThreads ? kMinThreads : TPR;
}

// NV chunks per thread, at most 4: a row of 4096 bf16 is 128 threads', and a
// multiprocessor has about ten such rows under way. (One warp per row with
// 16 chunks a thread needs no barrier, but its unrolled code missed the
// instruction cache: 16384 x 4096 bf16 took 132 us.)
template <typename T, bool kFull, int TPR, int NV>
__global__ void __launch_bounds__(forward_block<TPR>(),
                                  NV > 4 ? 1 : 1024 / forward_block<TPR>())
    norm_forward_kernel(const ForwardParams p)
{
    constexpr int kRowsPerBlock = forward_block<TPR>() / TPR, kWarps = TPR / 32, V = Chunk<T>::V;
    __shared__ float4 sh[2][32];
    launch_wait();
    launch_next();
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int warp = threadIdx.x / 32, warp0 = warp / kWarps * kWarps;
    // this warp's number of elements, the same in every row
    float mine = 0.0f;
#pragma unroll
    for (int q = 0; q < NV; q++)
#pragma unroll
        for (int i = 0; i < V; i++)
            mine += column<kFull, TPR, V>(q, t, i) < p.cols ? 1.0f : 0.0f;
    const float count = warp_sum(mine);
    const float inv_count = count > 0.0f ? 1.0f / count : 0.0f, inv_cols = 1.0f / (float)p.cols;
    int phase = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kRowsPerBlock; r0 < p.rows;
         r0 += (int64_t)gridDim.x * kRowsPerBlock, phase ^= 1) {
        const int64_t r = r0 + sub;
        // rows of one block meet no barrier of each other's unless a row is
        // several warps', and then the last rows' places are worked on as row
        // rows - 1, and not stored
        const bool live = r < p.rows;
        if (kWarps == 1 && !live)
            break;
        const T *x = static_cast<const T *>(p.x) + (live ? r : p.rows - 1) * p.ldx;
        Chunk<T> c[NV];
#pragma unroll
        for (int q = 0; q < NV; q++)
            load_chunk<T, kFull, TPR>(c[q], x, q, t, p.cols);
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < NV; q++) {
            float v[V];
            c[q].values(v);
#pragma unroll
            for (int i = 0; i < V; i++)
                s += v[i];
        }
        float mean = warp_sum(s) * inv_count, m2 = 0.0f;
#pragma unroll
        for (int q = 0; q < NV; q++) {
            c[q].keep_packed();
            float v[V];
            c[q].values(v);
            if (column<kFull, TPR, V>(q, t, V - 1) < p.cols) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    m2 += (v[i] - mean) * (v[i] - mean);
            } else if (!kFull) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    if (column<kFull, TPR, V>(q, t, i) < p.cols)
                        m2 += (v[i] - mean) * (v[i] - mean);
            }
        }
        m2 = warp_sum(m2);
        if (kWarps > 1) {
            if (threadIdx.x % 32 == 0)
                sh[phase][warp] = make_float4(mean, m2, count, 0.0f);
            __syncthreads();
            if (kWarps <= 4) {
                mean = m2 = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; w++)
                    mean += sh[phase][warp0 + w].x * sh[phase][warp0 + w].z;
                mean *= inv_cols;
#pragma unroll
                for (int w = 0; w < kWarps; w++) {
                    const float4 f = sh[phase][warp0 + w];
                    m2 += f.y + f.z * (f.x - mean) * (f.x - mean);
                }
            } else {  // a lane per warp of the row
                const int w = threadIdx.x % 32;
                const float4 f = w < kWarps ? sh[phase][warp0 + w] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                mean = warp_sum(f.x * f.z) * inv_cols;
                m2 = warp_sum(f.y + f.z * (f.x - mean) * (f.x - mean));
            }
        }
        const float rstd = 1.0f / sqrtf(m2 * inv_cols + p.eps);
        if (!live)
            continue;
        if (t == 0 && p.mean) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        T *y = static_cast<T *>(p.y) + r * p.ldy;
#pragma unroll
        for (int q = 0; q < NV; q++) {
            if (column<kFull, TPR, V>(q, t, 0) >= p.cols)
                break;
            float v[V], g[V], b[V];
            c[q].keep_packed();
            c[q].values(v);
            load_param<V, kFull, TPR>(p.gamma, p.param_bf16, q, t, p.cols, g);
#pragma unroll
            for (int i = 0; i < V; i++)
                b[i] = 0.0f;
            if (p.beta)
                load_param<V, kFull, TPR>(p.beta, p.param_bf16, q, t, p.cols, b);
#pragma unroll
            for (int i = 0; i < V; i++)
                v[i] = fmaf((v[i] - mean) * rstd, g[i], b[i]);
            store_chunk<T, kFull, TPR>(y, q, t, p.cols, v);
        }
    }
}

struct BackwardParams {
    int64_t rows, lddy, ldx, lddx;
    int cols;
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    void *dx;
    float *partial;  // [2][gridDim.x][cols]: sums of dy*xhat and of dy
    int param_bf16;
    int stages;      // of the staged form
};

template <int TPR>
constexpr int backward_block()
{
    return TPR < kBackThreads ? kBackThreads : TPR;
}

// 1-D bulk copy of one row into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(saddr(dst)),
        "l"(src), "r"(bytes), "r"(saddr(bar))
        : "memory");
}

// dgamma and dbeta: every thread sums its columns over the block's rows in
// registers; the rows that share a block then join in shared memory, and the
// block's sums go to its own line of `partial`, which norm_columns_kernel
// adds up in order.
//
// Staged (kStaged, for rows of whole chunks): a block's rows of x and dy come
// into a ring of `stages` shared-memory stages by bulk copies, so that loads
// are under way while a row waits for its sums. The one barrier per row, that
// of the sums, comes after every thread has read its chunks: behind it the
// stage is free and is filled again. Registers alone held too little: 16384 x
// 4096 bf16 took 107 us.
//
// bf16 rows are bound by instructions as much as by HBM. Two elements share
// each fp32 one (Pair), and xhat and dy gamma stay in registers for dx. x - mean
// and dy gamma - mean(dy gamma) are formed first, as one multiply-add less would
// not: a row of one value, or of one column, has xhat = 0 and dx = 0, where
// x rstd - mean rstd leaves a rounding times rstd, up to 1 / sqrt(eps).
template <typename T, bool kFull, bool kStaged, int TPR, int NV>
__global__ void __launch_bounds__(backward_block<TPR>(), backward_block<TPR>() > 256 ? 1 : 2)
    norm_backward_kernel(const BackwardParams p)
{
    constexpr int kSub = backward_block<TPR>() / TPR, kWarps = TPR / 32, V = Chunk<T>::V;
    __shared__ float2 sh[2][32];
    __shared__ uint64_t bars[8];
    extern __shared__ __align__(128) unsigned char dyn[];  // the ring, then the joining of the rows' sums
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int warp = threadIdx.x / 32, warp0 = warp / kWarps * kWarps;
    const uint32_t row_bytes = (uint32_t)p.cols * sizeof(T);
    const int64_t step = (int64_t)gridDim.x * kSub;
    const int64_t first = (int64_t)blockIdx.x * kSub;

    auto fill = [&](int stage, int64_t r0) {
        // thread 0: the rows r0 .. r0 + kSub of x, then of dy
        const int64_t left = p.rows - r0;
        const int n = left < kSub ? (int)left : kSub;
        bar_expect(bars + stage, 2 * n * row_bytes);
        unsigned char *d = dyn + (size_t)stage * 2 * kSub * row_bytes;
        for (int i = 0; i < n; i++) {
            bulk_load(d + i * row_bytes, static_cast<const T *>(p.x) + (r0 + i) * p.ldx, row_bytes, bars + stage);
            bulk_load(d + (kSub + i) * row_bytes, static_cast<const T *>(p.dy) + (r0 + i) * p.lddy, row_bytes,
                      bars + stage);
        }
    };
    launch_wait();
    launch_next();
    if (kStaged) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < p.stages; i++)
                bar_init(bars + i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            for (int i = 0; i < p.stages && first + i * step < p.rows; i++)
                fill(i, first + i * step);
        }
        __syncthreads();
    }
    Pair gamma[NV][V / 2], dg[NV][V / 2], db[NV][V / 2];
#pragma unroll
    for (int q = 0; q < NV; q++) {
        float g[V];
#pragma unroll
        for (int i = 0; i < V; i++)
            g[i] = 0.0f;
        if (column<kFull, TPR, V>(q, t, 0) < p.cols)
            load_param<V, kFull, TPR>(p.gamma, p.param_bf16, q, t, p.cols, g);
#pragma unroll
        for (int i = 0; i < V / 2; i++) {
            gamma[q][i] = Pair(g[2 * i], g[2 * i + 1]);
            dg[q][i] = db[q][i] = Pair(0.0f);
        }
    }
    const float inv = 1.0f / (float)p.cols;
    int phase = 0, stage = 0;
    uint32_t parity = 0;
    float next_mean = 0.0f, next_rstd = 0.0f;  // read a row ahead
    if (first + sub < p.rows) {
        next_mean = p.mean[first + sub];
        next_rstd = p.rstd[first + sub];
    }
    for (int64_t r0 = first; r0 < p.rows; r0 += step, phase ^= 1) {
        const int64_t r = r0 + sub;
        const bool live = r < p.rows;
        Chunk<T> cx[NV], cy[NV];
        const float mean = next_mean, rstd = next_rstd;
        next_mean = next_rstd = 0.0f;
        if (r + step < p.rows) {
            next_mean = p.mean[r + step];
            next_rstd = p.rstd[r + step];
        }
        bool ok = true;
        if (kStaged) {
            ok = bar_wait(bars + stage, parity);
            const unsigned char *d = dyn + (size_t)stage * 2 * kSub * row_bytes + sub * row_bytes;
#pragma unroll
            for (int q = 0; q < NV; q++) {
                const uint32_t at = (uint32_t)(q * TPR + t) * 16;
                const bool in = live && at < row_bytes;
                cx[q].raw = in ? *reinterpret_cast<const uint4 *>(d + at) : make_uint4(0, 0, 0, 0);
                cy[q].raw = in ? *reinterpret_cast<const uint4 *>(d + kSub * row_bytes + at) : make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int q = 0; q < NV; q++) {
                cx[q].raw = cy[q].raw = make_uint4(0, 0, 0, 0);
                if (live) {
                    load_chunk<T, kFull, TPR>(cx[q], static_cast<const T *>(p.x) + r * p.ldx, q, t, p.cols);
                    load_chunk<T, kFull, TPR>(cy[q], static_cast<const T *>(p.dy) + r * p.lddy, q, t, p.cols);
                }
            }
        }
        // xhat and dy gamma of a chunk; past the row's end dy and gamma are 0,
        // and so is all that xhat enters
        const Pair scale(rstd), shift(-mean);
        auto widen = [&](int q, Pair(&xhat)[V / 2], Pair(&gg)[V / 2], Pair(&g)[V / 2]) {
            cx[q].pairs(xhat);
            cy[q].pairs(g);
#pragma unroll
            for (int i = 0; i < V / 2; i++) {
                xhat[i] = (xhat[i] + shift) * scale;
                gg[i] = g[i] * gamma[q][i];
            }
        };
        constexpr bool kHold = NV * V <= 16;  // registers
        Pair held_x[kHold ? NV : 1][V / 2], held_g[kHold ? NV : 1][V / 2];
        Pair sa(0.0f), sb(0.0f);
#pragma unroll
        for (int q = 0; q < NV; q++) {
            Pair g[V / 2];
            Pair(&xhat)[V / 2] = held_x[kHold ? q : 0];
            Pair(&gg)[V / 2] = held_g[kHold ? q : 0];
            widen(q, xhat, gg, g);
#pragma unroll
            for (int i = 0; i < V / 2; i++) {
                dg[q][i] = fma2(g[i], xhat[i], dg[q][i]);
                db[q][i] = db[q][i] + g[i];
                sa = sa + gg[i];
                sb = fma2(gg[i], xhat[i], sb);
            }
        }
        float a = warp_sum(sa.sum()), b = warp_sum(sb.sum());
        if (kWarps > 1 && threadIdx.x % 32 == 0)
            sh[phase][warp] = make_float2(a, b);
        if (kStaged) {
            if (!__syncthreads_and(ok)) {
                if (threadIdx.x == 0) {
                    atomicAdd(&g_wait_timeouts, 1ull);
                    let_copies_land();
                }
                __syncthreads();
                return;
            }
            if (threadIdx.x == 0 && r0 + p.stages * step < p.rows)
                fill(stage, r0 + p.stages * step);
            if (++stage == p.stages) {
                stage = 0;
                parity ^= 1;
            }
        } else if (kWarps > 1) {
            __syncthreads();
        }
        if (kWarps > 1) {
            a = b = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float2 f = sh[phase][warp0 + w];
                a += f.x;
                b += f.y;
            }
        }
        if (!live)
            continue;
        // dx = rstd (dy gamma - mean(dy gamma) - xhat mean(dy gamma xhat))
        const Pair ca(-a * inv), cb(-b * inv);
        T *dx = static_cast<T *>(p.dx) + r * p.lddx;
#pragma unroll
        for (int q = 0; q < NV; q++) {
            if (column<kFull, TPR, V>(q, t, 0) >= p.cols)
                break;
            float out[V];
            Pair(&xhat)[V / 2] = held_x[kHold ? q : 0];
            Pair(&gg)[V / 2] = held_g[kHold ? q : 0];
            if (!kHold) {
                Pair g[V / 2];
                cx[q].keep_packed();
                cy[q].keep_packed();
                widen(q, xhat, gg, g);
            }
#pragma unroll
            for (int i = 0; i < V / 2; i++)
                (fma2(xhat[i], cb, gg[i] + ca) * scale).get(out[2 * i], out[2 * i + 1]);
            store_chunk<T, kFull, TPR>(dx, q, t, p.cols, out);
        }
    }
    float *pg = p.partial + (int64_t)blockIdx.x * p.cols;
    float *pb = pg + (int64_t)gridDim.x * p.cols;
    if (kSub == 1) {
#pragma unroll
        for (int q = 0; q < NV; q++)
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const int c = column<kFull, TPR, V>(q, t, i), c1 = column<kFull, TPR, V>(q, t, i + 1);
                float g0, g1, b0, b1;
                dg[q][i / 2].get(g0, g1);
                db[q][i / 2].get(b0, b1);
                if (c < p.cols)
                    pg[c] = g0, pb[c] = b0;
                if (c1 < p.cols)
                    pg[c1] = g1, pb[c1] = b1;
            }
    } else {
        // every copy has landed and been read; [kSub][TPR * NV * V] fp32
        float *col = reinterpret_cast<float *>(dyn);
        constexpr int kLine = TPR * NV * V;
        for (int which = 0; which < 2; which++) {
            __syncthreads();
#pragma unroll
            for (int q = 0; q < NV; q++)
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    float lo, hi;
                    (which ? db[q][i / 2] : dg[q][i / 2]).get(lo, hi);
                    float *at = col + sub * kLine + column<kFull, TPR, V>(q, t, i);
                    if (kFull) {
                        *reinterpret_cast<float2 *>(at) = make_float2(lo, hi);
                    } else {
                        at[0] = lo;
                        at[TPR] = hi;
                    }
                }
            __syncthreads();
            for (int c = threadIdx.x; c < p.cols; c += backward_block<TPR>()) {
                float s = 0.0f;
                for (int q = 0; q < kSub; q++)
                    s += col[q * kLine + c];
                (which ? pb : pg)[c] = s;
            }
        }
    }
}

// The widest rows: one block per row, which walks it once for the sum, once
// for the squares and once for the result.
__device__ __forceinline__ float block_sum(float v, float *sh)
{
    v = warp_sum(v);
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < kWide / 32; i++)
        v += sh[i];
    __syncthreads();
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kWide, 1) norm_forward_wide_kernel(const ForwardParams p)
{
    __shared__ float sh[kWide / 32];
    launch_wait();
    launch_next();
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        T *y = static_cast<T *>(p.y) + r * p.ldy;
        float s = 0.0f;
        for (int c = threadIdx.x; c < p.cols; c += kWide)
            s += to_f32(x[c]);
        const float mean = block_sum(s, sh) / (float)p.cols;
        s = 0.0f;
        for (int c = threadIdx.x; c < p.cols; c += kWide) {
            const float d = to_f32(x[c]) - mean;
            s += d * d;
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, sh) / (float)p.cols + p.eps);
        if (threadIdx.x == 0 && p.mean) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        for (int c = threadIdx.x; c < p.cols; c += kWide) {
            const float ga = p.param_bf16 ? to_f32(static_cast<const uint16_t *>(p.gamma)[c])
                                          : static_cast<const float *>(p.gamma)[c];
            const float be = !p.beta        ? 0.0f
                             : p.param_bf16 ? to_f32(static_cast<const uint16_t *>(p.beta)[c])
                                            : static_cast<const float *>(p.beta)[c];
            from_f32(y[c], (to_f32(x[c]) - mean) * rstd * ga + be);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kWide, 1) norm_backward_wide_kernel(const BackwardParams p)
{
    __shared__ float sh[kWide / 32];
    launch_wait();
    launch_next();
    float *pg = p.partial + (int64_t)blockIdx.x * p.cols;
    float *pb = pg + (int64_t)gridDim.x * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += kWide)
        pg[c] = pb[c] = 0.0f;  // each column is one thread's throughout
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        const T *dy = static_cast<const T *>(p.dy) + r * p.lddy;
        T *dx = static_cast<T *>(p.dx) + r * p.lddx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float a = 0.0f, b = 0.0f;
        for (int c = threadIdx.x; c < p.cols; c += kWide) {
            const float xh = (to_f32(x[c]) - mean) * rstd, d = to_f32(dy[c]);
            const float ga = p.param_bf16 ? to_f32(static_cast<const uint16_t *>(p.gamma)[c])
                                          : static_cast<const float *>(p.gamma)[c];
            pg[c] += d * xh;
            pb[c] += d;
            a += d * ga;
            b += d * ga * xh;
        }
        a = block_sum(a, sh) / (float)p.cols;
        b = block_sum(b, sh) / (float)p.cols;
        for (int c = threadIdx.x; c < p.cols; c += kWide) {
            const float xh = (to_f32(x[c]) - mean) * rstd, d = to_f32(dy[c]);
            const float ga = p.param_bf16 ? to_f32(static_cast<const uint16_t *>(p.gamma)[c])
                                          : static_cast<const float *>(p.gamma)[c];
            from_f32(dx[c], rstd * (d * ga - a - xh * b));
        }
    }
}

// dgamma, dbeta: the parts' sums, added in a fixed order. A block has 32
// columns and 32 slices of the parts.
__global__ void __launch_bounds__(1024) norm_columns_kernel(const float *partial, int parts, int cols, void *dgamma,
                                                            void *dbeta, int param_bf16)
{
    __shared__ float sh[32][33];
    launch_wait();
    launch_next();
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane;
    void *out = blockIdx.y ? dbeta : dgamma;
    const float *src = partial + (int64_t)blockIdx.y * parts * cols + c;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int q = slice; q < parts; q += 32)
            s += src[(int64_t)q * cols];
    }
    sh[slice][lane] = s;
    __syncthreads();
    // warp w sums column w's slices
    s = warp_sum(sh[lane][slice]);
    const int w = blockIdx.x * 32 + slice;
    if (lane == 0 && w < cols) {
        if (param_bf16)
            from_f32(static_cast<uint16_t *>(out)[w], s);
        else
            static_cast<float *>(out)[w] = s;
    }
}

bool vec_ok(const void *p, int64_t ld, int64_t size)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
}

// The shape of a kernel: threads per row and chunks per thread. Calls
// f.template run<T, kFull, TPR, NV>(); false if no shape holds the row.
template <typename T, bool kFull, class F>
bool forward_shape(int64_t rows, int64_t cols, int sms, F f)
{
    const int64_t chunks = (cols + Chunk<T>::V - 1) / Chunk<T>::V;
    // 4 chunks a thread where the rows fill the multiprocessors; with few rows
    // their latency counts, and a thread has one chunk.
    const bool many = rows >= 4 * sms;
    if (chunks <= 32)
        f.template run<T, kFull, 32, 1>();
    else if (chunks <= 32 * 4 && many)
        f.template run<T, kFull, 32, 4>();
    else if (chunks <= 128)
        f.template run<T, kFull, 128, 1>();
    else if (chunks <= 128 * 4 && many)
        f.template run<T, kFull, 128, 4>();
    else if (chunks <= 256 * 4 && many)
        f.template run<T, kFull, 256, 4>();
    else if (chunks <= 512)
        f.template run<T, kFull, 512, 1>();
    else if (chunks <= 512 * 4)
        f.template run<T, kFull, 512, 4>();
    else if (chunks <= 512 * 8)
        f.template run<T, kFull, 512, 8>();
    else
        return false;
    return true;
}

// The backward pass keeps 3 fp32 numbers per column and thread: 16 columns a
// thread, 32 where the block would be larger than 512 threads. Returns the
// rows that a block takes at a time, 0 if no shape holds the row.
template <typename T, bool kFull, class F>
int backward_shape(int64_t cols, F f)
{
    constexpr int NV = sizeof(T) == 2 ? 2 : 4;
    if (cols <= 32 * 16)
        return f.template run<T, kFull, 32, NV>(), 8;
    if (cols <= 64 * 16)
        return f.template run<T, kFull, 64, NV>(), 4;
    if (cols <= 128 * 16)
        return f.template run<T, kFull, 128, NV>(), 2;
    if (cols <= 256 * 16)
        return f.template run<T, kFull, 256, NV>(), 1;
    if (cols <= 512 * 16)
        return f.template run<T, kFull, 512, NV>(), 1;
    if (cols <= 512 * 32)
        return f.template run<T, kFull, 512, 2 * NV>(), 1;
    return 0;
}

struct Forward {
    const ForwardParams &p;
    int sms;
    cudaStream_t s;
    fsdp_status *st;
    template <typename T, bool kFull, int TPR, int NV>
    void run()
    {
        constexpr int kBlock = forward_block<TPR>(), kRows = kBlock / TPR;
        const int64_t blocks = (p.rows + kRows - 1) / kRows, most = (int64_t)sms * (2048 / kBlock);
        *st = launch("layer_norm", norm_forward_kernel<T, kFull, TPR, NV>, (unsigned)(blocks < most ? blocks : most),
                     kBlock, 0, s, 1, p);
    }
};

// Shared memory of a block's stages: two blocks of 256 threads share a
// multiprocessor, one of 512 has it alone.
constexpr int kStageBudget = 96 * 1024;
constexpr int kMaxStages = 6;

struct Backward {
    BackwardParams &p;
    int parts;
    cudaStream_t s;
    fsdp_status *st;
    template <typename T, bool kFull, int TPR, int NV>
    void run()
    {
        constexpr int kBlock = backward_block<TPR>(), kSub = kBlock / TPR;
        constexpr int kJoin = kSub > 1 ? kSub * TPR * NV * Chunk<T>::V * 4 : 0;
        constexpr int kBudget = kBlock > kBackThreads ? 192 * 1024 : kStageBudget;
        const int stage = 2 * kSub * p.cols * (int)sizeof(T);
        p.stages = kBudget / stage < kMaxStages ? kBudget / stage : kMaxStages;
        if (kFull && p.stages >= 2) {
            auto kernel = norm_backward_kernel<T, kFull, kFull, TPR, NV>;
            const int smem = p.stages * stage > kJoin ? p.stages * stage : kJoin;
            if (smem > 48 * 1024) {
                const cudaError_t err =
                    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBudget);
                if (err != cudaSuccess) {
                    *st = set_error(FSDP_ECUDA, "layer_norm_backward: cudaFuncSetAttribute: %s", cudaGetErrorString(err));
                    return;
                }
            }
            *st = launch("layer_norm_backward", kernel, parts, kBlock, smem, s, 1, p);
        } else {
            *st = launch("layer_norm_backward", norm_backward_kernel<T, kFull, false, TPR, NV>, parts, kBlock, kJoin, s,
                         1, p);
        }
    }
};
struct Nothing {
    template <typename T, bool kFull, int TPR, int NV>
    void run()
    {
    }
};

// Blocks of the backward pass, each with a line of partial sums: two per
// multiprocessor of a GB300, fewer where there are not so many rows.
int64_t backward_parts(int64_t rows, int64_t cols)
{
    const int per = backward_shape<float, true>(cols, Nothing{});
    const int64_t blocks = per ? (rows + per - 1) / per : rows;
    const int64_t most = 152 * 2;
    return blocks < 1 ? 1 : blocks < most ? blocks : most;
}

}  // namespace

int64_t norm_backward_workspace(int64_t rows, int64_t cols)
{
    return 2 * backward_parts(rows, cols) * cols * (int64_t)sizeof(float);
}

fsdp_status launch_layer_norm(const NormArgs &a, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = a.dtype == FSDP_BF16;
    const int64_t size = bf16 ? 2 : 4;
    ForwardParams p{a.rows, a.ldx,  a.ldy,  (int)a.cols, a.x, a.gamma, a.beta, a.y, a.mean, a.rstd, a.eps,
                    a.param_dtype == FSDP_BF16};
    const int sms = device_sms(dev);
    fsdp_status st = FSDP_OK;
    const Forward f{p, sms, s, &st};
    const bool full = vec_ok(a.x, a.ldx, size) && vec_ok(a.y, a.ldy, size) && vec_ok(a.gamma, a.cols, size) &&
                      vec_ok(a.beta, 0, 1);
    const bool held = bf16 ? (full ? forward_shape<uint16_t, true>(a.rows, a.cols, sms, f)
                                   : forward_shape<uint16_t, false>(a.rows, a.cols, sms, f))
                           : (full ? forward_shape<float, true>(a.rows, a.cols, sms, f)
                                   : forward_shape<float, false>(a.rows, a.cols, sms, f));
    if (!held) {
        const unsigned grid = (unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms);
        st = launch("layer_norm", bf16 ? norm_forward_wide_kernel<uint16_t> : norm_forward_wide_kernel<float>, grid, kWide,
                    0, s, 1, p);
    }
    return st;
}

fsdp_status launch_layer_norm_backward(const NormArgs &a, int dev, void *stream)
{
    (void)dev;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = a.dtype == FSDP_BF16;
    const int64_t size = bf16 ? 2 : 4;
    const int parts = (int)backward_parts(a.rows, a.cols);
    BackwardParams p{a.rows,  a.lddy,    a.ldx,  a.lddx, (int)a.cols, a.dy, a.x, a.gamma, a.mean_in, a.rstd_in,
                     a.dx, a.partial, a.param_dtype == FSDP_BF16, 0};
    fsdp_status st = FSDP_OK;
    const Backward f{p, parts, s, &st};
    const bool full = vec_ok(a.x, a.ldx, size) && vec_ok(a.dy, a.lddy, size) && vec_ok(a.dx, a.lddx, size) &&
                      vec_ok(a.gamma, a.cols, size);
    const int held = bf16 ? (full ? backward_shape<uint16_t, true>(a.cols, f) : backward_shape<uint16_t, false>(a.cols, f))
                          : (full ? backward_shape<float, true>(a.cols, f) : backward_shape<float, false>(a.cols, f));
    if (!held)
        st = launch("layer_norm_backward", bf16 ? norm_backward_wide_kernel<uint16_t> : norm_backward_wide_kernel<float>,
                    parts, kWide, 0, s, 1, p);
    if (st != FSDP_OK)
        return st;
    return launch("layer_norm_backward (columns)", norm_columns_kernel, dim3((unsigned)((a.cols + 31) / 32), a.dbeta ? 2 : 1),
                  1024, 0, s, 1, a.partial, parts, a.cols, a.dgamma, a.dbeta, a.param_dtype == FSDP_BF16);
}

cudaError_t norm_wait_timeouts(unsigned long long *n) { return wait::wait_timeouts(n); }

}  // namespace fsdp
