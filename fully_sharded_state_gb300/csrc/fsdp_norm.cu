// fsdp_norm.cu -- layer norm, forward and backward, for sm_103a.
//
// Both passes are bound by HBM: 8 (forward) or 14 (backward) flops per
// element that is read or written once. TPR threads hold one row in
// registers, 16 elements each, so x (and dy) is read once whatever the
// statistics need; rows wider than 16,384 are walked again instead, from L2.
// A row's mean and its sum of squares about the mean are joined from the
// threads' own (count, mean, M2) in one exchange, which keeps fp32 precision
// under a large mean where sum(x^2) - mean^2 would lose it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fsdp_ops_internal.h"

namespace fsdp {
namespace {

constexpr int kElems = 16;        // of a row, per thread
constexpr int kMaxTpr = 1024;
constexpr int kMinThreads = 256;  // narrow rows share a block

__device__ __forceinline__ float to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(uint16_t &d, float f) { d = __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ void from_f32(float &d, float f) { d = f; }

// Element i of a thread's 16 is column col(i): pieces of V adjacent ones, the
// pieces of one row's threads side by side.
template <typename T, bool kVec>
struct Cols {
    static constexpr int V = kVec ? 16 / (int)sizeof(T) : 1;
    static constexpr int kPieces = kElems / V;
    template <int TPR>
    static __device__ __forceinline__ int at(int i, int t)
    {
        return ((i / V) * TPR + t) * V + i % V;
    }
};

template <typename T, bool kVec, int TPR>
__device__ __forceinline__ void load_row(const T *p, int cols, int t, float (&v)[kElems])
{
    using C = Cols<T, kVec>;
#pragma unroll
    for (int q = 0; q < C::kPieces; q++) {
        const int c = (q * TPR + t) * C::V;
        if (kVec && c + C::V <= cols) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + c);
            const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
            for (int i = 0; i < C::V; i++)
                v[q * C::V + i] = to_f32(e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < C::V; i++)
                v[q * C::V + i] = c + i < cols ? to_f32(p[c + i]) : 0.0f;
        }
    }
}

template <typename T, bool kVec, int TPR>
__device__ __forceinline__ void store_row(T *p, int cols, int t, const float (&v)[kElems], bool vec)
{
    using C = Cols<T, kVec>;
#pragma unroll
    for (int q = 0; q < C::kPieces; q++) {
        const int c = (q * TPR + t) * C::V;
        if (kVec && vec && c + C::V <= cols) {
            uint4 u;
            T *e = reinterpret_cast<T *>(&u);
#pragma unroll
            for (int i = 0; i < C::V; i++)
                from_f32(e[i], v[q * C::V + i]);
            *reinterpret_cast<uint4 *>(p + c) = u;
        } else {
#pragma unroll
            for (int i = 0; i < C::V; i++)
                if (c + i < cols)
                    from_f32(p[c + i], v[q * C::V + i]);
        }
    }
}

// gamma or beta of the thread's columns, of either type.
template <typename T, bool kVec, int TPR>
__device__ __forceinline__ void load_param(const void *p, bool bf16, int cols, int t, float (&v)[kElems])
{
    using C = Cols<T, kVec>;
#pragma unroll
    for (int i = 0; i < kElems; i++) {
        const int c = C::template at<TPR>(i, t);
        v[i] = c >= cols ? 0.0f
               : bf16    ? to_f32(static_cast<const uint16_t *>(p)[c])
                         : static_cast<const float *>(p)[c];
    }
}

// Count, mean and sum of squares about the mean of a part of a row.
struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments &a, const Moments &b)
{
    const float n = a.n + b.n;
    if (n == 0.0f)
        return a;
    const float d = b.mean - a.mean, r = b.n / n;
    return {n, a.mean + d * r, a.m2 + b.m2 + d * d * a.n * r};
}

// Joins over the TPR threads of a row; every one gets the same bits.
template <int TPR>
__device__ __forceinline__ Moments join_row(Moments m, float (*sh)[3])
{
    constexpr int kWarps = TPR / 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Moments b;
        b.n = __shfl_xor_sync(0xffffffffu, m.n, o);
        b.mean = __shfl_xor_sync(0xffffffffu, m.mean, o);
        b.m2 = __shfl_xor_sync(0xffffffffu, m.m2, o);
        // the lower lane's part first, on both sides
        m = (threadIdx.x & o) ? join(b, m) : join(m, b);
    }
    if (kWarps > 1) {
        const int w = threadIdx.x / 32;
        if (threadIdx.x % 32 == 0) {
            sh[w][0] = m.n;
            sh[w][1] = m.mean;
            sh[w][2] = m.m2;
        }
        __syncthreads();
        const int w0 = w / kWarps * kWarps;
        m = {sh[w0][0], sh[w0][1], sh[w0][2]};
        for (int i = 1; i < kWarps; i++)
            m = join(m, {sh[w0 + i][0], sh[w0 + i][1], sh[w0 + i][2]});
        __syncthreads();
    }
    return m;
}

// Two sums over the TPR threads of a row.
template <int TPR>
__device__ __forceinline__ void sum_row(float &a, float &b, float (*sh)[3])
{
    constexpr int kWarps = TPR / 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (kWarps > 1) {
        const int w = threadIdx.x / 32;
        if (threadIdx.x % 32 == 0) {
            sh[w][0] = a;
            sh[w][1] = b;
        }
        __syncthreads();
        const int w0 = w / kWarps * kWarps;
        a = sh[w0][0];
        b = sh[w0][1];
        for (int i = 1; i < kWarps; i++) {
            a += sh[w0 + i][0];
            b += sh[w0 + i][1];
        }
        __syncthreads();
    }
}

template <int TPR>
constexpr int block_of()
{
    return TPR < kMinThreads ? kMinThreads : TPR;
}

struct ForwardParams {
    int64_t rows, ldx, ldy;
    int cols;
    const void *x, *gamma, *beta;
    void *y;
    float *mean, *rstd;
    float eps;
    int param_bf16, vec_out;
};

template <typename T, bool kVec, int TPR>
__global__ void __launch_bounds__(block_of<TPR>()) norm_forward_kernel(const ForwardParams p)
{
    constexpr int kRowsPerBlock = block_of<TPR>() / TPR;
    __shared__ float sh[32][3];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    using C = Cols<T, kVec>;
    float gamma[kElems], beta[kElems];
    load_param<T, kVec, TPR>(p.gamma, p.param_bf16, p.cols, t, gamma);
    if (p.beta) {
        load_param<T, kVec, TPR>(p.beta, p.param_bf16, p.cols, t, beta);
    } else {
#pragma unroll
        for (int i = 0; i < kElems; i++)
            beta[i] = 0.0f;
    }
    for (int64_t r0 = (int64_t)blockIdx.x * kRowsPerBlock; r0 < p.rows; r0 += (int64_t)gridDim.x * kRowsPerBlock) {
        const int64_t r = r0 + sub;
        const bool live = r < p.rows;
        float v[kElems];
        if (live) {
            load_row<T, kVec, TPR>(static_cast<const T *>(p.x) + r * p.ldx, p.cols, t, v);
        } else {
#pragma unroll
            for (int i = 0; i < kElems; i++)
                v[i] = 0.0f;
        }
        float n = 0.0f, s = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int i = 0; i < kElems; i++)
            if (C::template at<TPR>(i, t) < p.cols) {
                n += 1.0f;
                s += v[i];
            }
        const float mu = n > 0.0f ? s / n : 0.0f;
#pragma unroll
        for (int i = 0; i < kElems; i++)
            if (C::template at<TPR>(i, t) < p.cols) {
                const float d = v[i] - mu;
                m2 += d * d;
            }
        const Moments m = join_row<TPR>({n, mu, m2}, sh);
        const float rstd = 1.0f / sqrtf(m.m2 / (float)p.cols + p.eps);
        if (!live)
            continue;
        if (t == 0 && p.mean) {
            p.mean[r] = m.mean;
            p.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < kElems; i++)
            v[i] = (v[i] - m.mean) * rstd * gamma[i] + beta[i];
        store_row<T, kVec, TPR>(static_cast<T *>(p.y) + r * p.ldy, p.cols, t, v, p.vec_out);
    }
}

struct BackwardParams {
    int64_t rows, lddy, ldx, lddx;
    int cols;
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    void *dx;
    float *partial;  // [2][gridDim.x][cols]: sums of dy*xhat and of dy
    int param_bf16, vec_out;
};

// dgamma and dbeta: every thread sums its 16 columns over the block's rows in
// registers; a block's rows then join in shared memory, and its sums go to
// its own line of `partial`, which norm_columns_kernel adds up in order.
template <typename T, bool kVec, int TPR>
__global__ void __launch_bounds__(block_of<TPR>()) norm_backward_kernel(const BackwardParams p)
{
    constexpr int kRowsPerBlock = block_of<TPR>() / TPR;
    __shared__ float sh[32][3];
    __shared__ float col[kRowsPerBlock > 1 ? kRowsPerBlock : 1][kRowsPerBlock > 1 ? TPR * kElems : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    using C = Cols<T, kVec>;
    float gamma[kElems], dg[kElems], db[kElems];
    load_param<T, kVec, TPR>(p.gamma, p.param_bf16, p.cols, t, gamma);
#pragma unroll
    for (int i = 0; i < kElems; i++)
        dg[i] = db[i] = 0.0f;
    const float inv = 1.0f / (float)p.cols;
    for (int64_t r0 = (int64_t)blockIdx.x * kRowsPerBlock; r0 < p.rows; r0 += (int64_t)gridDim.x * kRowsPerBlock) {
        const int64_t r = r0 + sub;
        const bool live = r < p.rows;
        float x[kElems], g[kElems], mean = 0.0f, rstd = 0.0f;
        if (live) {
            mean = p.mean[r];
            rstd = p.rstd[r];
            load_row<T, kVec, TPR>(static_cast<const T *>(p.x) + r * p.ldx, p.cols, t, x);
            load_row<T, kVec, TPR>(static_cast<const T *>(p.dy) + r * p.lddy, p.cols, t, g);
        } else {
#pragma unroll
            for (int i = 0; i < kElems; i++)
                x[i] = g[i] = 0.0f;
        }
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < kElems; i++) {
            x[i] = C::template at<TPR>(i, t) < p.cols ? (x[i] - mean) * rstd : 0.0f;
            dg[i] += g[i] * x[i];
            db[i] += g[i];
            g[i] *= gamma[i];
            a += g[i];
            b += g[i] * x[i];
        }
        sum_row<TPR>(a, b, sh);
        if (!live)
            continue;
        a *= inv;
        b *= inv;
#pragma unroll
        for (int i = 0; i < kElems; i++)
            g[i] = rstd * (g[i] - a - x[i] * b);
        store_row<T, kVec, TPR>(static_cast<T *>(p.dx) + r * p.lddx, p.cols, t, g, p.vec_out);
    }
    float *pg = p.partial + (int64_t)blockIdx.x * p.cols;
    float *pb = pg + (int64_t)gridDim.x * p.cols;
    if (kRowsPerBlock == 1) {
#pragma unroll
        for (int i = 0; i < kElems; i++) {
            const int c = C::template at<TPR>(i, t);
            if (c < p.cols) {
                pg[c] = dg[i];
                pb[c] = db[i];
            }
        }
    } else {
        for (int which = 0; which < 2; which++) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kElems; i++)
                col[sub][C::template at<TPR>(i, t)] = which ? db[i] : dg[i];
            __syncthreads();
            for (int c = threadIdx.x; c < p.cols; c += block_of<TPR>()) {
                float s = 0.0f;
                for (int q = 0; q < kRowsPerBlock; q++)
                    s += col[q][c];
                (which ? pb : pg)[c] = s;
            }
        }
    }
}

// Rows wider than 16 x 1024 elements: one block per row, which walks it once
// for the sum, once for the squares and once for the result.
__device__ __forceinline__ float block_sum(float a, float (*sh)[3])
{
    float b = 0.0f;
    sum_row<kMaxTpr>(a, b, sh);
    return a;
}

template <typename T>
__global__ void __launch_bounds__(kMaxTpr) norm_forward_wide_kernel(const ForwardParams p)
{
    __shared__ float sh[32][3];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        T *y = static_cast<T *>(p.y) + r * p.ldy;
        float s = 0.0f;
        for (int c = threadIdx.x; c < p.cols; c += kMaxTpr)
            s += to_f32(x[c]);
        const float mean = block_sum(s, sh) / (float)p.cols;
        s = 0.0f;
        for (int c = threadIdx.x; c < p.cols; c += kMaxTpr) {
            const float d = to_f32(x[c]) - mean;
            s += d * d;
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, sh) / (float)p.cols + p.eps);
        if (threadIdx.x == 0 && p.mean) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        for (int c = threadIdx.x; c < p.cols; c += kMaxTpr) {
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
__global__ void __launch_bounds__(kMaxTpr) norm_backward_wide_kernel(const BackwardParams p)
{
    __shared__ float sh[32][3];
    float *pg = p.partial + (int64_t)blockIdx.x * p.cols;
    float *pb = pg + (int64_t)gridDim.x * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += kMaxTpr)
        pg[c] = pb[c] = 0.0f;  // each column is one thread's throughout
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        const T *dy = static_cast<const T *>(p.dy) + r * p.lddy;
        T *dx = static_cast<T *>(p.dx) + r * p.lddx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float a = 0.0f, b = 0.0f;
        for (int c = threadIdx.x; c < p.cols; c += kMaxTpr) {
            const float xh = (to_f32(x[c]) - mean) * rstd, d = to_f32(dy[c]);
            const float ga = p.param_bf16 ? to_f32(static_cast<const uint16_t *>(p.gamma)[c])
                                          : static_cast<const float *>(p.gamma)[c];
            pg[c] += d * xh;
            pb[c] += d;
            a += d * ga;
            b += d * ga * xh;
        }
        sum_row<kMaxTpr>(a, b, sh);
        a /= (float)p.cols;
        b /= (float)p.cols;
        for (int c = threadIdx.x; c < p.cols; c += kMaxTpr) {
            const float xh = (to_f32(x[c]) - mean) * rstd, d = to_f32(dy[c]);
            const float ga = p.param_bf16 ? to_f32(static_cast<const uint16_t *>(p.gamma)[c])
                                          : static_cast<const float *>(p.gamma)[c];
            from_f32(dx[c], rstd * (d * ga - a - xh * b));
        }
    }
}

// dgamma, dbeta: the parts' sums, added in the parts' order. 32 columns and
// 8 slices of the parts per block.
__global__ void __launch_bounds__(256) norm_columns_kernel(const float *partial, int parts, int cols, void *dgamma,
                                                           void *dbeta, int param_bf16)
{
    __shared__ float sh[8][33];
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane;
    void *out = blockIdx.y ? dbeta : dgamma;
    const float *src = partial + (int64_t)blockIdx.y * parts * cols;
    float s = 0.0f;
    if (c < cols)
        for (int q = slice; q < parts; q += 8)
            s += src[(int64_t)q * cols + c];
    sh[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
        for (int q = 1; q < 8; q++)
            s += sh[q][lane];
        if (param_bf16)
            from_f32(static_cast<uint16_t *>(out)[c], s);
        else
            static_cast<float *>(out)[c] = s;
    }
}

bool vec_ok(const void *p, int64_t ld, int64_t size)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
}

int tpr_for(int64_t cols)
{
    int t = 32;
    while ((int64_t)t * kElems < cols && t < kMaxTpr)
        t *= 2;
    return t;
}

fsdp_status launched(const char *what)
{
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? FSDP_OK
                              : set_error(FSDP_ECUDA, "%s launch failed: %s", what, cudaGetErrorString(err));
}

// Calls f.template run<T, kVec, TPR>() for the types and widths given.
template <class F>
void with_shape(fsdp_dtype dt, bool vec, int tpr, F f)
{
    auto width = [&](auto type, auto v) {
        using T = decltype(type);
        constexpr bool kVec = decltype(v)::value;
        switch (tpr) {
        case 32: f.template run<T, kVec, 32>(); break;
        case 64: f.template run<T, kVec, 64>(); break;
        case 128: f.template run<T, kVec, 128>(); break;
        case 256: f.template run<T, kVec, 256>(); break;
        case 512: f.template run<T, kVec, 512>(); break;
        default: f.template run<T, kVec, 1024>(); break;
        }
    };
    if (dt == FSDP_BF16)
        vec ? width(uint16_t{}, std::true_type{}) : width(uint16_t{}, std::false_type{});
    else
        vec ? width(float{}, std::true_type{}) : width(float{}, std::false_type{});
}

struct Forward {
    const ForwardParams &p;
    int sms;
    cudaStream_t s;
    template <typename T, bool kVec, int TPR>
    void run()
    {
        const int64_t blocks = (p.rows + block_of<TPR>() / TPR - 1) / (block_of<TPR>() / TPR);
        const int64_t most = (int64_t)sms * (2048 / block_of<TPR>());
        norm_forward_kernel<T, kVec, TPR>
            <<<(unsigned)(blocks < most ? blocks : most), block_of<TPR>(), 0, s>>>(p);
    }
};
struct Backward {
    const BackwardParams &p;
    int parts;
    cudaStream_t s;
    template <typename T, bool kVec, int TPR>
    void run()
    {
        norm_backward_kernel<T, kVec, TPR><<<parts, block_of<TPR>(), 0, s>>>(p);
    }
};

int64_t backward_parts(int64_t rows, int64_t cols)
{
    const int tpr = tpr_for(cols);
    const int per = tpr < kMinThreads ? kMinThreads / tpr : 1;
    const int64_t blocks = (rows + per - 1) / per;
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
    if (a.rows == 0)
        return FSDP_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t size = a.dtype == FSDP_BF16 ? 2 : 4;
    ForwardParams p{a.rows, a.ldx, a.ldy, (int)a.cols, a.x, a.gamma, a.beta, a.y, a.mean, a.rstd, a.eps,
                    a.param_dtype == FSDP_BF16, vec_ok(a.y, a.ldy, size)};
    const int sms = device_sms(dev);
    if (a.cols > kElems * kMaxTpr) {
        const unsigned grid = (unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms);
        if (a.dtype == FSDP_BF16)
            norm_forward_wide_kernel<uint16_t><<<grid, kMaxTpr, 0, s>>>(p);
        else
            norm_forward_wide_kernel<float><<<grid, kMaxTpr, 0, s>>>(p);
    } else {
        with_shape(a.dtype, vec_ok(a.x, a.ldx, size), tpr_for(a.cols), Forward{p, sms, s});
    }
    return launched("layer_norm");
}

fsdp_status launch_layer_norm_backward(const NormArgs &a, int dev, void *stream)
{
    (void)dev;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t size = a.dtype == FSDP_BF16 ? 2 : 4;
    const int parts = (int)backward_parts(a.rows, a.cols);
    BackwardParams p{a.rows,  a.lddy,    a.ldx,  a.lddx, (int)a.cols, a.dy, a.x, a.gamma, a.mean_in, a.rstd_in,
                     a.dx, a.partial, a.param_dtype == FSDP_BF16, vec_ok(a.dx, a.lddx, size)};
    if (a.cols > kElems * kMaxTpr) {
        if (a.dtype == FSDP_BF16)
            norm_backward_wide_kernel<uint16_t><<<parts, kMaxTpr, 0, s>>>(p);
        else
            norm_backward_wide_kernel<float><<<parts, kMaxTpr, 0, s>>>(p);
    } else {
        with_shape(a.dtype, vec_ok(a.x, a.ldx, size) && vec_ok(a.dy, a.lddy, size), tpr_for(a.cols),
                   Backward{p, parts, s});
    }
    fsdp_status st = launched("layer_norm_backward");
    if (st != FSDP_OK)
        return st;
    const dim3 grid((unsigned)((a.cols + 31) / 32), a.dbeta ? 2 : 1);
    norm_columns_kernel<<<grid, 256, 0, s>>>(a.partial, parts, (int)a.cols, a.dgamma, a.dbeta,
                                             a.param_dtype == FSDP_BF16);
    return launched("layer_norm_backward (columns)");
}

}  // namespace fsdp
