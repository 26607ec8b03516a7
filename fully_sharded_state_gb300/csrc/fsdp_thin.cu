// fsdp_thin.cu -- the Newton-Schulz iteration of thin matrices, whose shorter
// side is at most 32, for sm_103a.
//
// All that the steps do to x they do by polynomials of S = x x^T (of the
// shorter side), and those commute: with T = a I + b S + c S^2 a step is
//     x <- T x,   S <- T S T,   so that   x_5 = T_5 ... T_1 x_0 = Q x_0 .
// So x is read once for S, the steps are products of k x k matrices in shared
// memory, and one more pass makes Q x_0: k^2 l flops twice instead of in every
// step, and one block per matrix instead of 15 products of a pipeline that
// starts and ends. All of it is fp32: S's rounding, 2^-24 of its largest
// element, reaches the small directions as T S T multiplies them by a^2 a step
// and ends at 7e-4 of the result at most (k = 25, rank 2 under 1 % noise), at
// 1e-6 for a Gaussian gradient. S is made symmetric after each step: left to
// itself the difference grows likewise, but between large directions and
// small ones (16 x 16: 3e-3 to 2e-2 off). Larger k would need more bits, and
// has the tensor cores.
//
// A block's threads are 2 x 2 tiles of S times slices of the longer side. x
// stays in shared memory where it fits (24 K elements); else it is read twice,
// with a block's few loads under way: there the team's or the products' many
// blocks win. us, here and there, one matrix and 64: 8 x 512 23 and 53, 23 and
// 84; 8 x 8192 101 and 108, 105 and 460; 32 x 512 36 and 55, 36 and 92; 32 x
// 2048 231 and 82, 234 and 183. (20 us and more of each are the caller's.)
#include "fsdp_muon.cuh"

namespace fsdp {
namespace {

constexpr int kThin = 32;
constexpr int kThinThreads = 512;
constexpr int kThinFloats = 24 * 1024;  // of x in shared memory at a time
constexpr double kMostGrowth = 32768.0;
constexpr int kLd = 36;                 // row stride of the k x k matrices: rows start on 16 bytes

struct ThinParams {
    int m, n, k, l, tall;
    int chunk, pitch;  // columns (of the longer side) at a time; a multiple of 4, and 4 more
    int steps, bf16;
    float eps, a, b, c;
    // newton_schulz
    const void *g;
    int64_t ldg, g_stride;
    uint16_t *out;
    int64_t ldo, out_stride;
    // muon
    int R, nesterov;
    float inv_r, mu, decay, lr;
    float *u;  // [batch][k][l], where x takes more than one chunk
    float *momentum[kMuonMaxMats];
    float *master[kMuonMaxMats];
    uint16_t *param[kMuonMaxMats];
    const void *grads[kMuonMaxGrads];
};

__device__ __forceinline__ float element(const void *p, int64_t at, int bf16)
{
    return bf16 ? bf16_at(static_cast<const uint16_t *>(p) + at) : static_cast<const float *>(p)[at];
}

// A 2 x 2 tile of A B, A symmetric.
__device__ __forceinline__ void tile_product(const float *a, const float *b, int k, int i, int j, float (&v)[2][2])
{
    v[0][0] = v[0][1] = v[1][0] = v[1][1] = 0.0f;
#pragma unroll 4
    for (int q = 0; q < k; q++) {
        const float2 x = *reinterpret_cast<const float2 *>(a + q * kLd + i);
        const float2 y = *reinterpret_cast<const float2 *>(b + q * kLd + j);
        v[0][0] = fmaf(x.x, y.x, v[0][0]);
        v[0][1] = fmaf(x.x, y.y, v[0][1]);
        v[1][0] = fmaf(x.y, y.x, v[1][0]);
        v[1][1] = fmaf(x.y, y.y, v[1][1]);
    }
}
__device__ __forceinline__ void put_tile(float *d, int i, int j, const float (&v)[2][2])
{
    *reinterpret_cast<float2 *>(d + i * kLd + j) = make_float2(v[0][0], v[0][1]);
    *reinterpret_cast<float2 *>(d + (i + 1) * kLd + j) = make_float2(v[1][0], v[1][1]);
}

// Columns c0 .. c0 + count of x to x[row][column], zeros up to whole groups of
// 4 columns and in the row that makes the rows even. first: u is formed from
// the gradients (kMuon), otherwise read back.
template <bool kMuon>
__device__ __forceinline__ void load_chunk(const ThinParams &p, int z, int c0, int count, bool first, float *x)
{
    constexpr int kFlight = 8;
    const int total = p.k * count;
    float *kept = p.u + (int64_t)z * p.k * p.l;
    for (int e0 = threadIdx.x; e0 < total; e0 += kFlight * kThinThreads) {
        float v[kFlight], m[kFlight];
        int row[kFlight], col[kFlight];
        int64_t at[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; f++) {
            const int e = e0 + f * kThinThreads < total ? e0 + f * kThinThreads : e0;
            // along the rows in memory
            const int per = p.tall ? p.k : count, q = e / per, r = e - q * per;
            row[f] = p.tall ? r : q;
            col[f] = p.tall ? q : r;
            const int64_t mr = p.tall ? c0 + q : q, mc = p.tall ? r : c0 + r;
            if (!kMuon) {
                v[f] = element(p.g, z * p.g_stride + mr * p.ldg + mc, p.bf16);
            } else if (first) {
                at[f] = mr * p.n + mc;
                m[f] = p.momentum[z][at[f]];
            } else {
                v[f] = kept[(int64_t)row[f] * p.l + c0 + col[f]];
            }
        }
        if (kMuon && first) {
            const void *const *grads = p.grads + z * p.R;
#pragma unroll 4
            for (int q = 0; q < p.R; q++) {
#pragma unroll
                for (int f = 0; f < kFlight; f++) {
                    const float o = element(grads[q], at[f], p.bf16);
                    v[f] = q == 0 ? o : __fadd_rn(v[f], o);
                }
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; f++) {
            if (e0 + f * kThinThreads >= total)
                break;
            if (kMuon && first) {
                v[f] = __fmul_rn(v[f], p.inv_r);
                m[f] = fmaf(p.mu, m[f], v[f]);
                v[f] = p.nesterov ? fmaf(p.mu, m[f], v[f]) : m[f];
                p.momentum[z][at[f]] = m[f];
                if (p.chunk < p.l)
                    kept[(int64_t)row[f] * p.l + c0 + col[f]] = v[f];
            }
            x[row[f] * p.pitch + col[f]] = v[f];
        }
    }
    const int end = (count + 3) / 4 * 4;
    for (int i = threadIdx.x; i < p.k * (end - count); i += kThinThreads)
        x[i / (end - count) * p.pitch + count + i % (end - count)] = 0.0f;
    if (p.k & 1)
        for (int c = threadIdx.x; c < end; c += kThinThreads)
            x[p.k * p.pitch + c] = 0.0f;
}

template <bool kMuon>
__global__ void __launch_bounds__(kThinThreads) thin_kernel(const __grid_constant__ ThinParams p)
{
    extern __shared__ __align__(16) float x[];
    __shared__ __align__(16) float mats[5][kThin * kLd];
    __shared__ float4 part[kThinThreads];
    launch_wait();
    launch_next();
    const int z = blockIdx.x, k = p.k;
    const int side = (k + 1) / 2, tiles = side * side, slices = kThinThreads / tiles;
    const int slice = threadIdx.x / tiles, tile = threadIdx.x % tiles;
    const int ti = tile / side * 2, tj = tile % side * 2;
    const bool mine = slice == 0;

    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c0 = 0; c0 < p.l; c0 += p.chunk) {
        const int count = p.l - c0 < p.chunk ? p.l - c0 : p.chunk;
        __syncthreads();
        load_chunk<kMuon>(p, z, c0, count, true, x);
        __syncthreads();
        if (slice < slices) {
            const float *a = x + ti * p.pitch, *b = x + tj * p.pitch;
#pragma unroll 2
            for (int c = slice * 4; c < count; c += slices * 4) {
                const float4 a0 = *reinterpret_cast<const float4 *>(a + c);
                const float4 a1 = *reinterpret_cast<const float4 *>(a + p.pitch + c);
                const float4 b0 = *reinterpret_cast<const float4 *>(b + c);
                const float4 b1 = *reinterpret_cast<const float4 *>(b + p.pitch + c);
                acc.x = fmaf(a0.x, b0.x, fmaf(a0.y, b0.y, fmaf(a0.z, b0.z, fmaf(a0.w, b0.w, acc.x))));
                acc.y = fmaf(a0.x, b1.x, fmaf(a0.y, b1.y, fmaf(a0.z, b1.z, fmaf(a0.w, b1.w, acc.y))));
                acc.z = fmaf(a1.x, b0.x, fmaf(a1.y, b0.y, fmaf(a1.z, b0.z, fmaf(a1.w, b0.w, acc.z))));
                acc.w = fmaf(a1.x, b1.x, fmaf(a1.y, b1.y, fmaf(a1.z, b1.z, fmaf(a1.w, b1.w, acc.w))));
            }
        }
    }
    part[threadIdx.x] = acc;
    // the slices, by halves
    int half = 1;
    while (half < slices)
        half *= 2;
    for (half /= 2; half > 0; half /= 2) {
        __syncthreads();
        if (slice < half && slice + half < slices) {
            const float4 o = part[threadIdx.x + half * tiles];
            acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
            part[threadIdx.x] = acc;
        }
    }
    float *s = mats[0], *t = mats[1], *v = mats[2], *q = mats[3], *w = mats[4];
    float d[2][2];
    if (mine) {
        d[0][0] = acc.x, d[0][1] = acc.y, d[1][0] = acc.z, d[1][1] = acc.w;
        put_tile(s, ti, tj, d);
    }
    __syncthreads();
    // the trace is the squared Frobenius norm
    float trace = 0.0f;
    for (int i = 0; i < k; i++)
        trace += s[i * kLd + i];
    const float inv = 1.0f / (sqrtf(trace) + p.eps);
    __syncthreads();
    if (mine) {
        // (inv S) inv: inv^2 alone may leave the range
        for (int i = 0; i < 4; i++)
            d[i / 2][i % 2] = d[i / 2][i % 2] * inv * inv;
        put_tile(s, ti, tj, d);
    }
    __syncthreads();
    for (int step = 0; step < p.steps; step++) {
        if (mine) {
            tile_product(s, s, k, ti, tj, d);
            for (int i = 0; i < 4; i++)
                d[i / 2][i % 2] = fmaf(p.c, d[i / 2][i % 2],
                                       fmaf(p.b, s[(ti + i / 2) * kLd + tj + i % 2], ti + i / 2 == tj + i % 2 ? p.a : 0.0f));
            put_tile(t, ti, tj, d);
            if (step == 0)
                put_tile(q, ti, tj, d);
        }
        __syncthreads();
        if (mine) {
            if (step > 0) {
                tile_product(t, q, k, ti, tj, d);
                put_tile(w, ti, tj, d);
            }
            if (step + 1 < p.steps) {
                tile_product(t, s, k, ti, tj, d);
                put_tile(v, ti, tj, d);
            }
        }
        if (step > 0) {
            float *old = q;
            q = w, w = old;
        }
        __syncthreads();
        if (step + 1 < p.steps) {
            if (mine) {
                tile_product(t, v, k, ti, tj, d);
                put_tile(w, ti, tj, d);
            }
            __syncthreads();
            if (mine) {
                for (int i = 0; i < 4; i++) {
                    const int r = ti + i / 2, c = tj + i % 2;
                    d[i / 2][i % 2] = 0.5f * (w[r * kLd + c] + w[c * kLd + r]);
                }
                put_tile(s, ti, tj, d);
            }
            __syncthreads();
        }
    }
    const bool again = p.chunk < p.l;
    for (int c0 = 0; c0 < p.l; c0 += p.chunk) {
        const int count = p.l - c0 < p.chunk ? p.l - c0 : p.chunk, groups = (count + 3) / 4;
        if (again) {
            __syncthreads();
            load_chunk<kMuon>(p, z, c0, count, false, x);
            __syncthreads();
        }
        for (int e = threadIdx.x; e < (k + 3) / 4 * groups; e += kThinThreads) {
            const int i0 = e / groups * 4, c = e % groups * 4;
            float r[4][4] = {};
#pragma unroll 4
            for (int j = 0; j < k; j++) {
                const float4 f = *reinterpret_cast<const float4 *>(q + j * kLd + i0);
                const float4 y = *reinterpret_cast<const float4 *>(x + j * p.pitch + c);
                const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    r[i][0] = fmaf(fs[i], y.x, r[i][0]);
                    r[i][1] = fmaf(fs[i], y.y, r[i][1]);
                    r[i][2] = fmaf(fs[i], y.z, r[i][2]);
                    r[i][3] = fmaf(fs[i], y.w, r[i][3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (i0 + i >= k || c + j >= count)
                        continue;
                    const int64_t mr = p.tall ? c0 + c + j : i0 + i, mc = p.tall ? i0 + i : c0 + c + j;
                    const float y = r[i][j] * inv;
                    if (kMuon) {
                        const int64_t at = mr * p.n + mc;
                        const float o = fmaf(-p.lr, y, p.master[z][at] * p.decay);
                        p.master[z][at] = o;
                        if (p.param[z])
                            p.param[z][at] = to_bf16(o);
                    } else {
                        p.out[z * p.out_stride + mr * p.ldo + mc] = to_bf16(y);
                    }
                }
        }
    }
}

}  // namespace

// Estimated clocks, or -1 where the matrices do not fit.
int64_t thin_clocks(const SchulzArgs &a, int sms)
{
    const int64_t k = a.m < a.n ? a.m : a.n, l = a.m < a.n ? a.n : a.m;
    // an error of S's small directions grows by a^2 a step: 2^-24 to 1e-3 in
    // the default five, not further
    double growth = 1.0;
    for (int i = 1; i < a.steps && growth <= kMostGrowth; i++)
        growth *= (double)a.a * a.a > 1.0 ? (double)a.a * a.a : 1.0;
    if (k > kThin || a.steps < 1 || l > (1 << 24) || !(growth <= kMostGrowth))
        return -1;
    // per element of x: its loads, and the k products of either pass; twice
    // the loads, and fewer of them under way, where x does not stay
    const bool stays = (k + 1) / 2 * 2 * (l + 4) <= kThinFloats;
    const double each = (stays ? 1.0 + 0.06 * (double)k : 2.0 + 0.14 * (double)k) + (a.grads ? 0.08 * a.R : 0.0);
    return (a.batch + sms - 1) / sms * ((int64_t)((double)(k * l) * each) + a.steps * (1200 + 60 * k)) + 6000;
}

fsdp_status launch_thin(const SchulzArgs &a, void *workspace, int dev, void *stream)
{
    const bool muon = a.grads != nullptr;
    ThinParams p{};
    p.m = (int)a.m;
    p.n = (int)a.n;
    p.tall = a.m > a.n;
    p.k = p.tall ? p.n : p.m;
    p.l = p.tall ? p.m : p.n;
    const int rows = (p.k + 1) / 2 * 2, most = (kThinFloats / rows - 4) / 4 * 4, all = (p.l + 3) / 4 * 4;
    p.chunk = all < most ? all : most;
    p.pitch = p.chunk + 4;
    p.steps = a.steps;
    p.bf16 = a.dtype == FSDP_BF16;
    p.eps = a.eps, p.a = a.a, p.b = a.b, p.c = a.c;
    p.g = a.g, p.ldg = a.ldg, p.g_stride = a.g_stride;
    p.out = static_cast<uint16_t *>(a.out), p.ldo = a.ldo, p.out_stride = a.out_stride;
    if (muon) {
        p.R = a.R, p.nesterov = a.nesterov;
        p.inv_r = 1.0f / (float)a.R, p.mu = a.mu, p.decay = a.decay, p.lr = a.lr;
        p.u = schulz_plan(a.batch, a.m, a.n, true, workspace).x32;
        for (int i = 0; i < a.batch; i++) {
            p.momentum[i] = a.momentum[i];
            p.master[i] = a.master[i];
            p.param[i] = a.param_out ? static_cast<uint16_t *>(a.param_out[i]) : nullptr;
        }
        for (int i = 0; i < a.batch * a.R; i++)
            p.grads[i] = a.grads[i];
    }
    auto kernel = muon ? thin_kernel<true> : thin_kernel<false>;
    const size_t smem = (size_t)rows * p.pitch * sizeof(float);
    if (smem > 16 * 1024 && !current_record()) {  // with the 31 KB of its own, past what needs no leave
        const cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kThinFloats * (int)sizeof(float));
        if (err != cudaSuccess)
            return set_error(FSDP_ECUDA, "newton_schulz (thin): cudaFuncSetAttribute: %s", cudaGetErrorString(err));
    }
    return launch(muon ? "muon (thin)" : "newton_schulz (thin)", kernel, dim3((unsigned)a.batch), kThinThreads, smem,
                  static_cast<cudaStream_t>(stream), 1, p);
}

}  // namespace fsdp
