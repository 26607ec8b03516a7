// fsdp_muon.cu -- Newton-Schulz orthogonalisation and the Muon step, for
// sm_103a.
//
//   start    one pass over the input: the norm's partial sums; for the Muon
//            step also the fold of the R ranks' gradients and the momentum
//   scale    x = u / (||u||_F + eps), in fp32 and, for the products, fp16
//   steps x  S = x x^T (or x^T x: the smaller side), P = b S + c S^2 and
//            x = a x + P x, three products on the tensor cores. S and P are
//            symmetric: only the squares on and above the diagonal are
//            multiplied, and the epilogue stores both triangles.
//   the last product's epilogue writes the result, or updates the master
//
// Numbers: the operands are fp16 (all are at most about 1 in size; 2^-11
// each), sums are fp32, and x itself is carried in fp32, so that the linear
// term a x is never rounded: with x kept in fp16 alone, a 512 x 512 gradient
// of rank 16 under 1 % noise comes out 4e-2 off (its small directions grow by
// a per step, and the rounding with them); so it is 4e-4 off. Full-rank
// gradients: 1.5e-3 either way.
#include "fsdp_tc.cuh"

namespace fsdp {
namespace {

using namespace tc;

constexpr int kTileN = 256;
constexpr int kStartThreads = 256;
constexpr int kMaxParts = 256;  // partial sums of one matrix's norm

__device__ __forceinline__ float block_sum(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < kStartThreads / 32; i++)
        v += sh[i];
    __syncthreads();
    return v;
}

// 8 elements of a row, from column c on; zeros past the end.
__device__ __forceinline__ void load8(const void *base, int64_t at, int left, bool bf16, float (&v)[8])
{
    if (bf16) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (left >= 8 && aligned(p, 16)) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            const uint32_t *w = reinterpret_cast<const uint32_t *>(&u);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = i < left ? bf16_at(p + i) : 0.0f;
        }
    } else {
        const float *p = static_cast<const float *>(base) + at;
        if (left >= 8 && aligned(p, 16)) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = i < left ? p[i] : 0.0f;
        }
    }
}
__device__ __forceinline__ void store8(float *p, int left, const float (&v)[8])
{
    if (left >= 8 && aligned(p, 16)) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < left)
                p[i] = v[i];
    }
}

struct StartParams {
    int m, n, groups;       // groups of 8 columns per row
    int64_t ldx;            // stride of x
    int parts;
    float *x32;             // [batch][m][ldx]: u
    float *partial;         // [batch][kMaxParts]
    // newton_schulz
    const void *g;
    int64_t ldg, g_stride;
    int bf16;
    // muon
    int R, nesterov;
    float inv_r, mu;
    float *momentum[kMuonMaxMats];
    const void *grads[kMuonMaxGrads];
};

// Grid (parts, batch). A block's share of a matrix and so the norm's order
// depend on the sizes alone.
template <bool kMuon>
__global__ void __launch_bounds__(kStartThreads) start_kernel(const __grid_constant__ StartParams p)
{
    __shared__ float sh[kStartThreads / 32];
    const int z = blockIdx.y;
    float *x = p.x32 + (int64_t)z * p.m * p.ldx;
    const int64_t total = (int64_t)p.m * p.groups;
    float sq = 0.0f;
    for (int64_t i = (int64_t)blockIdx.x * kStartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kStartThreads) {
        const int r = (int)(i / p.groups), c = (int)(i - (int64_t)r * p.groups) * 8, left = p.n - c;
        float u[8];
        if (kMuon) {
            const int64_t at = (int64_t)r * p.n + c;
            load8(p.grads[z * p.R], at, left, p.bf16, u);
            for (int q = 1; q < p.R; q++) {
                float o[8];
                load8(p.grads[z * p.R + q], at, left, p.bf16, o);
#pragma unroll
                for (int k = 0; k < 8; k++)
                    u[k] = __fadd_rn(u[k], o[k]);
            }
            float m[8];
            load8(p.momentum[z], at, left, false, m);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                u[k] = __fmul_rn(u[k], p.inv_r);
                m[k] = fmaf(p.mu, m[k], u[k]);
                u[k] = p.nesterov ? fmaf(p.mu, m[k], u[k]) : m[k];
            }
            store8(p.momentum[z] + at, left, m);
        } else {
            load8(p.g, z * p.g_stride + r * p.ldg + c, left, p.bf16, u);
        }
        store8(x + r * p.ldx + c, 8, u);
#pragma unroll
        for (int k = 0; k < 8; k++)
            sq += u[k] * u[k];
    }
    sq = block_sum(sq, sh);
    if (threadIdx.x == 0)
        p.partial[z * kMaxParts + blockIdx.x] = sq;
}

__global__ void __launch_bounds__(kStartThreads) scale_kernel(float *x32, uint16_t *x16, const float *partial, int parts,
                                                              float eps, int64_t count)
{
    __shared__ float sh[kStartThreads / 32];
    const int z = blockIdx.y;
    const float sq = block_sum(threadIdx.x < parts ? partial[z * kMaxParts + threadIdx.x] : 0.0f, sh);
    const float inv = 1.0f / (sqrtf(sq) + eps);
    for (int64_t i = ((int64_t)blockIdx.x * kStartThreads + threadIdx.x) * 8; i < count;
         i += (int64_t)gridDim.x * kStartThreads * 8) {
        float v[8];
        load8(x32 + z * count, i, 8, false, v);
        uint4 u;
        uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
        for (int k = 0; k < 8; k++)
            v[k] *= inv;
#pragma unroll
        for (int k = 0; k < 4; k++)
            w[k] = pack_f16(v[2 * k], v[2 * k + 1]);
        store8(x32 + z * count + i, 8, v);
        *reinterpret_cast<uint4 *>(x16 + z * count + i) = u;
    }
}

// S, or P = b S + c S^2 (from != NULL), in fp16, both triangles.
struct SquareEpi {
    struct Params {
        uint16_t *out;
        const uint16_t *from;
        int64_t ld, stride;
        float b, c;
    };
    template <int COLS>
    static __device__ __forceinline__ void run(const Params &p, const Slot &x)
    {
        uint16_t *out = p.out + x.z * p.stride;
        const int64_t row = (int64_t)x.row * p.ld;
#pragma unroll 1
        for (int c = 0; c < COLS / 32; c++) {
            float v[32];
            x.load(c, v);
            const int col = x.col + c * 32, n = x.N - col;
            if (x.row >= x.M || n <= 0)
                continue;
            if (p.from) {
                const uint16_t *f = p.from + x.z * p.stride + row + col;
#pragma unroll
                for (int i = 0; i < 32; i++)
                    if (i < n)
                        v[i] = fmaf(p.c, v[i], p.b * __half2float(__ushort_as_half(f[i])));
            }
            store16<false>(out + row + col, v, n);
            if (x.mirror) {
#pragma unroll
                for (int i = 0; i < 32; i++)
                    if (i < n)
                        out[(int64_t)(col + i) * p.ld + x.row] = __half_as_ushort(__float2half_rn(v[i]));
            }
        }
    }
};

// x = a x + (P x): fp32 in place and the next step's fp16 operand.
struct StepEpi {
    struct Params {
        float *x32;
        uint16_t *x16;
        int64_t ld, stride;
        float a;
    };
    template <int COLS>
    static __device__ __forceinline__ void run(const Params &p, const Slot &x)
    {
        const int64_t at = x.z * p.stride + (int64_t)x.row * p.ld + x.col;
#pragma unroll 1
        for (int c = 0; c < COLS / 32; c++) {
            float v[32], o[32];
            x.load(c, v);
            const int n = x.N - x.col - c * 32;
            if (x.row >= x.M || n <= 0)
                continue;
            load_f32(p.x32 + at + c * 32, o, n);
#pragma unroll
            for (int i = 0; i < 32; i++)
                v[i] = fmaf(p.a, o[i], v[i]);
            store_f32(p.x32 + at + c * 32, v, n);
            store16<false>(p.x16 + at + c * 32, v, n);
        }
    }
};

// The last step: the result in bf16.
struct OutEpi {
    struct Params {
        const float *x32;
        int64_t ld, stride;
        float a;
        uint16_t *out;
        int64_t ldo, out_stride;
    };
    template <int COLS>
    static __device__ __forceinline__ void run(const Params &p, const Slot &x)
    {
        const int64_t at = x.z * p.stride + (int64_t)x.row * p.ld + x.col;
        uint16_t *out = p.out + x.z * p.out_stride + x.row * p.ldo + x.col;
#pragma unroll 1
        for (int c = 0; c < COLS / 32; c++) {
            float v[32], o[32];
            x.load(c, v);
            const int n = x.N - x.col - c * 32;
            if (x.row >= x.M || n <= 0)
                continue;
            load_f32(p.x32 + at + c * 32, o, n);
#pragma unroll
            for (int i = 0; i < 32; i++)
                v[i] = fmaf(p.a, o[i], v[i]);
            store16<true>(out + c * 32, v, n);
        }
    }
};

// The last step of a Muon step: w = w decay - lr x.
struct MasterEpi {
    struct Params {
        const float *x32;
        int64_t ld, stride;
        float a, decay, lr;
        int64_t n;
        float *master[kMuonMaxMats];
        uint16_t *param[kMuonMaxMats];
    };
    template <int COLS>
    static __device__ __forceinline__ void run(const Params &p, const Slot &x)
    {
        const int64_t at = x.z * p.stride + (int64_t)x.row * p.ld + x.col;
        const int64_t to = (int64_t)x.row * p.n + x.col;
        float *master = p.master[x.z];
        uint16_t *param = p.param[x.z];
#pragma unroll 1
        for (int c = 0; c < COLS / 32; c++) {
            float v[32], o[32];
            x.load(c, v);
            const int n = x.N - x.col - c * 32;
            if (x.row >= x.M || n <= 0)
                continue;
            load_f32(p.x32 + at + c * 32, o, n);
#pragma unroll
            for (int i = 0; i < 32; i++)
                v[i] = fmaf(p.a, o[i], v[i]);
            load_f32(master + to + c * 32, o, n);
#pragma unroll
            for (int i = 0; i < 32; i++)
                v[i] = fmaf(-p.lr, v[i], o[i] * p.decay);
            store_f32(master + to + c * 32, v, n);
            if (param)
                store16<true>(param + to + c * 32, v, n);
        }
    }
};

// steps = 0: the scaled input is the result.
struct FinishParams {
    const float *x32;
    int m, n, groups;
    int64_t ld;
    uint16_t *out;
    int64_t ldo, out_stride;
    float decay, lr;
    float *master[kMuonMaxMats];
    uint16_t *param[kMuonMaxMats];
};
template <bool kMuon>
__global__ void __launch_bounds__(kStartThreads) finish_kernel(const __grid_constant__ FinishParams p)
{
    const int z = blockIdx.y;
    const float *x = p.x32 + (int64_t)z * p.m * p.ld;
    for (int64_t i = (int64_t)blockIdx.x * kStartThreads + threadIdx.x; i < (int64_t)p.m * p.n;
         i += (int64_t)gridDim.x * kStartThreads) {
        const int64_t r = i / p.n, c = i - r * p.n;
        const float v = x[r * p.ld + c];
        if (kMuon) {
            const float w = fmaf(-p.lr, v, p.master[z][i] * p.decay);
            p.master[z][i] = w;
            if (p.param[z])
                p.param[z][i] = to_bf16(w);
        } else {
            p.out[z * p.out_stride + r * p.ldo + c] = to_bf16(v);
        }
    }
}

struct Plan {
    int64_t ldx, ldk, k;
    float *x32, *partial;
    uint16_t *x16[2], *s, *p;
    int64_t bytes;
};

Plan plan_of(int64_t batch, int64_t m, int64_t n, void *base)
{
    Plan q{};
    q.k = m < n ? m : n;
    q.ldx = ceil_to(n, 16);
    q.ldk = ceil_to(q.k, 16);
    Carver c(base);
    q.partial = c.take<float>(batch * kMaxParts);
    q.x32 = c.take<float>(batch * m * q.ldx);
    q.x16[0] = c.take<uint16_t>(batch * m * q.ldx);
    q.x16[1] = c.take<uint16_t>(batch * m * q.ldx);
    q.s = c.take<uint16_t>(batch * q.k * q.ldk);
    q.p = c.take<uint16_t>(batch * q.k * q.ldk);
    q.bytes = c.used();
    return q;
}

fsdp_status launched(const char *what)
{
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? FSDP_OK
                              : set_error(FSDP_ECUDA, "%s launch failed: %s", what, cudaGetErrorString(err));
}

}  // namespace

int64_t schulz_workspace(int64_t batch, int64_t m, int64_t n) { return plan_of(batch, m, n, nullptr).bytes; }

fsdp_status launch_newton_schulz(const SchulzArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool muon = a.grads != nullptr;
    const int sms = device_sms(dev);
    const Plan q = plan_of(a.batch, a.m, a.n, workspace);
    const int batch = (int)a.batch, m = (int)a.m, n = (int)a.n;
    fsdp_status st;

    StartParams sp{};
    sp.m = m;
    sp.n = n;
    sp.groups = (int)(q.ldx / 8);
    sp.ldx = q.ldx;
    const int64_t need = (a.m * sp.groups + kStartThreads - 1) / kStartThreads;
    const int64_t fill = (4 * sms + a.batch - 1) / a.batch;
    int64_t parts = need < fill ? need : fill;
    sp.parts = (int)(parts < kMaxParts ? parts : kMaxParts);
    sp.x32 = q.x32;
    sp.partial = q.partial;
    sp.bf16 = a.dtype == FSDP_BF16;
    const dim3 grid(sp.parts, batch);
    if (muon) {
        sp.R = a.R;
        sp.nesterov = a.nesterov;
        sp.inv_r = 1.0f / (float)a.R;
        sp.mu = a.mu;
        for (int i = 0; i < batch; i++)
            sp.momentum[i] = a.momentum[i];
        for (int i = 0; i < batch * a.R; i++)
            sp.grads[i] = a.grads[i];
        start_kernel<true><<<grid, kStartThreads, 0, s>>>(sp);
    } else {
        sp.g = a.g;
        sp.ldg = a.ldg;
        sp.g_stride = a.g_stride;
        start_kernel<false><<<grid, kStartThreads, 0, s>>>(sp);
    }
    if ((st = launched("newton_schulz (start)")) != FSDP_OK)
        return st;
    scale_kernel<<<grid, kStartThreads, 0, s>>>(q.x32, q.x16[0], q.partial, sp.parts, a.eps, a.m * q.ldx);
    if ((st = launched("newton_schulz (scale)")) != FSDP_OK)
        return st;

    if (a.steps == 0) {
        FinishParams fp{};
        fp.x32 = q.x32;
        fp.m = m;
        fp.n = n;
        fp.ld = q.ldx;
        fp.out = static_cast<uint16_t *>(a.out);
        fp.ldo = a.ldo;
        fp.out_stride = a.out_stride;
        fp.decay = a.decay;
        fp.lr = a.lr;
        for (int i = 0; muon && i < batch; i++) {
            fp.master[i] = a.master[i];
            fp.param[i] = a.param_out ? static_cast<uint16_t *>(a.param_out[i]) : nullptr;
        }
        if (muon)
            finish_kernel<true><<<grid, kStartThreads, 0, s>>>(fp);
        else
            finish_kernel<false><<<grid, kStartThreads, 0, s>>>(fp);
        return launched("newton_schulz (result)");
    }

    const bool wide = a.m <= a.n;
    const int64_t xs = a.m * q.ldx, ks = q.k * q.ldk;
    MasterEpi::Params mp{};
    if (muon) {
        mp.x32 = q.x32;
        mp.ld = q.ldx;
        mp.stride = xs;
        mp.a = a.a;
        mp.decay = a.decay;
        mp.lr = a.lr;
        mp.n = a.n;
        for (int i = 0; i < batch; i++) {
            mp.master[i] = a.master[i];
            mp.param[i] = a.param_out ? static_cast<uint16_t *>(a.param_out[i]) : nullptr;
        }
    }
    for (int step = 0; step < a.steps; step++) {
        const Operand x{q.x16[step % 2], a.n, a.m, q.ldx, xs};
        const Operand gram{q.s, q.k, q.k, q.ldk, ks}, poly{q.p, q.k, q.k, q.ldk, ks};
        Shape sq{};
        sq.M = sq.N = (int)q.k;
        sq.K = wide ? n : m;
        sq.batch = batch;
        sq.sym = 1;
        const SquareEpi::Params e1{q.s, nullptr, q.ldk, ks, 0.0f, 0.0f};
        const SquareEpi::Params e2{q.p, q.s, q.ldk, ks, a.b, a.c};
        st = wide ? product<1, kTileN, false, false, SquareEpi>(sq, x, x, false, e1, dev, s, "newton_schulz (S)")
                  : product<1, kTileN, true, true, SquareEpi>(sq, x, x, false, e1, dev, s, "newton_schulz (S)");
        if (st != FSDP_OK)
            return st;
        sq.K = (int)q.k;
        if ((st = product<1, kTileN, false, false, SquareEpi>(sq, gram, gram, false, e2, dev, s,
                                                              "newton_schulz (P)")) != FSDP_OK)
            return st;
        Shape up{};
        up.M = m;
        up.N = n;
        up.K = (int)q.k;
        up.batch = batch;
        auto update = [&](auto epi, const auto &ep) {
            using E = decltype(epi);
            // wide: P x, x with its columns adjacent; tall: x P, P symmetric
            return wide ? product<1, kTileN, false, true, E>(up, poly, x, false, ep, dev, s, "newton_schulz (x)")
                        : product<1, kTileN, false, false, E>(up, x, poly, false, ep, dev, s, "newton_schulz (x)");
        };
        if (step + 1 < a.steps)
            st = update(StepEpi{}, StepEpi::Params{q.x32, q.x16[(step + 1) % 2], q.ldx, xs, a.a});
        else if (muon)
            st = update(MasterEpi{}, mp);
        else
            st = update(OutEpi{}, OutEpi::Params{q.x32, q.ldx, xs, a.a, static_cast<uint16_t *>(a.out), a.ldo,
                                                 a.out_stride});
        if (st != FSDP_OK)
            return st;
    }
    return FSDP_OK;
}

cudaError_t muon_wait_timeouts(unsigned long long *n) { return tc::wait_timeouts(n); }

}  // namespace fsdp
