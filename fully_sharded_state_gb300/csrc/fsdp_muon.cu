// fsdp_muon.cu -- Newton-Schulz orthogonalisation and the Muon step, for
// sm_103a.
//
//   start    one pass over the input: the norm's partial sums; for the Muon
//            step also the fold of the R ranks' gradients and the momentum
//   scale    x = u / (||u||_F + eps) in fp16, for the products; the fp32 u
//            is scaled where it is read next, in the first step's epilogue
//   steps x  S = x x^T (or x^T x: the smaller side), P = b S + c S^2 - d I and
//            x = (a + d) x + P x, three products on the tensor cores. S and P are
//            symmetric: only the squares on and above the diagonal are
//            multiplied, and the epilogue stores both triangles.
//   the last product's epilogue writes the result, or updates the master
//
// Numbers: the operands are fp16 (all are at most about 5 in size; 2^-11
// each), sums are fp32, and x itself is carried in fp32, so that the linear
// term is never rounded: with x kept in fp16 alone, a 512 x 512 gradient of
// rank 16 under 1 % noise comes out 4e-2 off (its small directions grow by a
// per step, and the rounding with them). P is shifted along its diagonal
// (shift_of): 4e-4 to 7e-4 off for that gradient, 8e-4 for a Gaussian one.
#include "fsdp_muon.cuh"

namespace fsdp {
namespace {

using namespace tc;

struct StartParams {
    int m, n, groups;       // groups of 8 columns per row
    int64_t ldx;            // stride of x
    int vec;                // every row of every input starts on 16 bytes
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

// The sum of R ranks' 8 elements, in rank order. The loads of four ranks are
// under way together.
template <bool kBf16>
__device__ __forceinline__ void fold_vec(const void *const *grads, int R, int64_t at, float (&u)[8])
{
    constexpr int kWords = kBf16 ? 1 : 2, kFlight = 4;
    for (int q0 = 0; q0 < R; q0 += kFlight) {
        uint4 w[kFlight][kWords];
#pragma unroll
        for (int k = 0; k < kFlight; k++)
            if (q0 + k < R) {
                const char *p = static_cast<const char *>(grads[q0 + k]) + at * (kBf16 ? 2 : 4);
#pragma unroll
                for (int i = 0; i < kWords; i++)
                    w[k][i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
            }
#pragma unroll
        for (int k = 0; k < kFlight; k++)
            if (q0 + k < R) {
                const uint32_t *e = reinterpret_cast<const uint32_t *>(w[k]);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float o = !kBf16 ? __uint_as_float(e[i])
                                    : i % 2 ? __uint_as_float(e[i / 2] & 0xffff0000u)
                                            : __uint_as_float(e[i / 2] << 16);
                    u[i] = q0 + k == 0 ? o : __fadd_rn(u[i], o);
                }
            }
    }
}

// Grid (parts, batch). A block's share of a matrix and so the norm's order
// depend on the sizes alone.
template <bool kMuon>
__global__ void __launch_bounds__(kStartThreads) start_kernel(const __grid_constant__ StartParams p)
{
    __shared__ float sh[kStartThreads / 32];
    launch_wait();
    launch_next();
    const int z = blockIdx.y;
    float *x = p.x32 + (int64_t)z * p.m * p.ldx;
    const int64_t total = (int64_t)p.m * p.groups;
    float sq = 0.0f;
    for (int64_t i = (int64_t)blockIdx.x * kStartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kStartThreads) {
        const int r = (int)((uint64_t)i < 0x80000000u ? (uint32_t)i / (uint32_t)p.groups : i / p.groups);
        const int c = (int)(i - (int64_t)r * p.groups) * 8, left = p.n - c;
        float u[8];
        if (kMuon) {
            const int64_t at = (int64_t)r * p.n + c;
            const void *const *grads = p.grads + z * p.R;
            float m[8];
            if (p.vec && left >= 8) {
                load8(p.momentum[z], at, 8, false, m);
                if (p.bf16)
                    fold_vec<true>(grads, p.R, at, u);
                else
                    fold_vec<false>(grads, p.R, at, u);
            } else {
                load8(p.momentum[z], at, left, false, m);
                load8(grads[0], at, left, p.bf16, u);
                for (int q = 1; q < p.R; q++) {
                    float o[8];
                    load8(grads[q], at, left, p.bf16, o);
#pragma unroll
                    for (int k = 0; k < 8; k++)
                        u[k] = __fadd_rn(u[k], o[k]);
                }
            }
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

// x16 = u / (||u||_F + eps); inv[z]: that factor.
__global__ void __launch_bounds__(kStartThreads) scale_kernel(const float *x32, uint16_t *x16, const float *partial,
                                                              int parts, float eps, int64_t count, float *inv_out)
{
    __shared__ float sh[kStartThreads / 32];
    launch_wait();
    launch_next();
    const int z = blockIdx.y;
    float sq = 0.0f;
    for (int i = threadIdx.x; i < parts; i += kStartThreads)
        sq += partial[z * kMaxParts + i];
    sq = block_sum(sq, sh);
    const float inv = 1.0f / (sqrtf(sq) + eps);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        inv_out[z] = inv;
    const float *src = x32 + z * count;
    uint16_t *dst = x16 + z * count;
    const int64_t step = (int64_t)gridDim.x * kStartThreads * 8;
    for (int64_t i = ((int64_t)blockIdx.x * kStartThreads + threadIdx.x) * 8; i < count; i += step) {
        float v[8];
        load8(src, i, 8, false, v);
        uint4 u;
        uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
        for (int k = 0; k < 4; k++)
            w[k] = pack_f16(v[2 * k] * inv, v[2 * k + 1] * inv);
        *reinterpret_cast<uint4 *>(dst + i) = u;
    }
}

// S, or (kPoly) P = b S + c S^2 - d I, in fp16; both triangles where one is
// multiplied. Strides are multiples of 16, so groups of 8 and pairs of rows
// stay inside a padded row.
template <bool kPoly>
struct SquareEpi {
    static constexpr int kLeastTN = 64;
    struct Params {
        uint16_t *out;
        const uint16_t *from;  // S
        int64_t ld, stride;
        float b, c;
        float *trace;          // [batch][groups], of S
        int groups;
    };
    struct Pre {
        uint4 s[kPoly ? 8 : 1];  // this lane's groups of a unit of S
        float shift;
    };
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int unit, Pre &pre)
    {
        if (!kPoly)
            return;
        if (unit == x.part)
            pre.shift = shift_of(p.trace + x.z * p.groups, x.M, p.b, p.c, x.lane);
        const int rows = x.M - x.group_row(0);
        const uint16_t *from = p.from + x.z * p.stride + x.group_row(0) * p.ld + x.unit_col(unit);
        const bool in = x.unit_col(unit) < x.N;
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i * 4 < rows && in)
                pre.s[kPoly ? i : 0] = *reinterpret_cast<const uint4 *>(from + i * 4 * p.ld);
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const CUtensorMap *map)
    {
        uint16_t *out = p.out + x.z * p.stride;
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts) {
            uint4 own[kPoly ? 8 : 1];  // the thread's own row of the unit
            if (kPoly) {
                x.stage_free();
#pragma unroll
                for (int i = 0; i < 8; i++)
                    *x.group(i) = pre.s[kPoly ? i : 0];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; i++)
                    own[kPoly ? i : 0] = *x.piece(x.lane, i);
                __syncwarp();
                if (u + kParts < x.units())
                    fetch(p, x, u + kParts, pre);
            }
            auto finish = [&](int h, float(&v)[32]) {
                if (kPoly) {
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const uint4 &q = own[kPoly ? h * 4 + j / 4 : 0];
                        const uint32_t w = j % 4 == 0 ? q.x : j % 4 == 1 ? q.y : j % 4 == 2 ? q.z : q.w;
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                        v[2 * j] = fmaf(p.c, v[2 * j], p.b * f.x);
                        v[2 * j + 1] = fmaf(p.c, v[2 * j + 1], p.b * f.y);
                    }
                }
                if (x.col + (u * 2 + h) * 32 == x.row - x.lane) {  // the diagonal's chunk
                    if (kPoly) {
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            v[j] -= x.lane == j ? pre.shift : 0.0f;
                    } else {
                        const float sum = diagonal_sum(v, x.lane);
                        if (x.lane == 0 && x.row < x.M)
                            p.trace[x.z * p.groups + x.row / 32] = sum;
                    }
                }
                if (!x.mirror)
                    return;
                // the transposed elements: two rows' on a pair of lanes make
                // one 32-bit store, of column j on the even and j + 1 on the
                // odd lane
                const int odd = x.lane & 1, row = x.row & ~1, col = x.col + (u * 2 + h) * 32 + odd;
                const int cols = row < x.M ? x.N - col : 0;
                uint16_t *across = out + col * p.ld + row;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                    const uint32_t pair = odd ? pack_f16(other, v[j + 1]) : pack_f16(v[j], other);
                    if (j < cols)
                        *reinterpret_cast<uint32_t *>(across + j * p.ld) = pair;
                }
            };
            x.emit_map<false>(map, u, finish);
        }
    }
};

// S from the parts of its sum: a block has 32 rows, and their diagonal's sum.
__global__ void __launch_bounds__(256) join_square_kernel(const float *parts, const int *splits_used, int k, int64_t ld,
                                                          uint16_t *out, int64_t stride, float *trace, int groups)
{
    __shared__ float diagonal[32];
    launch_wait();
    launch_next();
    const int splits = *splits_used, z = blockIdx.y, row0 = blockIdx.x * 32;
    const float *src = parts + (int64_t)z * splits * k * ld;
    const int quads = (k + 3) / 4;  // groups of 4 columns
    if (threadIdx.x < 32)
        diagonal[threadIdx.x] = 0.0f;
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * quads; i += 256) {
        const int r = i / quads, row = row0 + r, c = (i - r * quads) * 4;
        if (row >= k)
            break;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int q = 0; q < splits; q++) {
            const float4 f = *reinterpret_cast<const float4 *>(src + ((int64_t)q * k + row) * ld + c);
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
        }
        *reinterpret_cast<uint2 *>(out + z * stride + row * ld + c) = four_16<false>(v);
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (c + j == row)
                diagonal[r] = v[j];
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        float s = diagonal[threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0)
            trace[z * groups + blockIdx.x] = s;
    }
}

// x = (a + d) x + (P x), x the fp32 one. What becomes of it:
//   kKeep    fp32 in place, and the next step's fp16 operand
//   kOut     the result, in bf16
//   kMaster  w = w decay - lr x, and the bf16 parameter
enum class Then { kKeep, kOut, kMaster };

struct StepParams {
    float *x32;
    const float *inv;  // the first step's factor of x32, per matrix; NULL: 1
    int64_t ld, stride;
    float a, b, c;
    const float *trace;
    int groups, k;
    uint16_t *x16;
    uint16_t *out;
    int64_t ldo, out_stride, n;
    float decay, lr;
    float *master[kMuonMaxMats];
    uint16_t *param[kMuonMaxMats];
};

template <Then kThen>
struct StepEpi {
    static constexpr int kLeastTN = 64;
    static constexpr bool kAhead = kThen != Then::kMaster;  // registers: it has twice the reads
    using Params = StepParams;
    static constexpr bool kMaster = kThen == Then::kMaster;
    struct Pre;
    static __device__ __forceinline__ void carry(const Pre &from, Pre &to) { to.a = from.a; }
    struct Pre {
        float a;
        float4 x[8];
    };
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int chunk, Pre &pre)
    {
        const int rows = x.M - x.group_row(0), left = x.N - x.group_col(chunk);
        if (chunk == x.part) {
            pre.a = p.a + shift_of(p.trace + x.z * p.groups, p.k, p.b, p.c, x.lane);
            if (p.inv)
                pre.a *= p.inv[x.z];
        }
        const float *from = p.x32 + x.z * p.stride + x.group_row(0) * p.ld + x.group_col(chunk);
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i * 4 < rows && left > 0)
                pre.x[i] = *reinterpret_cast<const float4 *>(from + i * 4 * p.ld);
    }
    template <class G>
    static __device__ __forceinline__ void chunk(const Params &p, const Slot &x, int c, Pre &pre, G staged)
    {
        const int rows = x.M - x.group_row(0), col = x.group_col(c), left = x.N - col;
        const int64_t at = x.z * p.stride + x.group_row(0) * p.ld + col;
        const int64_t to = x.group_row(0) * (kThen == Then::kOut ? p.ldo : p.n) + col;
        float mine[32];
        // the master's elements are read once the accumulator's registers are free
        float w[kMaster ? 8 : 1][4];
        auto read_master = [&] {
            staged();
            if (kMaster) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (i * 4 < rows && left > 0)
                        get4_f32(p.master[x.z] + to + i * 4 * p.n, w[kMaster ? i : 0], left);
            }
        };
        x.across<false>(c, mine, [&](int i, float(&v)[4]) {
            if (i * 4 >= rows || left <= 0)
                return;
            v[0] = fmaf(pre.a, pre.x[i].x, v[0]);
            v[1] = fmaf(pre.a, pre.x[i].y, v[1]);
            v[2] = fmaf(pre.a, pre.x[i].z, v[2]);
            v[3] = fmaf(pre.a, pre.x[i].w, v[3]);
            if (kThen == Then::kKeep) {
                *reinterpret_cast<float4 *>(p.x32 + at + i * 4 * p.ld) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<uint2 *>(p.x16 + at + i * 4 * p.ld) = four_16<false>(v);
            } else if (kThen == Then::kOut) {
                put4_16<true>(p.out + x.z * p.out_stride + to + i * 4 * p.ldo, v, left);
            } else {
#pragma unroll
                for (int k = 0; k < 4; k++)
                    v[k] = fmaf(-p.lr, v[k], w[kMaster ? i : 0][k] * p.decay);
                put4_f32(p.master[x.z] + to + i * 4 * p.n, v, left);
                if (p.param[x.z])
                    put4_16<true>(p.param[x.z] + to + i * 4 * p.n, v, left);
            }
        }, read_master);
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const CUtensorMap *)
    {
        finish_tile<StepEpi>(p, x, pre);
    }
};

// steps = 0: the scaled input is the result.
struct FinishParams {
    const float *x32, *inv;
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
    launch_wait();
    launch_next();
    const int z = blockIdx.y;
    const float *x = p.x32 + (int64_t)z * p.m * p.ld;
    for (int64_t i = (int64_t)blockIdx.x * kStartThreads + threadIdx.x; i < (int64_t)p.m * p.n;
         i += (int64_t)gridDim.x * kStartThreads) {
        const int64_t r = i / p.n, c = i - r * p.n;
        const float v = x[r * p.ld + c] * p.inv[z];
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

}  // namespace

int64_t schulz_workspace(int64_t batch, int64_t m, int64_t n) { return schulz_plan(batch, m, n, nullptr).bytes; }

fsdp_status launch_newton_schulz(const SchulzArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool muon = a.grads != nullptr;
    const int sms = device_sms(dev);
    const int64_t team = team_clocks(a, dev);
    if (team >= 0 && team < product_clocks(a, sms))
        return launch_team(a, workspace, dev, stream);
    const SchulzPlan q = schulz_plan(a.batch, a.m, a.n, workspace);
    const int batch = (int)a.batch, m = (int)a.m, n = (int)a.n;
    fsdp_status st;

    StartParams sp{};
    sp.m = m;
    sp.n = n;
    sp.groups = (int)(q.ldx / 8);
    sp.ldx = q.ldx;
    const int64_t need = (a.m * sp.groups + kStartThreads - 1) / kStartThreads;
    const int64_t fill = (6 * sms + a.batch - 1) / a.batch;
    int64_t parts = need < fill ? need : fill;
    parts = parts < kMaxParts ? parts : kMaxParts;
    sp.x32 = q.x32;
    sp.partial = q.partial;
    sp.bf16 = a.dtype == FSDP_BF16;
    const dim3 grid((unsigned)parts, batch);
    if (muon) {
        sp.R = a.R;
        sp.nesterov = a.nesterov;
        sp.inv_r = 1.0f / (float)a.R;
        sp.mu = a.mu;
        uintptr_t low = (uintptr_t)(a.n * (sp.bf16 ? 2 : 4));
        for (int i = 0; i < batch; i++) {
            sp.momentum[i] = a.momentum[i];
            low |= reinterpret_cast<uintptr_t>(a.momentum[i]);
        }
        for (int i = 0; i < batch * a.R; i++) {
            sp.grads[i] = a.grads[i];
            low |= reinterpret_cast<uintptr_t>(a.grads[i]);
        }
        sp.vec = (low & 15u) == 0;
        st = launch("muon (start)", start_kernel<true>, grid, kStartThreads, 0, s, 1, sp);
    } else {
        sp.g = a.g;
        sp.ldg = a.ldg;
        sp.g_stride = a.g_stride;
        st = launch("newton_schulz (start)", start_kernel<false>, grid, kStartThreads, 0, s, 1, sp);
    }
    if (st != FSDP_OK)
        return st;
    if ((st = launch("newton_schulz (scale)", scale_kernel, grid, kStartThreads, 0, s, 1, q.x32, q.x16[0], q.partial,
                     parts, a.eps, a.m * q.ldx, q.inv)) != FSDP_OK)
        return st;

    if (a.steps == 0) {
        FinishParams fp{};
        fp.x32 = q.x32;
        fp.inv = q.inv;
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
        return launch("newton_schulz (result)", muon ? finish_kernel<true> : finish_kernel<false>, grid, kStartThreads,
                      0, s, 1, fp);
    }

    const bool wide = a.m <= a.n;
    const int64_t xs = a.m * q.ldx, ks = q.k * q.ldk;
    StepParams ep{};
    ep.x32 = q.x32;
    ep.ld = q.ldx;
    ep.stride = xs;
    ep.a = a.a, ep.b = a.b, ep.c = a.c;
    ep.trace = q.trace;
    ep.groups = (int)q.groups;
    ep.k = (int)q.k;
    ep.out = static_cast<uint16_t *>(a.out);
    ep.ldo = a.ldo;
    ep.out_stride = a.out_stride;
    ep.n = a.n;
    ep.decay = a.decay;
    ep.lr = a.lr;
    for (int i = 0; muon && i < batch; i++) {
        ep.master[i] = a.master[i];
        ep.param[i] = a.param_out ? static_cast<uint16_t *>(a.param_out[i]) : nullptr;
    }
    for (int step = 0; step < a.steps; step++) {
        const Operand x{q.x16[step % 2], a.n, a.m, q.ldx, xs};
        const Operand gram{q.s, q.k, q.k, q.ldk, ks}, poly{q.p, q.k, q.k, q.ldk, ks};
        Shape sq = square_shape(q.k, wide ? n : m, batch, sms, false);
        const typename SquareEpi<false>::Params e1{q.s, nullptr, q.ldk, ks, 0.0f, 0.0f, q.trace, (int)q.groups};
        const typename SquareEpi<true>::Params e2{q.p, q.s, q.ldk, ks, a.b, a.c, q.trace, (int)q.groups};
        if (q.splits > 1) {
            sq.sym = sq.square = 0;
            sq.splits = q.splits;
            sq.splits_out = q.splits_used;
            const PartEpi::Params pe{q.parts, q.ldk};
            st = wide ? product<false, false, PartEpi>(sq, x, x, false, pe, dev, s, "newton_schulz (S, parts)")
                      : product<true, true, PartEpi>(sq, x, x, false, pe, dev, s, "newton_schulz (S, parts)");
            if (st == FSDP_OK)
                st = launch("newton_schulz (S, sum)", join_square_kernel, dim3((unsigned)q.groups, batch), 256, 0, s, 1,
                            q.parts, q.splits_used, q.k, q.ldk, q.s, ks, q.trace, q.groups);
        } else {
            st = wide ? product<false, false, SquareEpi<false>>(sq, x, x, false, e1, dev, s, "newton_schulz (S)", &gram)
                      : product<true, true, SquareEpi<false>>(sq, x, x, false, e1, dev, s, "newton_schulz (S)", &gram);
        }
        if (st != FSDP_OK)
            return st;
        sq = square_shape(q.k, q.k, batch, sms, true);
        if ((st = product<false, false, SquareEpi<true>>(sq, gram, gram, false, e2, dev, s, "newton_schulz (P)",
                                                         &poly)) != FSDP_OK)
            return st;
        Shape up{};
        up.M = m;
        up.N = n;
        up.K = (int)q.k;
        up.batch = batch;
        up.epi_bytes = kStepBytes;
        ep.inv = step == 0 ? q.inv : nullptr;
        ep.x16 = q.x16[(step + 1) % 2];
        auto update = [&](auto epi) {
            using E = decltype(epi);
            // wide: P x, x with its columns adjacent; tall: x P, P symmetric
            return wide ? product<false, true, E>(up, poly, x, false, ep, dev, s, "newton_schulz (x)")
                        : product<false, false, E>(up, x, poly, false, ep, dev, s, "newton_schulz (x)");
        };
        st = step + 1 < a.steps ? update(StepEpi<Then::kKeep>{})
             : muon             ? update(StepEpi<Then::kMaster>{})
                                : update(StepEpi<Then::kOut>{});
        if (st != FSDP_OK)
            return st;
    }
    return FSDP_OK;
}

cudaError_t muon_wait_timeouts(unsigned long long *n) { return wait::wait_timeouts(n); }

}  // namespace fsdp
